"""Pins of the cross-entropy oracle: torch's own loss and autograd in fp64,
central differences, ln V of equal logits, ignored targets."""

import numpy as np
import pytest

from oracle import linear_ce as ce


def case(seed=0, N=7, V=11, d=5):
    rng = np.random.default_rng(seed)
    x, w = rng.standard_normal((N, d)), rng.standard_normal((V, d))
    t = rng.integers(0, V, N)
    t[2] = -1
    return x, w, t


@pytest.mark.parametrize("softcap", [0.0, 2.5])
def test_matches_torch(softcap):
    import torch
    x, w, t = case()
    xt, wt = (torch.tensor(a, requires_grad=True) for a in (x, w))
    z = xt @ wt.T
    if softcap:
        z = softcap * torch.tanh(z / softcap)
    tok = torch.nn.functional.cross_entropy(z, torch.tensor(t), ignore_index=-1, reduction="none")
    loss = torch.nn.functional.cross_entropy(z, torch.tensor(t), ignore_index=-1)
    l, tk, lse = ce.forward(x, w, t, softcap)
    np.testing.assert_allclose(l, loss.item(), rtol=1e-13)
    np.testing.assert_allclose(tk, tok.detach().numpy(), rtol=1e-12, atol=1e-14)
    np.testing.assert_allclose(lse, torch.logsumexp(z, 1).detach().numpy(), rtol=1e-13)
    (1.7 * loss).backward(retain_graph=True)
    dx, dw = ce.backward(x, w, t, softcap, dloss=1.7)
    np.testing.assert_allclose(dx, xt.grad.numpy(), rtol=1e-11, atol=1e-14)
    np.testing.assert_allclose(dw, wt.grad.numpy(), rtol=1e-11, atol=1e-14)
    xt.grad = wt.grad = None
    dtok = np.random.default_rng(3).standard_normal(len(x))
    (tok * torch.tensor(dtok)).sum().backward()
    dx, dw = ce.backward(x, w, t, softcap, dtok=dtok)
    np.testing.assert_allclose(dx, xt.grad.numpy(), rtol=1e-11, atol=1e-14)
    np.testing.assert_allclose(dw, wt.grad.numpy(), rtol=1e-11, atol=1e-14)


@pytest.mark.parametrize("softcap", [0.0, 2.5])
def test_central_differences(softcap):
    x, w, t = case(4)
    dx, dw = ce.backward(x, w, t, softcap)
    h = 1e-6
    for a, g in ((x, dx), (w, dw)):
        for idx in ((0, 0), (3, 2), (5, 4)):
            keep = a[idx]
            a[idx] = keep + h
            up = ce.forward(x, w, t, softcap)[0]
            a[idx] = keep - h
            down = ce.forward(x, w, t, softcap)[0]
            a[idx] = keep
            assert abs((up - down) / (2 * h) - g[idx]) < 1e-8


def test_closed_form_and_ignored():
    x, w, t = case()
    assert abs(ce.forward(np.zeros_like(x), w, t)[0] - np.log(11)) < 1e-14
    l, tok, _ = ce.forward(x, w, np.full(7, -1))
    assert l == 0 and not tok.any()
    assert not ce.backward(x, w, np.full(7, -1))[0].any()
    t[1] = 11                                      # past the vocabulary: ignored as well
    assert ce.forward(x, w, t)[1][1] == 0
