"""Global gradient norm and clipping over many tensors against fp64."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import torch
    import gpt_pretraining_step_decoder_b200 as g
    assert torch.cuda.is_available()
    return g


def call(g, grads, outs, max_norm, stream=None):
    import torch
    n = g.grad_clip_workspace_bytes(len(grads))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    norm = torch.full((1,), -1.0, device="cuda")
    g.grad_clip(grads, outs, max_norm, norm, ws, n, stream)
    torch.cuda.synchronize()
    return norm


def make(sizes, dtypes, seed=0, scale=1.0, offset=0):
    import torch
    gen = torch.Generator().manual_seed(seed)
    out = []
    for n, d in zip(sizes, dtypes):
        dt = torch.float32 if d == "f32" else torch.bfloat16
        buf = torch.zeros(n + offset, dtype=dt, device="cuda")
        t = buf[offset:]
        t.copy_((torch.randn(n, generator=gen) * scale).to(dt))
        out.append(t)
    return out


def reference(grads, max_norm):
    vals = [t.double().cpu().numpy() for t in grads]
    norm = float(np.sqrt(sum((v * v).sum() for v in vals)))
    coef = min(1.0, max_norm / (norm + 1e-6)) if max_norm > 0 else 1.0
    return norm, [v * coef for v in vals]


def check(g, got, ref, exact=False):
    import torch
    for t, v in zip(got, ref):
        # the coefficient and the product are each rounded to fp32, a bf16 result once more
        rel = 0.0 if exact else 2 * 2.0 ** -24 + (2.0 ** -8 if t.dtype == torch.bfloat16 else 0.0)
        assert (np.abs(t.double().cpu().numpy() - v) <= rel * 1.0001 * np.abs(v) + 2.0 ** -140).all()


SETS = {
    "one": ([1], ["f32"]),
    "odd": ([0, 1, 3, 0, 7, 8191, 8192, 8193, 100003, 0], ["f32", "bf16"] * 5),
    "bf16": ([16384 * 3 + 5, 17, 2], ["bf16"] * 3),
    "large": ([40_000_001, 5, 3_000_000], ["f32", "f32", "bf16"]),
    "many": ([37 * (i % 5) + 1 for i in range(150)], ["f32" if i % 3 else "bf16" for i in range(150)]),
    "tables": ([i % 7 for i in range(2500)], ["f32"] * 2500),
}


@pytest.mark.parametrize("max_norm", [0.0, 0.5, 1e9])
@pytest.mark.parametrize("name", SETS)
def test_norm_and_clip(g, name, max_norm):
    sizes, dtypes = SETS[name]
    grads = make(sizes, dtypes)
    norm, ref = reference(grads, max_norm)
    outs = [t.clone() * 0 - 3 for t in grads]
    keep = [t.clone() for t in grads]
    got = call(g, grads, outs, max_norm)
    assert abs(got.item() - norm) <= 2.0 ** -23 * norm
    check(g, outs, ref, exact=max_norm in (0.0, 1e9))
    for a, b in zip(grads, keep):
        assert (a == b).all()                         # inputs are left alone
    got2 = call(g, grads, None, max_norm)             # in place: the same values
    assert got2.item() == got.item()
    for a, b in zip(grads, outs):
        assert (a == b).all()
    assert g.ngram_sync_status() == g.GPT_OK


@pytest.mark.parametrize("offset", [1, 3])
def test_unaligned_tensors_and_neighbours(g, offset):
    """Views that start off 16-byte boundaries; what lies next to them stays."""
    import torch
    buf = torch.randn(50_000, device="cuda")
    keep = buf.clone()
    grads = [buf[offset:20_001], buf[20_003:20_003], buf[20_010:49_990]]
    norm, ref = reference(grads, 1.0)
    got = call(g, grads, None, 1.0)
    assert abs(got.item() - norm) <= 2.0 ** -23 * norm
    check(g, grads, ref)
    assert (buf[:offset] == keep[:offset]).all() and (buf[49_990:] == keep[49_990:]).all()
    assert (buf[20_001:20_010] == keep[20_001:20_010]).all()


@pytest.mark.parametrize("scale", [1e-30, 1e-22, 1e25, 1e33])
def test_squares_beyond_fp32(g, scale):
    grads = make([1000, 333], ["f32", "f32"], scale=scale)
    norm, ref = reference(grads, scale)
    got = call(g, grads, None, scale)
    assert abs(got.item() - norm) <= 2.0 ** -23 * norm
    check(g, grads, ref)
    assert g.ngram_sync_status() == g.GPT_OK


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_norm_that_is_not_finite(g, bad):
    import torch
    grads = make([1000, 70], ["f32", "bf16"])
    grads[1][3] = bad
    keep = [t.clone() for t in grads]
    got = call(g, grads, None, 1.0)
    assert not torch.isfinite(got).any()
    for a, b in zip(grads, keep):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))   # left unscaled
    assert g.ngram_sync_status() == g.GPT_ERR_NONFINITE
    assert g.ngram_sync_status() == g.GPT_OK


def test_no_tensors_and_all_zero(g):
    import torch
    assert call(g, [], None, 1.0).item() == 0.0
    z = torch.zeros(1000, device="cuda")
    assert call(g, [z], None, 1.0).item() == 0.0 and not z.any()


def test_captured_clip_reads_new_values(g):
    import torch
    grads = make([5000, 1234], ["f32", "bf16"])
    outs = [torch.empty_like(t) for t in grads]
    n = g.grad_clip_workspace_bytes(2)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    norm = torch.zeros(1, device="cuda")
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    g.grad_clip(grads, outs, 1.0, norm, ws, n, st)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        g.grad_clip(grads, outs, 1.0, norm, ws, n, st)
    for t in grads:
        t.mul_(0.001)
    want, ref = reference(grads, 1.0)
    graph.replay()
    torch.cuda.synchronize()
    assert abs(norm.item() - want) <= 2.0 ** -23 * want
    check(g, outs, ref)


def test_python_checks(g):
    import torch
    t = torch.zeros(4, 6, device="cuda")
    ws = torch.empty(g.grad_clip_workspace_bytes(1), dtype=torch.uint8, device="cuda")
    for grads, outs in (([t.T], None), ([t.half()], None), ([t], [t.bfloat16()]), ([t], [t[:2].clone()]), ([t], [t, t])):
        with pytest.raises(ValueError):
            g.grad_clip(grads, outs, 1.0, None, ws, ws.numel())
