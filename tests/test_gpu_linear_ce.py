"""Cross entropy without stored logits on the GPU against the fp64 oracle.

Tolerances, elementwise: a logit is an fp32 sum of d exact products, so it is
off by at most ez = (d + 16) 2^-23 sum |x||w|; lse moves no more than the
largest ez, plus the exponentials' and the sums' rounding (a few fp32 steps of
the exponents, which are as large as the logits); the softcap's tanh from an
approximate exponential adds cap 2^-19.  dz is off by those, relative to p g,
and in bf16 mode by half a bf16 step (2^-8 of its value); dx and dW by the
sums of that, and half a step of their own type."""

import numpy as np
import pytest

from oracle import linear_ce as ce

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import torch
    import gpt_pretraining_step_decoder_b200 as g
    assert torch.cuda.is_available()
    return g


class Case:
    def __init__(self, N, V, d, dtype="bf16", softcap=0.0, seed=0, ignored=0.2, spread=2.0, ldx=None, ldw=None):
        import torch
        rng = np.random.default_rng(seed + N + V + d)
        self.N, self.V, self.d, self.cap, self.dtype = N, V, d, softcap, dtype
        self.ldx, self.ldw = ldx or d, ldw or d
        self.dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        x = torch.from_numpy(rng.standard_normal((N, d))).to(self.dt)
        w = torch.from_numpy(rng.standard_normal((V, d)) * spread / np.sqrt(d)).to(self.dt)
        self.x, self.w = x.double().numpy(), w.double().numpy()
        self.t = rng.integers(0, V, N).astype(np.int32)
        self.t[rng.random(N) < ignored] = -1
        self.xd = self.place(x, self.ldx)
        self.wd = self.place(w, self.ldw)
        self.td = torch.from_numpy(self.t).cuda()
        self.code = 1 if dtype == "bf16" else 0

    def place(self, t, ld):
        import torch
        buf = torch.full((t.shape[0], ld), float("nan"), dtype=t.dtype, device="cuda")
        buf[:, :t.shape[1]] = t.cuda()
        return buf

    # ------------------------------------------------------------- bounds
    def ez(self):
        return (self.d + 16) * 2.0 ** -23 * (np.abs(self.x) @ np.abs(self.w).T) + (self.cap * 2.0 ** -19)

    def lse_tol(self):
        z = np.abs(ce.logits(self.x, self.w, self.cap)).max(axis=1)
        return self.ez().max(axis=1) + 2.0 ** -22 * (8 + 3 * z)

    def forward(self, g, piece=0, stream=None, ws=None):
        import torch
        N, V, d = self.N, self.V, self.d
        n = g.linear_ce_workspace_bytes(N, V, d, self.code, 0, piece)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda") if ws is None else ws
        loss, tok, lse = (torch.full((k,), 77.0, device="cuda") for k in (1, N, N))
        g.linear_ce_forward(self.xd, self.ldx, self.wd, self.ldw, self.code, N, V, d, self.td, self.cap, loss, tok, lse, ws,
                            n, stream, piece)
        torch.cuda.synchronize()
        return loss, tok, lse

    def backward(self, g, piece=0, dloss=None, dtok=None, dx=True, dw=True, dw_dtype=None, beta=0, dw0=None, pad=0, lse=None):
        import torch
        N, V, d = self.N, self.V, self.d
        n = g.linear_ce_workspace_bytes(N, V, d, self.code, 1, piece)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        if lse is None:
            lse = torch.from_numpy(ce.forward(self.x, self.w, self.t, self.cap)[2].astype(np.float32)).cuda()
        dw_dtype = self.code if dw_dtype is None else dw_dtype
        gx = torch.full((N, d + pad), 5.0, dtype=self.dt, device="cuda") if dx else None
        gw = None
        if dw:
            gw = torch.full((V, d + pad), 5.0, dtype=torch.bfloat16 if dw_dtype else torch.float32, device="cuda")
            if dw0 is not None:
                gw[:, :d] = dw0
        f = lambda v: None if v is None else torch.tensor(v, dtype=torch.float32, device="cuda")  # noqa: E731
        g.linear_ce_backward(self.xd, self.ldx, self.wd, self.ldw, self.code, N, V, d, self.td, self.cap, lse, f(dloss),
                             f(dtok), gx, d + pad, gw, d + pad, dw_dtype, beta, ws, n, None, piece)
        torch.cuda.synchronize()
        return gx, gw

    def check_forward(self, got):
        loss, tok, lse = got
        l0, t0, s0 = ce.forward(self.x, self.w, self.t, self.cap)
        tol = self.lse_tol()
        assert (np.abs(lse.double().cpu().numpy() - s0) <= tol).all(), np.abs(lse.cpu().numpy() - s0).max()
        tt = tol + self.ez().max(axis=1) + 2.0 ** -23 * (np.abs(s0) + np.abs(t0))
        assert (np.abs(tok.double().cpu().numpy() - t0) <= tt).all()
        assert (tok.cpu().numpy()[self.t < 0] == 0).all()
        assert abs(loss.item() - l0) <= tt.max() + 2.0 ** -23 * abs(l0)

    def check_backward(self, gx, gw, dloss=1.0, dtok=None, base=0.0):
        import torch
        dz = ce.dlogits(self.x, self.w, self.t, self.cap, dloss, dtok)
        valid = (self.t >= 0) & (self.t < self.V)
        gr = np.abs(np.where(valid, dloss / max(1, valid.sum()) if dtok is None else dtok, 0.0))[:, None]
        p = np.exp(ce.logits(self.x, self.w, self.cap) - ce.forward(self.x, self.w, self.t, self.cap)[2][:, None])
        edz = p * gr * 2 * (self.ez() + self.lse_tol()[:, None]) + 2.0 ** -21 * np.abs(dz)
        if self.cap:  # the slope 1 - (z / cap)^2
            onehot = np.zeros_like(p)
            onehot[np.nonzero(valid)[0], self.t[valid]] = 1
            edz += (p + onehot) * gr * 2.0 ** -17
        if self.dtype == "bf16":
            edz += 2.0 ** -8 * (np.abs(dz) + edz) + 2.0 ** -133
        for got, a, b, k in ((gx, dz, self.w, self.V), (gw, dz.T, self.x, self.N)):
            if got is None:
                continue
            e = edz if a is dz else edz.T
            ref = a @ b
            tol = e @ np.abs(b) + (k + 16) * 2.0 ** -22 * ((np.abs(a) + e) @ np.abs(b))
            if a is not dz:
                ref = ref + base
                tol = tol + 2.0 ** -23 * (np.abs(ref) + np.abs(base))
            tol += (2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -23) * (np.abs(ref) + tol)
            err = np.abs(got.double().cpu().numpy()[:, :self.d] - ref)
            assert (err <= tol + 1e-30).all(), (err.max(), np.argwhere(err > tol)[:3])


SHAPES = [(1, 64, 8), (1, 1, 8), (33, 1000, 64), (5000, 300, 64), (70, 300, 1096), (300, 520, 2056), (128, 256, 128), (130, 513, 72), (257, 4160, 128), (300, 5003, 256), (5, 50257, 64)]


@pytest.mark.parametrize("softcap", [0.0, 15.0])
@pytest.mark.parametrize("N,V,d", SHAPES)
def test_forward_bf16(g, N, V, d, softcap):
    c = Case(N, V, d, softcap=softcap)
    c.check_forward(c.forward(g))
    assert g.ngram_sync_status() == g.GPT_OK


@pytest.mark.parametrize("pairs", [1, 0])
@pytest.mark.parametrize("piece", [0, 64, 320])
@pytest.mark.parametrize("softcap", [0.0, 15.0])
@pytest.mark.parametrize("N,V,d", [s for s in SHAPES if s[1] < 50000])
def test_backward_bf16(g, N, V, d, softcap, piece, pairs):
    if piece == 64 and V > 1000 or (pairs == 0 and piece):
        pytest.skip("covered by the other pieces")
    g.gptx_set_gemm_cta_pairs(pairs)
    try:
        c = Case(N, V, d, softcap=softcap)
        c.check_backward(*c.backward(g, piece))
        c.check_forward(c.forward(g))
    finally:
        g.gptx_set_gemm_cta_pairs(1)
    assert g.ngram_sync_status() == g.GPT_OK


@pytest.mark.parametrize("piece", [0, 64])
@pytest.mark.parametrize("softcap", [0.0, 15.0])
@pytest.mark.parametrize("N,V,d", [(1, 1, 1), (1, 7, 3), (33, 100, 17), (65, 513, 64), (130, 300, 129), (513, 2300, 130),
                                   (1000, 1300, 72)])
def test_fp32(g, N, V, d, softcap, piece):
    c = Case(N, V, d, "f32", softcap)
    c.check_forward(c.forward(g, piece))
    c.check_backward(*c.backward(g, piece))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides_and_outputs_asked_for(g, dtype):
    c = Case(70, 300, 64, dtype, ldx=72, ldw=80)
    c.check_forward(c.forward(g))
    gx, gw = c.backward(g, dloss=0.5, pad=8)
    c.check_backward(gx, gw, dloss=0.5)
    assert (gx[:, 64:] == 5.0).all() and (gw[:, 64:] == 5.0).all()      # what lies between the rows stays
    only_x, none = c.backward(g, dloss=0.5, dw=False)
    assert none is None and (only_x == gx[:, :64]).all()
    none, only_w = c.backward(g, dloss=0.5, dx=False)
    assert none is None and (only_w == gw[:, :64]).all()


@pytest.mark.parametrize("piece", [0, 128])
def test_fp32_weight_gradient_accumulates(g, piece):
    import torch
    c = Case(100, 400, 64)
    base = np.random.default_rng(1).standard_normal((400, 64)).astype(np.float32) * 1e-3
    gx, gw = c.backward(g, piece, dw_dtype=0)
    c.check_backward(gx, gw)
    gx, gw = c.backward(g, piece, dw_dtype=0, beta=1, dw0=torch.from_numpy(base).cuda())
    c.check_backward(gx, gw, base=base.astype(np.float64))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_per_token_gradients(g, dtype):
    c = Case(90, 200, 64, dtype, softcap=15.0)
    dtok = np.random.default_rng(2).standard_normal(90).astype(np.float32)
    c.check_backward(*c.backward(g, dtok=dtok), dtok=dtok.astype(np.float64))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_target_ignored(g, dtype):
    c = Case(40, 200, 64, dtype, ignored=1.1)
    loss, tok, lse = c.forward(g)
    assert loss.item() == 0.0 and not tok.any()
    gx, gw = c.backward(g)
    assert not gx.any() and not gw.any()
    assert g.ngram_sync_status() == g.GPT_OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_targets_out_of_range(g, dtype):
    import torch
    c = Case(40, 200, 64, dtype)
    c.t[[3, 20]] = [200, -7]
    c.td = torch.from_numpy(c.t).cuda()
    got = c.forward(g)
    assert g.ngram_sync_status() == g.GPT_ERR_INPUT
    c.check_forward(got)
    gx, gw = c.backward(g)
    assert g.ngram_sync_status() == g.GPT_ERR_INPUT
    c.check_backward(gx, gw)
    assert not gx[3].any() and not gx[20].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_logits_and_a_hopeless_target(g, dtype):
    """Logits in the thousands: no overflow, the loss as large as they are."""
    c = Case(50, 300, 64, dtype, spread=2000.0)
    c.check_forward(c.forward(g))
    assert g.ngram_sync_status() == g.GPT_OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_masked_row_of_nan(g, dtype):
    """A NaN hidden state in an ignored row: the mean and the other rows do not see it."""
    c = Case(60, 300, 64, dtype)
    c.t[7] = -1
    c.td[7] = -1
    c.xd[7, :c.d] = float("nan")
    loss, tok, lse = c.forward(g)
    l0, t0, _ = ce.forward(c.x, c.w, c.t, c.cap)
    assert np.isnan(lse[7].item()) and abs(loss.item() - l0) < 1e-5 * l0 and tok[7].item() == 0
    gx, _ = c.backward(g, dw=False)
    assert not gx[7].any() and np.isfinite(gx.float().cpu().numpy()).all()
    assert g.ngram_sync_status() == g.GPT_OK
    c.td[7] = 3                                    # and unmasked it is reported
    assert np.isnan(c.forward(g)[0].item())
    assert g.ngram_sync_status() == g.GPT_ERR_NONFINITE


def test_no_rows(g):
    import torch
    c = Case(1, 200, 64)
    ws = torch.empty(g.linear_ce_workspace_bytes(0, 200, 64, 1, 0), dtype=torch.uint8, device="cuda")
    ws = torch.empty(max(256, ws.numel()), dtype=torch.uint8, device="cuda")
    loss = torch.full((1,), 9.0, device="cuda")
    g.linear_ce_forward(None, 64, c.wd, 64, 1, 0, 200, 64, None, 0.0, loss, None, None, ws, ws.numel())
    dw = torch.full((200, 72), 9.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(max(256, g.linear_ce_workspace_bytes(0, 200, 64, 1, 1)), dtype=torch.uint8, device="cuda")
    g.linear_ce_backward(None, 64, c.wd, 64, 1, 0, 200, 64, None, 0.0, None, None, None, None, 0, dw, 72, 1, 0, ws,
                         ws.numel())
    torch.cuda.synchronize()
    assert loss.item() == 0.0 and not dw[:, :64].any() and (dw[:, 64:] == 9.0).all()


def test_same_inputs_same_bits_and_stale_workspace(g):
    """Results do not depend on what the workspace held, nor on the run."""
    import torch
    c = Case(300, 2000, 128, softcap=15.0)
    first = c.forward(g) + c.backward(g, 320)
    n = g.linear_ce_workspace_bytes(300, 2000, 128, 1, 0)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    again = c.forward(g, ws=ws) + c.backward(g, 320)
    for a, b in zip(first, again):
        assert torch.equal(a, b)


def test_captured_step(g):
    """Forward and backward captured on another stream, replayed on new values
    while an eager call of the same tensors follows."""
    import torch
    c = Case(130, 700, 64)
    N, V, d = 130, 700, 64
    nf, nb = (g.linear_ce_workspace_bytes(N, V, d, 1, k) for k in (0, 1))
    wf, wb = (torch.empty(n, dtype=torch.uint8, device="cuda") for n in (nf, nb))
    loss, tok, lse = (torch.empty(k, device="cuda") for k in (1, N, N))
    dx, dw = torch.empty(N, d, dtype=c.dt, device="cuda"), torch.empty(V, d, dtype=c.dt, device="cuda")
    st = torch.cuda.Stream()

    def run():
        g.linear_ce_forward(c.xd, d, c.wd, d, 1, N, V, d, c.td, 0.0, loss, tok, lse, wf, nf, st)
        g.linear_ce_backward(c.xd, d, c.wd, d, 1, N, V, d, c.td, 0.0, lse, None, None, dx, d, dw, d, 1, 0, wb, nb, st)

    torch.cuda.synchronize()
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        run()
    new = Case(130, 700, 64, seed=5)
    c.xd.copy_(new.xd); c.wd.copy_(new.wd); c.td.copy_(new.td)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    new.check_forward((loss, tok, lse))
    new.check_backward(dx, dw)
    got = [t.clone() for t in (loss, tok, lse, dx, dw)]
    run()
    torch.cuda.synchronize()
    for a, b in zip(got, (loss, tok, lse, dx, dw)):
        assert torch.equal(a, b)


def test_gradient_against_differences(g):
    """The loss of the GPU moves along a direction as its gradient says (fp32)."""
    import torch
    c = Case(20, 60, 32, "f32", spread=1.0)
    gx, gw = c.backward(g)
    rng = np.random.default_rng(8)
    for t, grad in ((c.xd, gx), (c.wd, gw)):
        v = torch.from_numpy(rng.standard_normal(tuple(t.shape)).astype(np.float32)).cuda()
        h, keep = 1e-2, t.clone()
        t.add_(v, alpha=h)
        up = c.forward(g)[1].double().sum().item()
        t.copy_(keep).sub_(v, alpha=h)
        down = c.forward(g)[1].double().sum().item()
        t.copy_(keep)
        count = (c.t >= 0).sum()
        want = (grad.double() * v.double()).sum().item()
        # third-order term: |v|^3 h^2 / 6 of a loss whose third derivative is below 1 per logit
        assert abs((up - down) / (2 * h) / count - want) <= 5e-3 * max(1.0, abs(want))


class WideCap(Case):
    """A cap far above the logits: there z is nearly v, and its error has to stay a
    part of z, not of the cap (the quotient's series is right to 2^-21 of tanh; the
    exponential's form, from a half on, to 2^-22 of 1: 2^-20 of z, doubled here)."""

    def ez(self):
        z = np.abs(ce.logits(self.x, self.w, self.cap))
        return (self.d + 16) * 2.0 ** -23 * (np.abs(self.x) @ np.abs(self.w).T) + z * 2.0 ** -19


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("cap,spread", [(65.0, 2.0), (100.0, 150.0), (1e4, 2.0), (1e6, 2.0), (1e20, 2.0)])
@pytest.mark.parametrize("N,V,d", [(33, 1000, 64), (300, 520, 2056)])
def test_wide_softcap(g, N, V, d, cap, spread, dtype):
    c = WideCap(N, V, d, dtype=dtype, softcap=cap, spread=spread)
    c.check_forward(c.forward(g))
    c.check_backward(*c.backward(g, dloss=1.5), dloss=1.5)
    assert g.ngram_sync_status() == g.GPT_OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cap", [0.0, 15.0, 100.0])
def test_row_of_nan_with_a_zero_gradient(g, cap, dtype):
    """A per-token gradient of 0 keeps a NaN row out of dx, its target's term too."""
    import torch
    c = Case(60, 300, 64, dtype, softcap=cap, ignored=0.0)
    c.xd[7, :c.d] = float("nan")
    lse = c.forward(g)[2]
    dtok = np.ones(60, dtype=np.float32)
    dtok[7] = 0
    gx, _ = c.backward(g, dtok=dtok, dw=False, lse=lse)
    assert not gx[7].any() and torch.isfinite(gx).all()
    g.ngram_sync_status()
