"""The standalone training operators as a program uses them together: a linear
layer in block-scaled e4m3, the LM head's loss and gradient without stored
logits, the layer's gradients from the same quantized operands, the global
clip, Muon on the layer's weight.  Every stage is checked against fp64 from
the stage before it; then the whole step runs captured and on two streams at once."""

import numpy as np
import pytest

from oracle import fp8_block as fb
from oracle import linear_ce as ce
from oracle import muon
from tests.helpers import rel_l2

pytestmark = pytest.mark.gpu

T, I, O, V = 300, 264, 392, 1000


@pytest.fixture(scope="module")
def g():
    import torch
    import gpt_pretraining_step_decoder_b200 as g
    assert torch.cuda.is_available()
    return g


def pitch(n):
    return -(-n // 16) * 16


class Step:
    """Buffers of one step, as a program keeps them."""

    def __init__(self, g, seed, stream=None):
        import torch
        gen = torch.Generator().manual_seed(seed)
        self.g, self.stream = g, stream
        new = lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
        bf = torch.bfloat16
        self.x = torch.randn(T, I, generator=gen).to(bf).cuda()
        self.w = (torch.randn(O, I, generator=gen) / I ** 0.5).cuda()
        self.head = (torch.randn(V, O, generator=gen) * 2 / O ** 0.5).to(bf).cuda()
        t = torch.randint(0, V, (T,), generator=gen)
        t[torch.rand(T, generator=gen) < 0.1] = -1
        self.t = t.to(torch.int32).cuda()
        q = {}
        for name, r, c in (("x", T, I), ("w", O, I), ("dh", T, O)):
            for key, rr, cc in ((name, r, c), (name + "t", c, r)):
                q[key] = (new(rr, pitch(cc), dt=torch.uint8), new(g.fp8_block_scale_bytes(rr, cc), dt=torch.uint8))
        self.q = q
        self.h, self.dh, self.dx = new(T, O, dt=bf), new(T, O, dt=bf), new(T, I)
        self.loss, self.lse, self.norm = new(1), new(T), new(1)
        self.dw, self.dhead, self.m = new(O, I), new(V, O), torch.zeros(O, I, device="cuda")
        sizes = [g.gptx_gemm_fp8_block_workspace_bytes(*s) for s in ((T, O, I), (T, I, O), (O, I, T))]
        sizes += [g.linear_ce_workspace_bytes(T, V, O, 1, k) for k in (0, 1)] + [g.grad_clip_workspace_bytes(2),
                                                                                g.muon_update_workspace_bytes(O, I)]
        self.ws = new(max(sizes), dt=torch.uint8)      # the stages follow one another: one workspace

    def quantize(self, name, x, dtype, square):
        r, c = x.shape
        (q, s), (qt, st) = self.q[name], self.q[name + "t"]
        self.g.fp8_block_quantize(x, dtype, r, c, c, square, q, pitch(c), s, qt, pitch(r), st, self.stream)

    def product(self, a, b, M, N, K, out, dtype):
        (qa, sa), (qb, sb) = self.q[a], self.q[b]
        self.g.gptx_gemm_fp8_block(M, N, K, qa, pitch(K), sa, qb, pitch(K), sb, dtype, out, N, 0, self.ws,
                                   self.ws.numel(), self.stream)

    def gradients(self):
        g, ws, n, st = self.g, self.ws, self.ws.numel(), self.stream
        self.quantize("x", self.x, 1, 0)
        self.quantize("w", self.w, 0, 1)
        self.product("x", "w", T, O, I, self.h, 1)
        g.linear_ce_forward(self.h, O, self.head, O, 1, T, V, O, self.t, 15.0, self.loss, None, self.lse, ws, n, st)
        g.linear_ce_backward(self.h, O, self.head, O, 1, T, V, O, self.t, 15.0, self.lse, None, None, self.dh, O,
                             self.dhead, O, 0, 0, ws, n, st)
        self.quantize("dh", self.dh, 1, 0)
        self.product("dh", "wt", T, I, O, self.dx, 0)
        self.product("dht", "xt", O, I, T, self.dw, 0)

    def update(self):
        ws, n, st = self.ws, self.ws.numel(), self.stream
        self.g.grad_clip([self.dw, self.dhead], None, 1e-3, self.norm, ws, n, st)
        self.g.muon_update(self.w, self.m, self.dw, O, I, 1, 0.02, 0.95, 1, 5, ws, n, st)

    def results(self):
        return [t.clone() for t in (self.h, self.loss, self.lse, self.dh, self.dhead, self.dx, self.dw, self.norm, self.w, self.m)]


def f64(t):
    return t.double().cpu().numpy()


def test_step_stage_by_stage(g):
    import torch
    s = Step(g, 1)
    w0 = f64(s.w)
    s.gradients()
    torch.cuda.synchronize()
    assert g.ngram_sync_status() == g.GPT_OK
    dq = lambda m, sq: fb.decode(*fb.quantize(m, sq))  # noqa: E731
    x, w = f64(s.x), w0

    def close(got, a, b, half_step):
        # exact products, K fp32 additions of at most one step each, one rounding of the result
        bound = (a.shape[1] + 16) * 2.0 ** -23 * (np.abs(a) @ np.abs(b).T)
        ref = a @ b.T
        assert (np.abs(f64(got) - ref) <= bound + half_step * (np.abs(ref) + bound)).all()

    close(s.h, dq(x, 0), dq(w, 1), 2.0 ** -8)
    h, head, t = f64(s.h), f64(s.head), s.t.cpu().numpy()
    loss, _, lse = ce.forward(h, head, t, 15.0)
    assert abs(s.loss.item() - loss) < 1e-4 and np.abs(f64(s.lse) - lse).max() < 1e-4
    dh, dhead = ce.backward(h, head, t, 15.0)
    # dz and dh rounded to bf16 (half a step 2^-8 each), everything else fp32
    assert rel_l2(f64(s.dh), dh) < 2 * 2.0 ** -8 and rel_l2(f64(s.dhead), dhead) < 2.0 ** -8 + 1e-4
    d = f64(s.dh)
    close(s.dx, dq(d, 0), dq(w.T, 1), 0.0)
    close(s.dw, dq(d.T, 0), dq(x.T, 0), 0.0)
    dw, dhead = f64(s.dw), f64(s.dhead)
    s.update()
    torch.cuda.synchronize()
    assert g.ngram_sync_status() == g.GPT_OK
    norm = np.sqrt((dw ** 2).sum() + (dhead ** 2).sum())
    coef = min(1.0, 1e-3 / (norm + 1e-6))
    assert coef < 1 and abs(s.norm.item() - norm) <= 2.0 ** -23 * norm
    for got, ref in ((s.dw, dw), (s.dhead, dhead)):
        assert (np.abs(f64(got) - coef * ref) <= 2.0 ** -22 * coef * np.abs(ref) + 2.0 ** -149).all()
    # Muon has parity tests of its own; here its momentum shows which gradient it took
    _, m = muon.muon_update(w0, f64(s.dw), np.zeros_like(w0), 0.02, 0.95)
    assert rel_l2(f64(s.m), m) < 1e-6 and np.isfinite(f64(s.w)).all()
    assert np.abs(f64(s.w) - w0).max() > 0


def test_step_captured_equals_eager(g):
    """The whole step in one graph, replayed on other inputs, against the same calls made one by one."""
    import torch
    st = torch.cuda.Stream()
    a, b = Step(g, 2, st), Step(g, 3)
    torch.cuda.synchronize()
    a.gradients(); a.update()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        a.gradients()
        a.update()
    for k in ("x", "w", "head", "t", "m"):
        getattr(a, k).copy_(getattr(b, k))
    torch.cuda.synchronize()
    graph.replay()
    b.gradients(); b.update()
    torch.cuda.synchronize()
    assert g.ngram_sync_status() == g.GPT_OK
    for p, q in zip(a.results(), b.results()):
        assert torch.equal(p, q)


def test_two_steps_at_once(g):
    """Two steps with buffers of their own, interleaved on two streams, give what each gives alone."""
    import torch
    alone = []
    for seed in (4, 5):
        s = Step(g, seed)
        s.gradients(); s.update()
        torch.cuda.synchronize()
        alone.append(s.results())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        steps = [Step(g, seed, st) for seed, st in zip((4, 5), streams)]
        torch.cuda.synchronize()
        for s in steps:
            s.gradients()
        for s in steps:
            s.update()
        torch.cuda.synchronize()
        for s, want in zip(steps, alone):
            for p, q in zip(s.results(), want):
                assert torch.equal(p, q)
    assert g.ngram_sync_status() == g.GPT_OK
