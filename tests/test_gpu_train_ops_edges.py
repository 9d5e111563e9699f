"""Calls of the standalone training operators at the edges of what their
documentation allows."""

import threading

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import torch
    import gpt_pretraining_step_decoder_b200 as g
    assert torch.cuda.is_available()
    return g


def ce_inputs(N, V, d, seed=0, spread=2.0):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(N, d, generator=gen, device="cuda").bfloat16()
    w = (torch.randn(V, d, generator=gen, device="cuda") * spread / d ** 0.5).bfloat16()
    t = torch.randint(0, V, (N,), generator=gen, device="cuda", dtype=torch.int32)
    return x, w, t


def ce_forward(g, x, w, t, softcap=0.0, ws=None):
    import torch
    (N, d), V = x.shape, w.shape[0]
    code = g.DTYPE_BF16 if x.dtype == torch.bfloat16 else g.DTYPE_F32
    if ws is None:
        ws = torch.empty(g.linear_ce_workspace_bytes(N, V, d, code, 0), dtype=torch.uint8, device="cuda")
    loss, tok, lse = (torch.empty(k, device="cuda") for k in (1, N, N))
    g.linear_ce_forward(x, d, w, d, code, N, V, d, t, softcap, loss, tok, lse, ws, ws.numel())
    torch.cuda.synchronize()
    return loss, tok, lse


def test_tile_forms_switched_during_calls(g):
    """A thread that switches the GEMMs' tile forms while another one forms losses:
    each loss is that of one form or the other (the number of statistics that the
    product writes is the number that the workspace and the joining kernel count on)."""
    import torch
    N, V, d = 300, 16384, 768
    x, w, t = ce_inputs(N, V, d)
    want, sizes = [], []
    for on in (False, True):
        g.gptx_set_gemm_cta_pairs(on)
        sizes.append(g.linear_ce_workspace_bytes(N, V, d, g.DTYPE_BF16, 0))
        want.append(ce_forward(g, x, w, t))
    assert sizes[0] != sizes[1]                       # the forms leave different numbers of statistics
    ws = torch.empty(max(sizes), dtype=torch.uint8, device="cuda")
    stop = threading.Event()

    def switch():
        while not stop.is_set():
            for on in (0, 1):
                g._lib.gptx_set_gemm_cta_pairs(on)

    th = threading.Thread(target=switch)
    th.start()
    try:
        for _ in range(1500):
            got = ce_forward(g, x, w, t, ws=ws)
            assert any(all(torch.equal(a, b) for a, b in zip(got, ref)) for ref in want)
    finally:
        stop.set()
        th.join()
        g.gptx_set_gemm_cta_pairs(True)
    assert g.ngram_sync_status() == g.GPT_OK


@pytest.mark.parametrize("softcap", [0.0, 15.0, 100.0])
@pytest.mark.parametrize("N,V,d,rows", [
    (33, 50112, 768, (49984, 50048)),     # one row block: runs of three 128-column tiles, the last run of two
    (33, 50048, 64, (49792, 49920)),      # runs of two 256-column tiles
    (16384, 50560, 64, (50304, 50432)),   # pairs, runs of four 256-column tiles, the last run of two
])
def test_nan_rows_of_the_weight_before_an_empty_half_tile(g, N, V, d, rows, softcap):
    """NaN in the classes of a whole half tile whose neighbour in the run lies past
    the vocabulary: the row's sum is NaN, and the loss is reported as not finite."""
    import torch
    x, w, t = ce_inputs(N, V, d)
    t.clamp_(max=rows[0] - 1)
    loss, _, lse = ce_forward(g, x, w, t, softcap)
    assert torch.isfinite(lse).all() and g.ngram_sync_status() == g.GPT_OK
    w[rows[0]:rows[1]] = float("nan")
    loss, _, lse = ce_forward(g, x, w, t, softcap)
    assert torch.isnan(lse).all() and torch.isnan(loss).all()
    assert g.ngram_sync_status() == g.GPT_ERR_NONFINITE


def test_norm_alone_counts_a_shared_tensor_each_time(g):
    import torch
    t = torch.randn(1000, device="cuda")
    ws = torch.empty(g.grad_clip_workspace_bytes(3), dtype=torch.uint8, device="cuda")
    norm, keep = torch.zeros(1, device="cuda"), t.clone()
    g.grad_clip([t, t, t[100:]], None, 0.0, norm, ws, ws.numel())
    want = (2 * t.double().square().sum() + t[100:].double().square().sum()).sqrt().item()
    assert abs(norm.item() - want) <= 2.0 ** -23 * want and torch.equal(t, keep)


def test_clip_of_an_iterator_of_tensors(g):
    import torch
    grads = [torch.randn(n, device="cuda") for n in (300, 7)]
    ws = torch.empty(g.grad_clip_workspace_bytes(2), dtype=torch.uint8, device="cuda")
    norm = torch.zeros(1, device="cuda")
    want = sum(t.double().square().sum() for t in grads).sqrt().item()
    g.grad_clip((t for t in grads), None, 0.5, norm, ws, ws.numel())
    after = sum(t.double().square().sum() for t in grads).sqrt().item()
    assert abs(norm.item() - want) <= 2.0 ** -23 * want and abs(after - 0.5) <= 1e-6


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_empty_batch(g, dtype):
    """A batch of no tokens through quantizer, loss and gradient, as a program's empty
    tensors arrive (their addresses are null)."""
    import torch
    dt, code = (torch.bfloat16, g.DTYPE_BF16) if dtype == "bf16" else (torch.float32, g.DTYPE_F32)
    new = lambda *s, dt=dt: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    x, t, tok, dx = new(0, 64), new(0, dt=torch.int32), new(0, dt=torch.float32), new(0, 64)
    w = torch.randn(200, 64, device="cuda").to(dt)
    q, sc = new(0, 64, dt=torch.uint8), new(0, dt=torch.uint8)
    g.fp8_block_quantize(x, code, 0, 64, 64, False, q, 64, sc)
    ws = new(g.linear_ce_workspace_bytes(0, 200, 64, code, 1), dt=torch.uint8)
    g.linear_ce_forward(x, 64, w, 64, code, 0, 200, 64, t, 0.0, None, tok, tok, ws, ws.numel())
    g.linear_ce_backward(x, 64, w, 64, code, 0, 200, 64, t, 0.0, tok, None, None, dx, 64, None, 64, code, 0, ws, ws.numel())
    torch.cuda.synchronize()
    assert g.ngram_sync_status() == g.GPT_OK


def device_ms(call, n=3):
    import torch
    call()
    times = []
    for _ in range(n):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        call()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b))
    return min(times)


def test_counting_the_targets_does_not_grow_with_the_product(g):
    """fp32, many rows and a small width: the gradient of the mean costs what that of
    per-token losses does, which has no targets to count (three times as much where
    every block of the product counted all of them)."""
    import torch
    N, V, d = 65536, 4096, 16
    x, w = torch.randn(N, d, device="cuda"), torch.randn(V, d, device="cuda") / 4
    t = torch.randint(-1, V, (N,), device="cuda", dtype=torch.int32)
    lse = ce_forward(g, x, w, t)[2]
    n = g.linear_ce_workspace_bytes(N, V, d, g.DTYPE_F32, 1)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    dtok = torch.full((N,), 1.0, device="cuda") / (t >= 0).sum()
    grads = [(torch.empty_like(x), torch.empty_like(w)) for _ in range(2)]

    def backward(dtok, dx, dw):
        g.linear_ce_backward(x, d, w, d, g.DTYPE_F32, N, V, d, t, 0.0, lse, None, dtok, dx, d, dw, d, g.DTYPE_F32, 0, ws, n)

    mean = device_ms(lambda: backward(None, *grads[0]))
    tokens = device_ms(lambda: backward(dtok, *grads[1]))
    assert mean < 1.5 * tokens, (mean, tokens)
    for a, b in zip(*grads):  # the two factors differ by the rounding of 1 / count at most
        assert ((a - b).abs() <= 2.0 ** -22 * b.abs() + 2.0 ** -22 * b.abs().max()).all()


# The tensor cores add the 32 (bf16: 16) products of an instruction to an fp32
# accumulator and cut the sum off, always towards zero, so a long sum of positive products
# comes out low: 64 instructions, the chunks that are added rounded, each lose
# less than a step (2^-23) of a partial sum that grows evenly, 65 / 2 steps of the
# whole, and the chunks' own additions half a step each.  In one chunk the products
# below were 6.1e-6 (K = 16384) and 1.7e-5 (K = 32768) low.
CHUNKED = 65 / 2 * 2.0 ** -23 + 16 * 2.0 ** -24


def quantized_uniform(g, rows, cols, gen):
    """Positive e4m3 operand: codes, scales and its values in fp64."""
    import torch
    x = torch.rand(rows, cols, generator=gen, device="cuda") + 0.01
    q = torch.empty(rows, cols, dtype=torch.uint8, device="cuda")
    s = torch.empty(g.fp8_block_scale_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    g.fp8_block_quantize(x, g.DTYPE_F32, rows, cols, cols, False, q, cols, s)
    scale = torch.exp2(g.fp8_block_scales(s, rows, cols).double() - 127)
    return q, s, q.view(torch.float8_e4m3fn).double() * scale.repeat_interleave(128, 1)


@pytest.mark.parametrize("pairs", [True, False])
@pytest.mark.parametrize("M,N,K,split", [(4096, 2048, 16384, False), (2304, 2304, 32768, False), (1000, 1000, 16384, True)])
def test_long_products_in_fp32_are_not_cut_off(g, M, N, K, split, pairs):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(K)
    qa, sa, va = quantized_uniform(g, M, K, gen)
    qb, sb, vb = quantized_uniform(g, N, K, gen)
    ref = va @ vb.T
    g.gptx_set_gemm_cta_pairs(pairs)
    try:
        n = g.gptx_gemm_fp8_block_workspace_bytes(M, N, K)
        assert (n > 0) == split
        ws = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
        c = torch.full((M, N), 9.0, device="cuda")
        for beta in (0, 1):
            g.gptx_gemm_fp8_block(M, N, K, qa, K, sa, qb, K, sb, g.DTYPE_F32, c, N, beta, ws, n)
            torch.cuda.synchronize()
            err = (c.double() / (1 + beta) - ref) / ref
            assert err.mean().abs() <= CHUNKED and err.square().mean().sqrt() <= CHUNKED, (err.mean(), err.abs().max())
    finally:
        g.gptx_set_gemm_cta_pairs(True)
    assert g.ngram_sync_status() == g.GPT_OK


@pytest.mark.parametrize("softcap", [0.0, 50.0, 100.0])
@pytest.mark.parametrize("N,V", [(40, 520), (3000, 20000)])
def test_long_logits_are_not_cut_off(g, N, V, softcap):
    """d = 8192, logits of about 50, all products positive."""
    import torch
    d = 8192
    gen = torch.Generator(device="cuda").manual_seed(V)
    x = torch.rand(N, d, generator=gen, device="cuda").bfloat16()
    w = (torch.rand(V, d, generator=gen, device="cuda") * (200.0 / d)).bfloat16()
    t = torch.randint(0, V, (N,), generator=gen, device="cuda", dtype=torch.int32)
    loss, tok, lse = ce_forward(g, x, w, t, softcap)
    u = x.double() @ w.double().T
    z = softcap * torch.tanh(u / softcap) if softcap else u
    slope = 1 - (z / softcap).square() if softcap else 1.0
    ref = torch.logsumexp(z, 1)
    # the cut-off logits, the soft-cap's 2^-22 of the cap, an fp32 step of the exponents and of the result
    tol = ((z - ref[:, None]).exp() * slope * u).sum(1) * CHUNKED + softcap * 2.0 ** -22 + 2.0 ** -23 * (ref + 8)
    err = lse.double() - ref
    assert err.mean().abs() <= tol.mean() and err.square().mean().sqrt() <= tol.square().mean().sqrt()
    zt = z.gather(1, t.long()[:, None]).squeeze(1)
    assert (tok.double() - (ref - zt)).square().mean().sqrt() <= 2 * tol.square().mean().sqrt()
    assert g.ngram_sync_status() == g.GPT_OK


@pytest.mark.parametrize("softcap", [0.0, 50.0, 100.0])
@pytest.mark.parametrize("N,V", [(40, 520), (3000, 20000)])
def test_gradient_of_long_logits_sums_to_zero(g, N, V, softcap):
    """d = 8192, all products positive: sum_v dz / slope is 0 for a softmax; with a column
    of ones in W and no soft-cap it is dx of that column.  With a soft-cap the column of
    dx is compared with fp64."""
    import torch
    d = 8192
    gen = torch.Generator(device="cuda").manual_seed(V)
    x = torch.rand(N, d, generator=gen, device="cuda").bfloat16()
    w = (torch.rand(V, d, generator=gen, device="cuda") * (200.0 / d)).bfloat16()
    w[:, 0] = 1.0
    t = torch.randint(0, V, (N,), generator=gen, device="cuda", dtype=torch.int32)
    u = x.double() @ w.double().T
    z = softcap * torch.tanh(u / softcap) if softcap else u
    slope = 1 - (z / softcap).square() if softcap else torch.ones_like(u)
    lse = torch.logsumexp(z, 1)
    p = (z - lse[:, None]).exp()
    dz = p * slope
    at = t.long()[:, None]
    dz.scatter_add_(1, at, -slope.gather(1, at))
    ref = dz.sum(1)
    # every p is off by that of its logit; dz is rounded to bf16 (at random, but for the
    # target's term), and its sum of V / 16 additions cut off below a step of a sum below one
    ez = slope * u * CHUNKED + softcap * 2.0 ** -22 + 2.0 ** -23 * (lse[:, None].abs() + 8)
    if softcap:  # and the slope, 2^-22 of tanh
        ez = ez + 2.0 ** -21 / slope
    tol = (p * slope * ez).sum(1) + slope.gather(1, at).squeeze(1) * 2.0 ** -21
    tol += 4 * 2.0 ** -9 * (dz.square().sum(1) - dz.gather(1, at).squeeze(1).square()).clamp(min=0).sqrt()
    tgt = dz.gather(1, at).squeeze(1)
    tol += (tgt.bfloat16().double() - tgt).abs() + (V / 16 + 16) * 2.0 ** -23 * (p * slope).sum(1) + 2.0 ** -8 * ref.abs()
    n = g.linear_ce_workspace_bytes(N, V, d, g.DTYPE_BF16, 1)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    dx, dtok, lse32 = torch.empty_like(x), torch.ones(N, device="cuda"), lse.float()
    g.linear_ce_backward(x, d, w, d, g.DTYPE_BF16, N, V, d, t, softcap, lse32, None, dtok, dx, d, None, d, g.DTYPE_BF16, 0,
                         ws, n)
    torch.cuda.synchronize()
    err = dx[:, 0].double() - ref
    assert err.mean().abs() <= tol.mean() and err.square().mean().sqrt() <= tol.square().mean().sqrt(), (err.mean(), tol.mean())
    assert g.ngram_sync_status() == g.GPT_OK


@pytest.fixture(params=[True, False], ids=["sm_pairs", "one_sm"])
def pairs(request, g):
    g.gptx_set_gemm_cta_pairs(request.param)
    yield request.param
    g.gptx_set_gemm_cta_pairs(True)


def e4m3(rows, K, seed):
    """Codes [rows, pitch] of values in (-2, 2) that fill fp32 sums exactly, and the values."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.randint(-4, 5, (rows, K), generator=gen, device="cuda").double() / 4
    q = torch.zeros(rows, -(-K // 16) * 16, dtype=torch.uint8, device="cuda")
    q[:, :K] = v.float().to(torch.float8_e4m3fn).view(torch.uint8)
    return q, v


@pytest.mark.parametrize("M,N", [(33, 5), (300, 333), (70, 127), (1000, 1001), (9001, 2315)])
@pytest.mark.parametrize("op", ["block", "block_beta", "tensor", "bf16", "bf16_beta"])
def test_products_leave_the_columns_behind_an_odd_width(g, pairs, op, M, N):
    """A result as some columns of a wider matrix, its last ones inside 16 bytes: the
    neighbours stay.  Small whole numbers of quarters: every sum is exact."""
    import torch
    K = 264
    (qa, va), (qb, vb) = e4m3(M, K, M), e4m3(N, K, N)
    ref = va @ vb.T
    for dt in (torch.float32, torch.bfloat16):
        beta = op.endswith("beta")
        if beta and dt == torch.bfloat16:
            continue
        ld, code = N + 16 - N % 8 + 8, g.DTYPE_F32 if dt == torch.float32 else g.DTYPE_BF16
        c = torch.full((M + 1, ld), 7.0, dtype=dt, device="cuda")
        one = torch.ones(1, device="cuda")
        if op.startswith("block"):
            sa, sb = (torch.full((g.fp8_block_scale_bytes(r, K),), 127, dtype=torch.uint8, device="cuda") for r in (M, N))
            g.gptx_gemm_fp8_block(M, N, K, qa, qa.shape[1], sa, qb, qb.shape[1], sb, code, c, ld, beta)
        elif op == "tensor":
            g.gptx_gemm_fp8(M, N, K, qa, qa.shape[1], qb, qb.shape[1], one, one, code, c, ld)
        else:
            mode = 0 if dt == torch.bfloat16 else 2 if beta else 1
            g.gptx_gemm_bf16(M, N, K, va.bfloat16(), K, 1, vb.bfloat16(), K, 1, c, ld, beta=int(beta), mode=mode)
        torch.cuda.synchronize()
        assert (c[M:] == 7).all() and (c[:, N:] == 7).all()
        assert torch.equal(c[:M, :N], (ref + 7 * beta).to(dt))
    assert g.ngram_sync_status() == g.GPT_OK


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (2, 3, 5), (129, 1, 127), (5, 129, 513), (1, 1, 4097), (257, 130, 8190)])
def test_products_of_tiny_and_odd_sizes(g, pairs, M, N, K):
    import torch
    (qa, va), (qb, vb) = e4m3(M, K, M + K), e4m3(N, K, N + K)
    sa, sb = (torch.full((g.fp8_block_scale_bytes(r, K),), 127, dtype=torch.uint8, device="cuda") for r in (M, N))
    n = g.gptx_gemm_fp8_block_workspace_bytes(M, N, K)
    ws = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
    for dt, code in ((torch.float32, g.DTYPE_F32), (torch.bfloat16, g.DTYPE_BF16)):
        ld = -(-N // 8) * 8
        c = torch.full((M, ld), 7.0, dtype=dt, device="cuda")
        g.gptx_gemm_fp8_block(M, N, K, qa, qa.shape[1], sa, qb, qb.shape[1], sb, code, c, ld, 0, ws, n)
        torch.cuda.synchronize()
        assert torch.equal(c[:, :N], (va @ vb.T).to(dt)) and (c[:, N:] == 7).all()
    assert g.ngram_sync_status() == g.GPT_OK


def test_clip_partly_in_place(g):
    """Outputs that are their own tensor beside others that are not."""
    import torch
    grads = [torch.randn(n, device="cuda") for n in (5000, 333, 70001)]
    keep = [t.clone() for t in grads]
    outs = [grads[0], torch.empty_like(grads[1]), grads[2]]
    ws = torch.empty(g.grad_clip_workspace_bytes(3), dtype=torch.uint8, device="cuda")
    norm = torch.zeros(1, device="cuda")
    want = sum(t.double().square().sum() for t in keep).sqrt().item()
    g.grad_clip(grads, outs, 0.25, norm, ws, ws.numel())
    coef = 0.25 / (want + 1e-6)
    for t, o in zip(keep, outs):
        assert ((o.double() - t.double() * coef).abs() <= 2.0 ** -22 * t.double().abs() * coef).all()
    assert torch.equal(grads[1], keep[1]) and abs(norm.item() - want) <= 2.0 ** -23 * want


def test_two_threads(g):
    """Every operator from two host threads, on streams, tensors and workspaces of their
    own: the bits are those of a single thread."""
    import torch
    N, V, d = 500, 3000, 264

    class Run:
        def __init__(self, seed):
            self.st = torch.cuda.Stream()
            self.x, self.w, self.t = ce_inputs(N, V, d, seed)
            self.ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
            new = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
            self.q, self.s = new(N, 272, dt=torch.uint8), new(g.fp8_block_scale_bytes(N, d), dt=torch.uint8)
            self.qw, self.sw = new(V, 272, dt=torch.uint8), new(g.fp8_block_scale_bytes(V, d), dt=torch.uint8)
            self.c, self.loss, self.lse = new(N, V), new(1), new(N)
            self.dx, self.dw, self.norm = torch.zeros_like(self.x), torch.zeros_like(self.w), new(1)
            self.outs = [torch.zeros_like(self.dx), torch.zeros_like(self.dw)]

        def __call__(self):
            st, ws, n, bf = self.st, self.ws, self.ws.numel(), g.DTYPE_BF16
            g.fp8_block_quantize(self.x, bf, N, d, d, False, self.q, 272, self.s, stream=st)
            g.fp8_block_quantize(self.w, bf, V, d, d, True, self.qw, 272, self.sw, stream=st)
            g.gptx_gemm_fp8_block(N, V, d, self.q, 272, self.s, self.qw, 272, self.sw, g.DTYPE_F32, self.c, V, 0, ws, n, st)
            g.linear_ce_forward(self.x, d, self.w, d, bf, N, V, d, self.t, 15.0, self.loss, None, self.lse, ws, n, st)
            g.linear_ce_backward(self.x, d, self.w, d, bf, N, V, d, self.t, 15.0, self.lse, None, None, self.dx, d, self.dw,
                                 d, bf, 0, ws, n, st)
            g.grad_clip([self.dx, self.dw], self.outs, 1e-3, self.norm, ws, n, st)
            st.synchronize()
            return [t.clone() for t in (self.q, self.s, self.c, self.loss, self.lse, self.dx, self.dw, self.norm, *self.outs)]

    runs = [Run(1), Run(2)]
    torch.cuda.synchronize()
    want = [r() for r in runs]
    bad = []

    def work(r, ref):
        try:
            for _ in range(60):
                if not all(torch.equal(a, b) for a, b in zip(r(), ref)):
                    bad.append("bits")
        except Exception as e:  # noqa: BLE001 -- reported below
            bad.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(runs, want)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    assert not bad and g.ngram_sync_status() == g.GPT_OK


def test_offsets_beyond_32_bits(g):
    """Row pitches that put the last rows of an operand or a result past 2^32 elements, a
    gradient of more than 2^31, statistics of more than 2^31 pairs."""
    import torch
    big, ld = torch.empty(9 << 30, dtype=torch.uint8, device="cuda"), 1 << 20
    # the quantizer: by TMA, and with rows off 16 bytes by plain loads
    for pitch_, dt, code in ((ld, torch.bfloat16, 1), (ld + 1, torch.bfloat16, 1)):
        rows, cols = 4200, 200
        x = big.view(dt)[:rows * pitch_].view(rows, pitch_)[:, :cols]
        x.copy_(torch.randn(rows, cols, device="cuda"))
        y = x.contiguous()
        out = []
        for src, p in ((x, pitch_), (y, cols)):
            q, s = torch.zeros(rows, 208, dtype=torch.uint8, device="cuda"), torch.zeros(g.fp8_block_scale_bytes(rows, cols), dtype=torch.uint8, device="cuda")
            g.fp8_block_quantize(src, code, rows, cols, p, False, q, 208, s)
            out += [q, s]
        assert torch.equal(out[0], out[2]) and torch.equal(out[1], out[3])
    # the product: operands and results, plain and element by element at the row's end
    M, K = 8300, 264
    (qa, va), (qb, vb) = e4m3(M, K, 1), e4m3(141, K, 2)
    sa, sb = (torch.full((g.fp8_block_scale_bytes(r, K),), 127, dtype=torch.uint8, device="cuda") for r in (M, 141))
    a = big[:M * ld].view(M, ld)
    a[:, :K] = qa[:, :K]
    for N in (136, 141):
        c = torch.zeros(M, 144, device="cuda")
        g.gptx_gemm_fp8_block(M, N, K, a, ld, sa, qb, qb.shape[1], sb, g.DTYPE_F32, c, 144)
        assert torch.equal(c[:, :N].double(), va @ vb[:N].T)
        wide = big.view(torch.bfloat16)[:4200 * ld].view(4200, ld)
        wide[:, N:160] = 7
        g.gptx_gemm_fp8_block(4200, N, K, qa, qa.shape[1], torch.full((g.fp8_block_scale_bytes(4200, K),), 127, dtype=torch.uint8, device="cuda"),
                              qb, qb.shape[1], sb, g.DTYPE_BF16, wide, ld)
        assert torch.equal(wide[:, :N], (va[:4200] @ vb[:N].T).bfloat16()) and (wide[:, N:160] == 7).all()
        a[:, :K] = qa[:, :K]                       # the result lay over it
    # the loss and its gradient
    N, V, d = 4200, 3000, 64
    x, w, t = ce_inputs(N, V, d)
    xs = big.view(torch.bfloat16)[:N * ld].view(N, ld)[:, :d]
    xs.copy_(x)
    ref = ce_forward(g, x, w, t)
    n = max(g.linear_ce_workspace_bytes(N, V, d, g.DTYPE_BF16, b) for b in (0, 1))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    loss, tok, lse = (torch.zeros_like(r) for r in ref)
    g.linear_ce_forward(xs, ld, w, d, g.DTYPE_BF16, N, V, d, t, 0.0, loss, tok, lse, ws, n)
    assert all(torch.equal(p, q) for p, q in zip((loss, tok, lse), ref))
    dx, dw, dw2 = torch.zeros_like(x), torch.zeros_like(w), torch.zeros_like(w)
    g.linear_ce_backward(x, d, w, d, g.DTYPE_BF16, N, V, d, t, 0.0, lse, None, None, dx, d, dw, d, g.DTYPE_BF16, 0, ws, n)
    g.linear_ce_backward(x, d, w, d, g.DTYPE_BF16, N, V, d, t, 0.0, lse, None, None, xs, ld, dw2, d, g.DTYPE_BF16, 0, ws, n)
    assert torch.equal(xs, dx) and torch.equal(dw, dw2)
    # the clip
    v = big.view(torch.bfloat16)[:(1 << 31) + 77777]
    v.fill_(0.5)
    v[-1] = 3.0
    norm = torch.zeros(1, device="cuda")
    g.grad_clip([v], None, 1.0, norm, ws, n)
    want = (0.25 * (v.numel() - 1) + 9) ** 0.5
    assert abs(norm.item() - want) <= 2.0 ** -23 * want
    assert abs(v[-1].item() - 3 / want) <= 2.0 ** -8 * 3 / want and (v[:-1] == v[0]).all()
    del big, a, wide, xs, v
    # the loss's statistics
    N, V, d = (1 << 22) + 5, 1 << 18, 16
    x, w, t = ce_inputs(N, V, d)
    assert g.linear_ce_workspace_bytes(N, V, d, g.DTYPE_BF16, 0) > 8 << 31
    lse = ce_forward(g, x, w, t)[2]
    for r in (slice(0, 100), slice(N - 100, N)):
        want = torch.logsumexp(x[r].double() @ w.double().T, 1)
        assert ((lse[r].double() - want).abs() <= 1e-5 * want).all()
    assert g.ngram_sync_status() == g.GPT_OK
