"""Block-scaled e4m3 on the GPU against the oracle: codes and scales bit for
bit (dividing by a power of two is exact, so there is one right answer), the
product elementwise within the fp32 accumulation's bound."""

import numpy as np
import pytest

from oracle import fp8_block as fb

pytestmark = pytest.mark.gpu

FILL = 0xA5


@pytest.fixture(scope="module")
def g():
    import torch
    import gpt_pretraining_step_decoder_b200 as g
    assert torch.cuda.is_available()
    return g


def pitch(n):
    return -(-n // 16) * 16


def values(rng, rows, cols):
    x = rng.standard_normal((rows, cols)) * 2.0 ** rng.uniform(-6, 6, (rows, 1))
    x[:, rng.random(cols) < 0.02] *= 50
    return x.astype(np.float32)


def rounded(x, dtype):
    import torch
    t = torch.from_numpy(x)
    return t.to(torch.bfloat16) if dtype == "bf16" else t


def gpu_quantize(g, t, square, both=(1, 1), ldx=None, offset=0):
    """t: CPU tensor [rows, cols]; placed with row pitch ldx, `offset` elements into a buffer."""
    import torch
    rows, cols = t.shape
    ldx = ldx or cols
    buf = torch.full((offset + rows * ldx,), 3e4, dtype=t.dtype, device="cuda")
    x = buf[offset:].view(rows, ldx)[:, :cols]
    x.copy_(t)
    out = []
    for on, (r, c) in zip(both, ((rows, cols), (cols, rows))):
        q = torch.full((r, pitch(c)), FILL, dtype=torch.uint8, device="cuda") if on else None
        s = torch.full((g.fp8_block_scale_bytes(r, c),), FILL, dtype=torch.uint8, device="cuda") if on else None
        out.append((q, s))
    (q, s), (qt, st) = out
    g.fp8_block_quantize(x, g.DTYPE_BF16 if t.dtype == torch.bfloat16 else g.DTYPE_F32, rows, cols, ldx, square, q,
                         pitch(cols), s, qt, pitch(rows), st)
    torch.cuda.synchronize()
    return out


def check(x, square, got):
    for m, (q, s) in zip((x, x.T), got):
        if q is None:
            continue
        qo, so = fb.quantize(m, square)
        np.testing.assert_array_equal(s.cpu().numpy(), fb.store(so))
        np.testing.assert_array_equal(q.cpu().numpy()[:, :m.shape[1]], qo)
        assert (q.cpu().numpy()[:, m.shape[1]:] == FILL).all()      # the pitch's tail is left alone


@pytest.mark.parametrize("square", [0, 1])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (3, 16), (127, 129), (128, 128), (129, 513), (257, 640), (40, 1000)])
def test_quantize_bit_exact(g, rows, cols, dtype, square):
    t = rounded(values(np.random.default_rng(rows * 1000 + cols), rows, cols), dtype)
    check(t.double().numpy(), square, gpu_quantize(g, t, square))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("ldx,offset,both", [(301, 0, (1, 1)), (304, 1, (1, 1)), (320, 8, (1, 0)), (300, 0, (0, 1))])
def test_quantize_strides_alignment_and_single_outputs(g, dtype, ldx, offset, both):
    t = rounded(values(np.random.default_rng(7), 150, 300), dtype)
    for square in (0, 1):
        check(t.double().numpy(), square, gpu_quantize(g, t, square, both, ldx, offset))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("square", [0, 1])
def test_quantize_special_values(g, dtype, square):
    x = values(np.random.default_rng(9), 260, 260)
    x[0] = 0.0
    x[1] = 1e-38
    x[2] = 1e-41          # below the smallest scale's codes
    x[3] = 3e38
    x[4, :128] = 448.0
    x[5, :128] = 449.0
    x[6, 200] = np.inf
    x[7, 3] = np.nan
    x[8, 255] = -np.inf
    x[9] = -0.0
    if square:            # keep some blocks finite
        x[:128, 128:256] = values(np.random.default_rng(10), 128, 128) * 1e-35
    t = rounded(x, dtype)
    check(t.double().numpy(), square, gpu_quantize(g, t, square))


def operands(g, M, N, K, square, seed=0):
    rng = np.random.default_rng(seed + M + N + K)
    a, b = values(rng, M, K), values(rng, N, K) * 0.02
    ((qa, sa), _), ((qb, sb), _) = (gpu_quantize(g, rounded(m, "f32"), sq, (1, 0)) for m, sq in ((a, 0), (b, square)))
    va = fb.decode(*(lambda q: (q[0], q[1]))(fb.quantize(a, 0)))
    vb = fb.decode(*fb.quantize(b, square))
    return (qa, sa, qb, sb), va, vb


def product(g, M, N, K, ops, out="f32", ldc=None, beta=0, c=None, stream=None):
    import torch
    qa, sa, qb, sb = ops
    ldc = ldc or N
    if c is None:
        c = torch.full((M, ldc), 9.0, dtype=torch.float32 if out == "f32" else torch.bfloat16, device="cuda")
    n = g.gptx_gemm_fp8_block_workspace_bytes(M, N, K)
    ws = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
    g.gptx_gemm_fp8_block(M, N, K, qa, pitch(K), sa, qb, pitch(K), sb, g.DTYPE_F32 if out == "f32" else g.DTYPE_BF16, c,
                          ldc, beta, ws, n, stream)
    torch.cuda.synchronize()
    assert g.ngram_sync_status() == g.GPT_OK, g.gpt_last_error()
    return c


def accumulation_bound(va, vb, K):
    """Products of e4m3 values and power-of-two scales are exact in fp32; each of
    the K additions loses at most one step (2^-23) of a partial sum, which is
    no larger than the sum of magnitudes."""
    return (K + 16) * 2.0 ** -23 * (np.abs(va) @ np.abs(vb).T)


@pytest.fixture(params=[1, 0], ids=["sm_pairs", "one_sm"])
def tiles(request, g):
    g.gptx_set_gemm_cta_pairs(request.param)
    yield request.param
    g.gptx_set_gemm_cta_pairs(1)


SHAPES = [(1, 8, 16), (1, 768, 768), (128, 128, 128), (129, 200, 160), (200, 384, 520), (257, 192, 1024),
          (777, 520, 1000), (300, 1000, 2100), (2048, 576, 640)]


@pytest.mark.parametrize("square", [0, 1])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product_matches_oracle(g, tiles, M, N, K, square):
    ops, va, vb = operands(g, M, N, K, square)
    ref, bound = va @ vb.T, accumulation_bound(va, vb, K)
    c = product(g, M, N, K, ops).cpu().numpy().astype(np.float64)
    assert (np.abs(c - ref) <= bound).all(), np.abs(c - ref).max()
    # bf16 output: one rounding (2^-8 of the value) more
    c = product(g, M, N, K, ops, "bf16").float().cpu().numpy().astype(np.float64)
    assert (np.abs(c - ref) <= bound + 2.0 ** -8 * (np.abs(ref) + bound)).all()


@pytest.mark.parametrize("M,N,K", [(96, 64, 8000), (384, 192, 16384), (130, 136, 5000)])
def test_split_product(g, tiles, M, N, K):
    """Few tiles and a long K: partial sums, fp32 and bf16 results, accumulation."""
    import torch
    assert g.gptx_gemm_fp8_block_workspace_bytes(M, N, K) > 0
    ops, va, vb = operands(g, M, N, K, 0)
    ref, bound = va @ vb.T, accumulation_bound(va, vb, K)
    first = product(g, M, N, K, ops)
    assert (np.abs(first.cpu().numpy() - ref) <= bound).all()
    assert torch.equal(first, product(g, M, N, K, ops))         # summed in order
    c = product(g, M, N, K, ops, "bf16").float().cpu().numpy().astype(np.float64)
    assert (np.abs(c - ref) <= bound + 2.0 ** -8 * (np.abs(ref) + bound)).all()
    twice = product(g, M, N, K, ops, beta=1, c=first.clone()).cpu().numpy().astype(np.float64)
    assert (np.abs(twice - 2 * ref) <= 2 * bound + 2.0 ** -23 * np.abs(2 * ref)).all()


@pytest.mark.parametrize("M,N,K", [(200, 392, 640), (1024, 768, 256)])
def test_product_accumulates_and_keeps_the_pitch(g, tiles, M, N, K):
    import torch
    ops, va, vb = operands(g, M, N, K, 1)
    ref, bound = va @ vb.T, accumulation_bound(va, vb, K)
    ldc = N + 8
    c = torch.full((M, ldc), 2.0, dtype=torch.float32, device="cuda")
    product(g, M, N, K, ops, ldc=ldc, beta=1, c=c)
    got = c.cpu().numpy().astype(np.float64)
    assert (got[:, N:] == 2.0).all()
    assert (np.abs(got[:, :N] - 2.0 - ref) <= bound + 2.0 ** -23 * (np.abs(ref) + 2)).all()


def test_nan_group_reaches_its_row_only(g, tiles):
    import torch
    M, N, K = 300, 256, 640
    rng = np.random.default_rng(4)
    a, b = values(rng, M, K), values(rng, N, K)
    a[7, 600] = np.inf
    b[11, 5] = np.nan
    (qa, sa), _ = gpu_quantize(g, rounded(a, "f32"), 0, (1, 0))
    (qb, sb), _ = gpu_quantize(g, rounded(b, "f32"), 0, (1, 0))
    c = product(g, M, N, K, (qa, sa, qb, sb))
    bad = torch.isnan(c)
    assert bad[7].all() and bad[:, 11].all()
    bad[7] = False
    bad[:, 11] = False
    assert not bad.any()


def test_linear_layer_products_share_one_quantization(g):
    """Forward, data-gradient and weight-gradient products of y = x W^T from x,
    W and dY quantized once each, in both orientations."""
    T, I, O = 300, 264, 392
    rng = np.random.default_rng(5)
    x, w, dy = values(rng, T, I), values(rng, O, I) * 0.02, values(rng, T, O) * 0.1
    qx, qw, qy = (gpu_quantize(g, rounded(m, "f32"), sq) for m, sq in ((x, 0), (w, 1), (dy, 0)))
    for (A, B, M, N, K, va, vb) in (
            (qx[0], qw[0], T, O, I, fb.decode(*fb.quantize(x, 0)), fb.decode(*fb.quantize(w, 1))),
            (qy[0], qw[1], T, I, O, fb.decode(*fb.quantize(dy, 0)), fb.decode(*fb.quantize(w.T, 1))),
            (qy[1], qx[1], O, I, T, fb.decode(*fb.quantize(dy.T, 0)), fb.decode(*fb.quantize(x.T, 0)))):
        c = product(g, M, N, K, (*A, *B)).cpu().numpy().astype(np.float64)
        assert (np.abs(c - va @ vb.T) <= accumulation_bound(va, vb, K)).all()


def test_captured_and_other_stream(g):
    """Quantization and product captured in a graph on another stream and replayed on new values."""
    import torch
    M, N, K = 200, 256, 384
    rng = np.random.default_rng(6)
    x = torch.from_numpy(values(rng, M, K)).cuda()
    (qb, sb), _ = gpu_quantize(g, rounded(values(rng, N, K), "f32"), 1, (1, 0))
    q = torch.empty(M, K, dtype=torch.uint8, device="cuda")
    s = torch.empty(g.fp8_block_scale_bytes(M, K), dtype=torch.uint8, device="cuda")
    c = torch.empty(M, N, device="cuda")
    st = torch.cuda.Stream()

    def run():
        g.fp8_block_quantize(x, g.DTYPE_F32, M, K, K, 0, q, K, s, stream=st)
        g.gptx_gemm_fp8_block(M, N, K, q, K, s, qb, K, sb, g.DTYPE_F32, c, N, stream=st)

    torch.cuda.synchronize()
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        run()
    x.copy_(torch.from_numpy(values(rng, M, K)))
    graph.replay()
    torch.cuda.synchronize()
    got = c.clone()
    run()
    torch.cuda.synchronize()
    assert torch.equal(got, c)
    va = fb.decode(*fb.quantize(x.double().cpu().numpy(), 0))
    vb = fb.decode(qb.cpu().numpy(), g.fp8_block_scales(sb, N, K).cpu().numpy())
    assert (np.abs(c.cpu().numpy() - va @ vb.T) <= accumulation_bound(va, vb, K)).all()


def test_host_memory_is_refused(g):
    import torch
    x = torch.zeros(4, 16)
    q = torch.empty(4, 16, dtype=torch.uint8, device="cuda")
    s = torch.empty(512, dtype=torch.uint8, device="cuda")
    with pytest.raises(g.GptError) as e:
        g.fp8_block_quantize(x, g.DTYPE_F32, 4, 16, 16, 0, q, 16, s)
    assert e.value.code == g.GPT_ERR_ARG
