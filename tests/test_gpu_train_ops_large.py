"""The standalone training operators at shapes that take the forms of large calls:
tiles shared by SM pairs, 256 columns, several tiles per CTA, runs of column tiles
over several row blocks, the quantizer's later tiles, split products.  Every test
asserts the form that it is about.  References in fp64 on the GPU, from elementary
operations; tolerances as in the tests of the small shapes (each is derived there:
tests/test_gpu_linear_ce.py, tests/test_gpu_fp8_block.py)."""

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import torch
    import gpt_pretraining_step_decoder_b200 as g
    assert torch.cuda.is_available()
    return g


@pytest.fixture(params=[True, False], ids=["sm_pairs", "one_sm"])
def pairs(request, g):
    g.gptx_set_gemm_cta_pairs(request.param)
    yield request.param
    g.gptx_set_gemm_cta_pairs(True)


def pitch(n):
    return -(-n // 16) * 16


# ------------------------------------------------------------------ block-scaled e4m3
def stored(s, rows, groups):
    """Scale bytes [rows, groups] in 512-byte atoms, 200 in what the atoms have beyond."""
    ra, ga = -(-rows // 128), -(-groups // 4)
    full = s.new_full((ra * 128, ga * 4), 200)
    full[:rows, :groups] = s
    return full.view(ra, 4, 32, ga, 4).permute(3, 0, 2, 1, 4).reshape(-1).contiguous()


def operand(rows, K, gen):
    """Random finite codes and scales: (codes with a pitch of NaNs, stored scales, values in fp64)."""
    import torch
    q = torch.full((rows, pitch(K) + 16), 0x7F, dtype=torch.uint8, device="cuda")
    code = torch.randint(0, 254, (rows, K), generator=gen, device="cuda", dtype=torch.int32)
    code += (code >= 127).int()                    # 0x7f and 0xff are NaN
    q[:, :K] = code.to(torch.uint8)
    groups = -(-K // 128)
    s = torch.randint(118, 130, (rows, groups), generator=gen, device="cuda", dtype=torch.int32).to(torch.uint8)
    v = q[:, :K].view(torch.float8_e4m3fn).double() * torch.exp2(s.double() - 127).repeat_interleave(128, 1)[:, :K]
    return q, stored(s, rows, groups), v


# (M, N, K): the form with pairs on, with pairs off (shares of K > 1: True)
PRODUCTS = [
    ((20001, 2312, 776), (256, 2, False), (256, 1, False)),     # many tiles per pair, ragged everywhere
    ((4100, 4104, 128), (256, 1, False), (256, 1, False)),      # one k-block, several tiles per SM
    ((50001, 120, 776), (128, 1, False), (128, 1, False)),
    ((30001, 5, 200), (128, 1, False), (128, 1, False)),        # a width that is no multiple of 4
    ((700, 1000, 20000), (256, 2, True), (256, 1, True)),
    ((1300, 2056, 9001), (256, 2, False), (256, 1, False)),     # fp32: chunks of K behind one accumulator
]


@pytest.mark.parametrize("out", ["f32", "beta", "bf16"])
@pytest.mark.parametrize("size,on,off", PRODUCTS, ids=[str(p[0]) for p in PRODUCTS])
def test_product(g, pairs, size, on, off, out):
    import torch
    M, N, K = size
    plan = g.gptx_gemm_fp8_block_plan(M, N, K)
    assert (plan[0], plan[1], plan[2] > 1) == (on if pairs else off)
    if plan[2] == 1:   # several tiles for some unit of the device
        assert -(-M // (128 * plan[1])) * -(-N // plan[0]) > 148 // plan[1] or K > 2048
    gen = torch.Generator(device="cuda").manual_seed(M + K)
    (qa, sa, va), (qb, sb, vb) = operand(M, K, gen), operand(N, K, gen)
    n = g.gptx_gemm_fp8_block_workspace_bytes(M, N, K)
    ws = torch.full((max(n, 256),), 0xFF, dtype=torch.uint8, device="cuda")
    ldc, dt = -(-N // 8) * 8 + 8, torch.bfloat16 if out == "bf16" else torch.float32
    c = torch.full((M + 2, ldc), 3.0, dtype=dt, device="cuda")
    g.gptx_gemm_fp8_block(M, N, K, qa, qa.shape[1], sa, qb, qb.shape[1], sb, g.DTYPE_BF16 if out == "bf16" else g.DTYPE_F32,
                          c, ldc, out == "beta", ws, n)
    torch.cuda.synchronize()
    assert g.ngram_sync_status() == g.GPT_OK, g.gpt_last_error()
    assert (c[M:] == 3).all() and (c[:, N:] == 3).all()         # rows behind the last, columns behind a row
    ref = va @ vb.T
    tol = (K + 16) * 2.0 ** -23 * (va.abs() @ vb.abs().T)
    got = c[:M, :N].double()
    if out == "beta":
        ref += 3
        tol += 2.0 ** -23 * (ref.abs() + 3)
    if out == "bf16":
        tol += 2.0 ** -8 * (ref.abs() + tol)
    assert ((got - ref).abs() <= tol).all(), (got - ref).abs().max()


def quantize_plain(x, square):
    """Codes and scale bytes [rows, groups] from the definition, in fp64."""
    import torch
    x = x.double()
    rows, cols = x.shape
    rb, cb = -(-rows // 128), -(-cols // 128)
    a = x.new_zeros(rb * 128, cb * 128)
    a[:rows, :cols] = x.abs()
    amax = a.view(rb, 128, cb, 128).amax((1, 3)).repeat_interleave(128, 0)[:rows] if square else a.view(-1, cb, 128).amax(2)[:rows]
    e = torch.floor(torch.log2(amax.clamp(min=1e-300))) - 9     # 448 = 0.875 * 2^9: at most two below the least
    for _ in range(3):
        e = torch.where(amax > 448 * torch.exp2(e), e + 1, e)
    e = torch.where(amax == 0, 0.0, e.clamp(min=-127))
    v = (x * torch.exp2(-e).repeat_interleave(128, 1)[:, :cols]).float()     # exact, at most 448
    return v.to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8)


@pytest.mark.parametrize("pad", [0, 11])
@pytest.mark.parametrize("square", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantizer_beyond_the_first_tiles(g, dtype, square, pad):
    """760 tiles, more than twice the persistent blocks; with pad 11 the rows are
    16-byte aligned and the tiles arrive by TMA, with 0 by plain loads."""
    import torch
    rows, cols = 5003, 2309
    assert -(-rows // 128) * -(-cols // 128) > 2 * 2 * torch.cuda.get_device_properties(0).multi_processor_count
    gen = torch.Generator(device="cuda").manual_seed(rows)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = torch.full((rows, cols + pad), 3e4, dtype=dt, device="cuda")
    x[:, :cols] = torch.randn(rows, cols, generator=gen, device="cuda") * torch.exp2(
        12 * torch.rand(rows, 1, generator=gen, device="cuda") - 6)
    x[130, 140:300] = 0
    out = []
    for r, c in ((rows, cols), (cols, rows)):
        out.append((torch.full((r + 1, pitch(c)), 0xA5, dtype=torch.uint8, device="cuda"),
                    torch.full((g.fp8_block_scale_bytes(r, c),), 0xA5, dtype=torch.uint8, device="cuda")))
    (q, s), (qt, st) = out
    g.fp8_block_quantize(x, g.DTYPE_BF16 if dtype == "bf16" else g.DTYPE_F32, rows, cols, cols + pad, square, q, pitch(cols),
                         s, qt, pitch(rows), st)
    torch.cuda.synchronize()
    for m, (codes, scales) in ((x[:, :cols], out[0]), (x[:, :cols].T, out[1])):
        r, c = m.shape
        want, by = quantize_plain(m, square)
        assert torch.equal(codes[:r, :c], want)
        assert (codes[r:] == 0xA5).all() and (codes[:, c:] == 0xA5).all()
        assert torch.equal(g.fp8_block_scales(scales, r, c), by)
        full = stored(by, r, by.shape[1])
        full[full == 200] = 127
        assert torch.equal(scales, full)
    assert g.ngram_sync_status() == g.GPT_OK


# ------------------------------------------------------------------ cross entropy
class Loss:
    """One call's inputs with its fp64 reference and tolerances, rows in pieces."""

    def __init__(self, N, V, d, cap, seed=0, dtype="bf16", spread=2.0):
        import torch
        gen = torch.Generator(device="cuda").manual_seed(seed + N + V)
        self.N, self.V, self.d, self.cap = N, V, d, cap
        self.dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.code = 1 if dtype == "bf16" else 0
        self.x = torch.randn(N, d, generator=gen, device="cuda").to(self.dt)
        self.w = (torch.randn(V, d, generator=gen, device="cuda") * spread / d ** 0.5).to(self.dt)
        t = torch.randint(0, V, (N,), generator=gen, device="cuda", dtype=torch.int32)
        self.t = torch.where(torch.rand(N, generator=gen, device="cuda") < 0.1, -1, t).to(torch.int32)
        self.t[-1] = V - 1                             # the last row's target in the last column

    def rows(self):
        """Per piece of rows: slice, z, error of z, lse, error of lse, slope."""
        import torch
        x, w = self.x.double(), self.w.double()
        aw = w.abs()
        step = max(1, (1 << 27) // self.V)
        for i in range(0, self.N, step):
            r = slice(i, i + step)
            z = x[r] @ w.T
            ez = (self.d + 16) * 2.0 ** -23 * (x[r].abs() @ aw.T)
            slope = None
            if self.cap:
                z = self.cap * torch.tanh(z / self.cap)
                ez += z.abs() * 2.0 ** -19 if self.cap > 64 else self.cap * 2.0 ** -19
                slope = 1 - (z / self.cap).square()
            lse = torch.logsumexp(z, 1)
            yield r, z, ez, lse, ez.amax(1) + 2.0 ** -22 * (8 + 3 * z.abs().amax(1)), slope

    def forward(self, g):
        import torch
        n = g.linear_ce_workspace_bytes(self.N, self.V, self.d, self.code, 0)
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
        loss, tok, lse = (torch.full((k + 2,), 77.0, device="cuda") for k in (1, self.N, self.N))
        g.linear_ce_forward(self.x, self.d, self.w, self.d, self.code, self.N, self.V, self.d, self.t, self.cap, loss, tok,
                            lse, ws, n)
        torch.cuda.synchronize()
        assert g.ngram_sync_status() == g.GPT_OK, g.gpt_last_error()
        assert all((v[-2:] == 77).all() for v in (loss, tok, lse))
        return loss[:1], tok[:-2], lse[:-2]

    def check_forward(self, got):
        import torch
        loss, tok, lse = got
        total, most = 0.0, 0.0
        for r, z, ez, l0, tol, _ in self.rows():
            assert ((lse[r].double() - l0).abs() <= tol).all()
            t = self.t[r].long()
            t0 = torch.where(t >= 0, l0 - z.gather(1, t.clamp(min=0)[:, None]).squeeze(1), 0.0)
            tt = tol + ez.amax(1) + 2.0 ** -23 * (l0.abs() + t0.abs())
            assert ((tok[r].double() - t0).abs() <= tt).all() and (tok[r][t < 0] == 0).all()
            total += t0.sum().item()
            most = max(most, tt.max().item())
        mean = total / (self.t >= 0).sum().item()
        assert abs(loss.item() - mean) <= most + 2.0 ** -23 * abs(mean)

    def check_backward(self, g, dtok=None, dw_dtype=None, beta=0):
        import torch
        N, V, d = self.N, self.V, self.d
        n = g.linear_ce_workspace_bytes(N, V, d, self.code, 1)
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
        dw_dtype = self.code if dw_dtype is None else dw_dtype
        lse = torch.cat([l0 for _, _, _, l0, _, _ in self.rows()])
        gx = torch.full((N + 2, d), 5.0, dtype=self.dt, device="cuda")
        gw = torch.full((V + 2, d), 1e-3, dtype=torch.bfloat16 if dw_dtype else torch.float32, device="cuda")
        base = gw[0, 0].double().item() if beta else 0.0
        dloss = None if dtok is not None else torch.full((1,), 1.5, device="cuda")
        g.linear_ce_backward(self.x, d, self.w, d, self.code, N, V, d, self.t, self.cap, lse.float(), dloss, dtok, gx, d, gw,
                             d, dw_dtype, beta, ws, n)
        torch.cuda.synchronize()
        assert g.ngram_sync_status() == g.GPT_OK, g.gpt_last_error()
        assert (gx[N:] == 5).all() and (gw[V:] == gw.new_tensor(1e-3)).all()
        x, w = self.x.double(), self.w.double()
        valid = self.t >= 0
        scale = dtok.double() if dtok is not None else torch.full((N,), 1.5 / valid.sum().item(), dtype=torch.float64, device="cuda")
        scale = torch.where(valid, scale, 0.0)
        w0, e0, m0 = (torch.zeros(V, d, dtype=torch.float64, device="cuda") for _ in range(3))
        step_w = 2.0 ** -8 if gw.dtype == torch.bfloat16 else 2.0 ** -23
        step_x = 2.0 ** -8 if self.code else 2.0 ** -23
        for r, z, ez, l0, tol, slope in self.rows():
            p = (z - l0[:, None]).exp()
            gr = scale[r][:, None]
            rows = torch.nonzero(valid[r]).squeeze(1)
            at = (rows, self.t[r][rows].long())
            dz = p.clone()
            dz[at] -= 1
            dz *= gr
            e = p * gr.abs() * 2 * (ez + tol[:, None])
            if self.cap:
                dz *= slope
                hot = p
                hot[at] += 1
                e += hot * gr.abs() * 2.0 ** -17
            e += 2.0 ** -21 * dz.abs()
            if self.code:
                e += 2.0 ** -8 * (dz.abs() + e) + 2.0 ** -133
            mag = dz.abs() + e
            ref = dz @ w
            bound = e @ w.abs() + (V + 16) * 2.0 ** -22 * (mag @ w.abs())
            bound += step_x * (ref.abs() + bound)
            assert ((gx[r.start:min(r.stop, N)].double() - ref).abs() <= bound + 1e-30).all()
            w0 += dz.T @ x[r]
            e0 += e.T @ x[r].abs()
            m0 += mag.T @ x[r].abs()
        assert not gx[:N][~valid].any()
        bound = e0 + (N + 16) * 2.0 ** -22 * m0
        w0 += base
        bound += 2.0 ** -23 * (w0.abs() + base)
        bound += step_w * (w0.abs() + bound)
        assert ((gw[:V].double() - w0).abs() <= bound + 1e-30).all()


CAPS = [0.0, 15.0, 100.0]


# (N, V, d): the loss's product with pairs on, off (columns, SMs, tiles in a run)
LOSSES = [
    ((12500, 50400, 256), (256, 2, 4), (256, 1, 4)),      # runs of four over several row blocks
    ((40001, 200, 64), (128, 1, 1), (128, 1, 1)),         # several tiles of 128 columns per SM
    ((300, 16384, 776), (256, 2, 1), (128, 1, 1)),
    ((131, 57048, 80), (256, 2, 4), (256, 1, 1)),         # the second row block nearly empty
    ((33, 50304, 768), (128, 1, 3), (128, 1, 3)),         # one row block: a run for every SM
    ((33, 50048, 64), (256, 1, 2), (256, 1, 2)),
    ((2100, 5003, 2056), (256, 2, 1), (256, 1, 1)),       # chunks of d between the tiles
]


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("size,on,off", LOSSES, ids=[str(p[0]) for p in LOSSES])
def test_loss(g, pairs, size, on, off, cap):
    assert g.linear_ce_plan(*size, g.DTYPE_BF16, 0)["logits"] == (on if pairs else off)
    c = Loss(*size, cap)
    c.check_forward(c.forward(g))


# (N, V, d): (columns, SMs, split?) of the products of z, dx and dW with pairs on, off
GRADIENTS = [
    ((12500, 50400, 256), ((256, 2), (256, 2, True), (256, 2, False)), ((256, 1), (256, 1, True), (256, 1, False))),
    ((6001, 4100, 264), ((256, 2), (128, 1, False), (256, 2, True)), ((256, 1), (128, 1, False), (256, 1, True))),
    ((1100, 4104, 1032), ((256, 2), (256, 1, True), (256, 2, False)), ((128, 1), (256, 1, True), (128, 1, False))),
    ((300, 20000, 2056), ((256, 1), (256, 2, True), (256, 2, False)), ((256, 1), (256, 1, True), (256, 1, False))),
    ((40001, 200, 64), ((128, 1), (128, 1, False), (128, 1, True)), ((128, 1), (128, 1, False), (128, 1, True))),
]


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("size,on,off", GRADIENTS, ids=[str(p[0]) for p in GRADIENTS])
def test_gradient(g, pairs, size, on, off, cap):
    p = g.linear_ce_plan(*size, g.DTYPE_BF16, 1)
    forms = (p["logits"][:2], *((*p[k][:2], p[k][2] > 1) for k in ("dx", "dw")))
    assert forms == (on if pairs else off)
    Loss(*size, cap).check_backward(g)


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("beta", [0, 1])
def test_gradient_of_token_losses_with_fp32_weight_gradient(g, pairs, cap, beta):
    """dtok, and dW in fp32, overwritten and added to, in several pieces of the
    vocabulary and with dW's product split (the last piece's)."""
    import torch
    for N, V, d in ((12500, 50400, 256), (6001, 4100, 264)):
        gen = torch.Generator(device="cuda").manual_seed(N)
        c = Loss(N, V, d, cap)
        dtok = torch.randn(N, generator=gen, device="cuda") / N
        dtok[::7] = 0
        c.check_backward(g, dtok=dtok, dw_dtype=g.DTYPE_F32, beta=beta)


@pytest.mark.parametrize("cap", [0.0, 15.0])
@pytest.mark.parametrize("N,V,d", [(5003, 4101, 77), (700, 20001, 129)])
def test_fp32(g, N, V, d, cap):
    """Above 512 rows the targets are counted by a launch of their own."""
    c = Loss(N, V, d, cap, dtype="f32")
    c.check_forward(c.forward(g))
    c.check_backward(g)
