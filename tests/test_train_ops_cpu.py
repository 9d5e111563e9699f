"""Argument checks of the standalone training operators: every call below is
refused on the host before any device work (no GPU needed).  Addresses are
stand-ins that are never dereferenced."""

import ctypes

import pytest

import gpt_pretraining_step_decoder_b200 as g

A, B, C, D, E, WS = (i << 24 for i in range(1, 7))


def test_scale_bytes():
    assert g.fp8_block_scale_bytes(1, 1) == 512
    assert g.fp8_block_scale_bytes(129, 513) == 4 * 512
    for bad in ((0, 1), (1, 0), (-1, 5), (1 << 40, 1)):
        with pytest.raises(g.GptError) as e:
            g.fp8_block_scale_bytes(*bad)
        assert e.value.code == g.GPT_ERR_ARG


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(dtype=2), dict(ldx=99), dict(rows=-1), dict(cols=-1),
    dict(q=None, qt=None), dict(sc=None), dict(ldq=96), dict(ldq=104), dict(q=B + 8), dict(sc=C + 4),
    dict(sct=None), dict(ldqt=32), dict(ldqt=72), dict(qt=D + 1), dict(x=A + 2),
    dict(rows=1 << 40), dict(rows=(1 << 30) + 1, ldqt=1 << 31),
    dict(q=A), dict(q=A + 800), dict(sc=B + 16), dict(qt=B + 64), dict(sct=A + 400), dict(sc=D + 4096),  # overlaps
])
def test_quantize_refusals(bad):
    a = dict(x=A, dtype=g.DTYPE_F32, rows=50, cols=100, ldx=100, square=0, q=B, ldq=112, sc=C, qt=D, ldqt=64, sct=E)
    a.update(bad)
    assert g._lib.fp8_block_quantize(*a.values(), None) == g.GPT_ERR_ARG
    assert "fp8_block_quantize" in g.gpt_last_error()


def test_quantize_of_nothing_is_no_call():
    assert g._lib.fp8_block_quantize(A, 0, 0, 100, 100, 0, B, 112, C, None, 0, None, None) == g.GPT_OK
    assert g._lib.fp8_block_quantize(A, 0, 5, 0, 0, 0, B, 0, C, None, 0, None, None) == g.GPT_OK


@pytest.mark.parametrize("bad", [
    dict(M=0), dict(N=0), dict(K=0), dict(a=None), dict(sa=None), dict(sb=None), dict(c=None), dict(lda=999),
    dict(lda=1016), dict(ldb=500), dict(ldc=519), dict(ldc=521), dict(out=2), dict(beta=1, out=g.DTYPE_BF16),
    dict(a=A + 8), dict(c=C + 4), dict(sa=D + 8), dict(M=(1 << 30) + 1),
    dict(c=A), dict(c=B + 4096), dict(c=D), dict(c=E - 4096),                                            # overlaps
])
def test_gemm_refusals(bad):
    a = dict(M=777, N=520, K=1000, a=A, lda=1008, sa=D, b=B, ldb=1008, sb=E, out=g.DTYPE_F32, c=C, ldc=520, beta=0)
    a.update(bad)
    assert g._lib.gptx_gemm_fp8_block(*a.values(), None, 0, None) == g.GPT_ERR_ARG
    assert "gptx_gemm_fp8_block" in g.gpt_last_error()


def test_gemm_workspace():
    need = g.gptx_gemm_fp8_block_workspace_bytes(768, 768, 32768)
    assert need > 0 and need % (768 * 768 * 4) == 0          # a long K over few tiles is split
    assert g.gptx_gemm_fp8_block_workspace_bytes(32768, 2304, 768) == 0
    assert g._lib.gptx_gemm_fp8_block(768, 768, 32768, A, 32768, D, B, 32768, E, 0, C, 768, 0, WS, need - 1,
                                      None) == g.GPT_ERR_WORKSPACE
    assert g._lib.gptx_gemm_fp8_block(768, 768, 32768, A, 32768, D, B, 32768, E, 0, C, 768, 0, WS + 16, need,
                                      None) == g.GPT_ERR_ARG


def clip(grads, sizes, dtypes=None, outs=None, max_norm=1.0, ws=WS, ws_bytes=1 << 20):
    n = len(grads)
    P, L, I = ctypes.c_void_p * n, ctypes.c_longlong * n, ctypes.c_int * n
    return g._lib.grad_clip(n, P(*grads), None if outs is None else P(*outs), L(*sizes), I(*(dtypes or [0] * n)),
                            max_norm, None, ws, ws_bytes, None)


@pytest.mark.parametrize("kw", [
    dict(grads=[A], sizes=[-1]), dict(grads=[None], sizes=[3]), dict(grads=[A], sizes=[3], dtypes=[2]),
    dict(grads=[A], sizes=[3], max_norm=-1.0), dict(grads=[A], sizes=[3], max_norm=float("nan")),
    dict(grads=[A + 2], sizes=[3]), dict(grads=[A + 1], sizes=[3], dtypes=[1]),
    dict(grads=[A], sizes=[3], outs=[None]), dict(grads=[A], sizes=[3], outs=[B + 1]),
    dict(grads=[A, A], sizes=[4, 4]),                                  # the same tensor twice
    dict(grads=[B, A + 12, A], sizes=[4, 4, 4]),                       # overlapping, out of order
    dict(grads=[A, B], sizes=[4, 4], outs=[C, C + 8]),                 # overlapping outputs
    dict(grads=[A, B], sizes=[4, 4], outs=[B, C]),                     # an output that is another input
    dict(grads=[A, B], sizes=[4, 4], outs=[A + 8, C]),                 # shifted onto its own input
    dict(grads=[A, B], sizes=[4, 4], outs=[C, A]),
    dict(grads=[A], sizes=[4], ws=WS + 8),
])
def test_clip_refusals(kw):
    assert clip(**kw) == g.GPT_ERR_ARG
    assert g.gpt_last_error()


def test_clip_workspace_refusal():
    need = g.grad_clip_workspace_bytes(3)
    assert clip([A], [4], ws_bytes=need - 1) == g.GPT_ERR_WORKSPACE
    assert clip([A], [4], ws=None) == g.GPT_ERR_WORKSPACE
    assert g.grad_clip_workspace_bytes(1025) == 2 * need
    with pytest.raises(g.GptError):
        g.grad_clip_workspace_bytes(-1)


CE = dict(x=A, ldx=64, w=B, ldw=64, dtype=g.DTYPE_BF16, N=10, V=100, d=64, t=C, cap=0.0)


def ce_forward(loss=D, ws=WS, ws_bytes=1 << 30, piece=0, **kw):
    a = dict(CE, **kw)
    return g._lib.linear_ce_forward(*a.values(), loss, None, None, piece, ws, ws_bytes, None)


def ce_backward(lse=D, dloss=None, dtok=None, dx=E, lddx=64, dw=E + (1 << 20), lddw=64, dwt=g.DTYPE_BF16, beta=0,
                ws=WS, ws_bytes=1 << 30, piece=0, **kw):
    a = dict(CE, **kw)
    return g._lib.linear_ce_backward(*a.values(), lse, dloss, dtok, dx, lddx, dw, lddw, dwt, beta, piece, ws, ws_bytes,
                                     None)


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(w=None), dict(t=None), dict(dtype=2), dict(N=-1), dict(V=0), dict(d=0), dict(ldx=56), dict(ldw=56),
    dict(cap=-1.0), dict(cap=float("nan")), dict(cap=float("inf")), dict(d=60), dict(ldx=68), dict(ldw=68), dict(x=A + 8),
    dict(w=B + 2), dict(t=C + 2), dict(dtype=g.DTYPE_F32, x=A + 2), dict(piece=-1), dict(ws=WS + 16),
])
def test_ce_refusals(bad):
    assert ce_forward(**bad) == g.GPT_ERR_ARG
    assert ce_backward(**bad) == g.GPT_ERR_ARG
    assert g.gpt_last_error()


@pytest.mark.parametrize("bad", [
    dict(lse=None), dict(dx=None, dw=None), dict(lddx=56), dict(lddw=56), dict(dloss=A, dtok=A), dict(dwt=2),
    dict(beta=1), dict(dx=E + 8), dict(lddx=68), dict(dw=E + 8), dict(lddw=68), dict(dtype=g.DTYPE_F32),
    dict(dx=A), dict(dw=B), dict(dw=E), dict(dx=B + 128), dict(dx=D), dict(dw=C), dict(dw=WS), dict(dx=A + 64 * 20 - 16),
])
def test_ce_backward_refusals(bad):
    assert ce_backward(**bad) == g.GPT_ERR_ARG


def test_ce_forward_overlaps():
    for bad in (A, B + 64, C, WS):
        assert ce_forward(loss=bad) == g.GPT_ERR_ARG
        assert "overlaps" in g.gpt_last_error()


def test_columns_side_by_side_do_not_overlap():
    """A gradient in the other half of rows that also hold its input is no overlap
    (the call goes on to the device, which this machine does not have)."""
    st = ce_backward(ldx=128, lddx=128, dx=A + 128, dw=None)
    assert st != g.GPT_ERR_ARG or "overlaps" not in g.gpt_last_error()
    assert ce_backward(ldx=128, lddx=128, dx=A + 112, dw=None) == g.GPT_ERR_ARG
    assert "overlaps" in g.gpt_last_error()


def test_ce_workspace():
    assert ce_forward(loss=None) == g.GPT_ERR_ARG
    for dtype in (g.DTYPE_BF16, g.DTYPE_F32):
        for back in (0, 1):
            assert g.linear_ce_workspace_bytes(0, 100, 64, dtype, back) >= 0
    for call, back in ((ce_forward, 0), (ce_backward, 1)):
        need = g.linear_ce_workspace_bytes(10, 100, 64, g.DTYPE_BF16, back)
        assert need > 0 and call(ws_bytes=need - 1) == g.GPT_ERR_WORKSPACE
        assert call(ws=None) == g.GPT_ERR_WORKSPACE
    # a smaller piece of the vocabulary takes less memory, and the pieces are bounded
    big = g.linear_ce_workspace_bytes(16384, 65536, 2048, g.DTYPE_BF16, 1)
    assert g.linear_ce_workspace_bytes(16384, 65536, 2048, g.DTYPE_BF16, 1, 1024) < big < 1 << 30
    with pytest.raises(g.GptError):
        g.linear_ce_workspace_bytes(1, 1, 1, 7, 0)
    with pytest.raises(g.GptError):
        g.linear_ce_workspace_bytes(1, 1, 1, 0, 0, -1)
