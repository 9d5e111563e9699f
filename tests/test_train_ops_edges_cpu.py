"""More argument checks of the standalone training operators, made on the host
before any device work (no GPU needed).  Addresses are stand-ins that are never
dereferenced; a call that passes the checks goes on to the device, which this
machine may not have, and ends with another status."""

import ctypes

import pytest

import gpt_pretraining_step_decoder_b200 as g

A, B, C, D, E, F, WS = (i << 24 for i in range(1, 8))


def ce_forward(loss=D, tok=E, lse=F, **kw):
    a = dict(x=A, ldx=64, w=B, ldw=64, dtype=g.DTYPE_BF16, N=10, V=100, d=64, t=C, cap=0.0)
    a.update(kw)
    return g._lib.linear_ce_forward(*a.values(), loss, tok, lse, 0, WS, 1 << 30, None)


def ce_backward(lse=D, dloss=None, dtok=None, dx=E, dw=F, **kw):
    a = dict(x=A, ldx=64, w=B, ldw=64, dtype=g.DTYPE_BF16, N=10, V=100, d=64, t=C, cap=0.0)
    a.update(kw)
    return g._lib.linear_ce_backward(*a.values(), lse, dloss, dtok, dx, 64, dw, 64, a["dtype"], 0, 0, WS, 1 << 30, None)


def clip(grads, sizes, dtypes=None, outs=None, max_norm=1.0, norm=None, ws=WS, ws_bytes=1 << 20):
    n = len(grads)
    P, L, I = ctypes.c_void_p * n, ctypes.c_longlong * n, ctypes.c_int * n
    return g._lib.grad_clip(n, P(*grads), None if outs is None else P(*outs), L(*sizes), I(*(dtypes or [0] * n)),
                            max_norm, norm, ws, ws_bytes, None)


@pytest.mark.parametrize("dtype", [g.DTYPE_BF16, g.DTYPE_F32])
@pytest.mark.parametrize("off", [1, 2])
def test_fp32_vectors_off_their_alignment(dtype, off):
    """Every float that a kernel reads or writes has to lie on 4 bytes."""
    for bad in (dict(loss=D + off), dict(tok=E + off), dict(lse=F + off)):
        assert ce_forward(dtype=dtype, **bad) == g.GPT_ERR_ARG
        assert "aligned" in g.gpt_last_error()
    for bad in (dict(lse=D + off), dict(dloss=D + 4096 + off), dict(dtok=D + 4096 + off)):
        assert ce_backward(dtype=dtype, **bad) == g.GPT_ERR_ARG
        assert "aligned" in g.gpt_last_error()
    assert clip([A], [3], norm=D + off) == g.GPT_ERR_ARG
    assert "aligned" in g.gpt_last_error()


@pytest.mark.parametrize("kw", [
    dict(grads=[A], sizes=[4], norm=WS), dict(grads=[A], sizes=[4], norm=WS + 1024), dict(grads=[], sizes=[], norm=WS + 8),
    dict(grads=[A], sizes=[4], norm=A + 12), dict(grads=[A], sizes=[4], outs=[B], norm=A),
    dict(grads=[A], sizes=[4], outs=[B], norm=B + 4), dict(grads=[A, WS - 8], sizes=[4, 4]),
    dict(grads=[A, WS + 512], sizes=[4, 4], dtypes=[0, 1]), dict(grads=[A, B], sizes=[4, 1 << 25], outs=[C, F - 512]),
])
def test_clip_norm_and_workspace_lie_apart(kw):
    """The norm is written while the partials and the tensors are still read."""
    assert clip(**kw) == g.GPT_ERR_ARG
    assert "overlaps" in g.gpt_last_error()


def test_clip_neighbours_of_norm_and_workspace_pass():
    need = g.grad_clip_workspace_bytes(1)
    for kw in (dict(grads=[A], sizes=[4], norm=A + 16), dict(grads=[A], sizes=[4], norm=A - 4),
               dict(grads=[WS - 16], sizes=[4], norm=WS + need), dict(grads=[WS + 8], sizes=[0])):
        clip(**kw)
        assert "overlaps" not in g.gpt_last_error()


def test_norm_alone_of_tensors_that_share_memory():
    """max_norm = 0 in place writes no tensor: a weight listed twice is no overlap."""
    for kw in (dict(grads=[A, A], sizes=[4, 4]), dict(grads=[A, A + 8, A], sizes=[4, 4, 1])):
        clip(max_norm=0.0, **kw)
        assert "overlaps" not in g.gpt_last_error()
        assert clip(max_norm=1.0, **kw) == g.GPT_ERR_ARG
        assert clip(max_norm=0.0, outs=[B + 64 * i for i in range(len(kw["grads"]) - 1)] + [A], **kw) == g.GPT_ERR_ARG


def test_clip_of_an_iterator_of_tensors():
    """A generator's tensors all reach the call (the same one twice is refused there)."""
    import torch
    t, u = torch.zeros(4), torch.zeros(4)
    for grads, outs in (((x for x in (t, t)), None), (iter([t, u]), (x for x in (t, t)))):
        with pytest.raises(g.GptError) as e:
            g.grad_clip(grads, outs, 1.0, None, WS, 1 << 20)
        assert e.value.code == g.GPT_ERR_ARG and "overlaps" in str(e.value)
    with pytest.raises(ValueError):
        g.grad_clip((x for x in (t, u)), (x for x in (t,)), 1.0, None, WS, 1 << 20)


@pytest.mark.parametrize("rows,cols", [(0, 100), (5, 0), (0, 0)])
@pytest.mark.parametrize("dtype", [g.DTYPE_BF16, g.DTYPE_F32])
def test_quantize_of_an_empty_tensor(rows, cols, dtype):
    """An empty tensor's address is null: still no call, in either orientation."""
    assert g._lib.fp8_block_quantize(None, dtype, rows, cols, cols, 0, None, 0, None, None, 0, None, None) == g.GPT_OK
    assert g._lib.fp8_block_quantize(None, dtype, rows, cols, cols, 1, None, 112, C, D, 0, None, None) == g.GPT_OK
    assert g._lib.fp8_block_quantize(None, 2, rows, cols, cols, 0, None, 0, None, None, 0, None, None) == g.GPT_ERR_ARG
    assert g._lib.fp8_block_quantize(None, dtype, -1, cols, cols, 0, None, 0, None, None, 0, None, None) == g.GPT_ERR_ARG


def test_ce_of_no_rows_with_empty_outputs():
    """N = 0: per-token outputs and dx are empty, their addresses null; the call passes the checks."""
    for st in (ce_forward(N=0, x=None, t=None, loss=None, tok=None, lse=None),
               ce_backward(N=0, x=None, t=None, lse=None, dx=None, dw=None)):
        assert st != g.GPT_ERR_ARG or "device" in g.gpt_last_error()
    assert ce_forward(loss=None, tok=None, lse=None) == g.GPT_ERR_ARG
    assert ce_backward(dx=None, dw=None) == g.GPT_ERR_ARG


@pytest.mark.parametrize("N,V", [(1000, 10_000_000), (1, 1 << 30), (64, 1 << 28)])
def test_choice_of_the_vocabulary_pieces_is_quick(N, V):
    """Every gradient call chooses its pieces; a huge vocabulary of few rows must not
    cost more host time than a launch does."""
    import time
    best = 1.0
    for _ in range(50):
        t0 = time.perf_counter()
        g.linear_ce_workspace_bytes(N, V, 64, g.DTYPE_BF16, 1)
        best = min(best, time.perf_counter() - t0)
    assert best < 40e-6, best
