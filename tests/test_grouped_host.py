"""Refusals of the grouped and 8-bit integer entry points: every bad argument
comes back as its status before anything is enqueued, so no GPU is needed.
Pointers are fake aligned addresses that validation never follows."""
import ctypes

import pytest
import torch

A = 0x100000


@pytest.fixture(scope="module")
def fp8():
    import fp8_delayed_scaling_03_b200 as m
    return m


def groups(fp8, **kw):
    g = dict(groups=4, offsets=A, offsets_64=0, stride_b=128 * 128, stride_d=0, scale_b_step=1)
    g.update(kw)
    return fp8.Groups(**g)


def grouped(fp8, ragged=0, g=None, **kw):
    a = dict(m=128, n=128, k=128, a=A, fmt_a=0, a_major=0, lda=128, b=A, fmt_b=0, b_major=0, ldb=128, scale_a=A,
             scale_b=A, bias=None, bias_dtype=0, bias_scale=None, d=A, ldd=128, tile_cfg=0, workspace=None,
             workspace_bytes=0)
    if ragged == 1:
        a.update(a_major=1, b_major=1)
    a.update(kw)
    args = fp8.MmArgs(**a)
    return fp8._lib.fp8_mm_grouped(ctypes.byref(args), ragged, ctypes.byref(groups(fp8, **(g or {}))), None)


def test_grouped_refusals(fp8):
    E = fp8
    bad, mis, uns, big = E.FP8_ERR_INVALID_ARG, E.FP8_ERR_MISALIGNED, E.FP8_ERR_UNSUPPORTED, E.FP8_ERR_TOO_LARGE
    assert fp8._lib.fp8_mm_grouped(None, 0, None, None) == bad
    for ragged in (0, 1):
        for kw in (dict(m=-1), dict(n=1 << 31), dict(n=(1 << 31) - 1), dict(k=-5), dict(fmt_a=2), dict(fmt_b=-1), dict(scale_a=None),
                   dict(scale_b=None), dict(a_major=7), dict(a=None), dict(b=None), dict(lda=100), dict(ldb=112),
                   dict(d=None), dict(ldd=127), dict(d=A + 1)):
            assert grouped(fp8, ragged, **kw) == bad, (ragged, kw)
        for kw in (dict(a=A + 8), dict(b=A + 1), dict(lda=136), dict(ldb=136)):
            assert grouped(fp8, ragged, **kw) == mis, (ragged, kw)
        assert grouped(fp8, ragged, bias=A) == uns
        for cfg in (1, 3, 4, 9):
            assert grouped(fp8, ragged, tile_cfg=cfg) == uns
        for g in (dict(groups=-1), dict(offsets=None), dict(offsets=A + 2), dict(offsets_64=1, offsets=A + 4),
                  dict(offsets_64=2), dict(scale_b_step=2), dict(stride_b=-16), dict(stride_d=-1)):
            assert grouped(fp8, ragged, g) == bad, (ragged, g)
        assert grouped(fp8, ragged, dict(groups=1025)) == big
    assert grouped(fp8, 2) == bad
    assert grouped(fp8, 0, a_major=1) == uns
    assert grouped(fp8, 1, a_major=0) == uns and grouped(fp8, 1, b_major=0) == uns
    assert grouped(fp8, 0, dict(stride_b=128 * 128 + 8)) == mis
    assert grouped(fp8, 0, dict(stride_b=64 * 128)) == bad          # the groups' weights overlap
    assert grouped(fp8, 1, dict(stride_d=128 * 128 - 1)) == bad     # the groups' gradients overlap


def test_grouped_empty_sizes_enqueue_nothing(fp8):
    none = dict(a=None, b=None, d=None, lda=0, ldb=0, ldd=0)
    assert grouped(fp8, 0, dict(groups=0, offsets=None)) == fp8.FP8_OK
    assert grouped(fp8, 0, m=0, **none | dict(b=A, ldb=128)) == fp8.FP8_OK
    assert grouped(fp8, 0, n=0, **none | dict(a=A, lda=128)) == fp8.FP8_OK
    assert grouped(fp8, 1, m=0, **none | dict(b=A, ldb=128)) == fp8.FP8_OK
    assert grouped(fp8, 1, n=0, **none | dict(a=A, lda=128)) == fp8.FP8_OK


def int8(fp8, **kw):
    a = dict(m=16, n=32, k=64, a=A, lda=64, b=A, ldb=64, scale_a=A, scale_b=A, bias=None, bias_dtype=0, d=A, d_dtype=0,
             ldd=32)
    a.update(kw)
    args = fp8.MmInt8Args(**a)
    return fp8._lib.fp8_mm_int8(ctypes.byref(args), None)


def test_int8_refusals(fp8):
    E = fp8
    assert fp8._lib.fp8_mm_int8(None, None) == E.FP8_ERR_INVALID_ARG
    for kw in (dict(m=-1), dict(n=-1), dict(k=-1), dict(m=1 << 31), dict(m=(1 << 31) - 1024), dict(a=None), dict(b=None), dict(lda=48), dict(ldb=48),
               dict(scale_a=None), dict(scale_b=None), dict(scale_a=A + 2), dict(scale_b=A + 1), dict(d=None), dict(ldd=31),
               dict(d=A + 1), dict(d=A + 2, d_dtype=2), dict(d_dtype=3), dict(d_dtype=-1), dict(bias=A, bias_dtype=3),
               dict(bias=A + 1), dict(bias=A + 2, bias_dtype=2)):
        assert int8(fp8, **kw) == E.FP8_ERR_INVALID_ARG, kw
    for kw in (dict(a=A + 4), dict(b=A + 8), dict(lda=72), dict(ldb=65)):
        assert int8(fp8, **kw) == E.FP8_ERR_MISALIGNED, kw
    assert int8(fp8, k=131072, lda=131072, ldb=131072) == E.FP8_ERR_TOO_LARGE
    assert int8(fp8, m=0, a=None, d=None, scale_a=None) == E.FP8_OK
    assert int8(fp8, n=0, b=None, d=None, scale_b=None) == E.FP8_OK


def test_quantize_int8_refusals(fp8):
    E = fp8

    def q(inp=A, dt=0, rows=4, cols=32, ld=32, out=A, ldo=32, scale=A):
        return fp8._lib.fp8_quantize_int8(inp, dt, rows, cols, ld, out, ldo, scale, None)

    for kw in (dict(inp=None), dict(out=None), dict(scale=None), dict(dt=3), dict(dt=-1), dict(rows=-1), dict(cols=-1),
               dict(rows=1 << 31), dict(ld=31), dict(ldo=16), dict(inp=A + 1), dict(inp=A + 2, dt=2), dict(scale=A + 2)):
        assert q(**kw) == E.FP8_ERR_INVALID_ARG, kw
    assert q(ldo=40) == E.FP8_ERR_MISALIGNED and q(out=A + 8) == E.FP8_ERR_MISALIGNED
    assert q(rows=0, inp=None, out=None, scale=None) == E.FP8_OK
    assert q(cols=0, ld=0, ldo=0, inp=None, out=None) == E.FP8_OK


def test_linear_refusals(fp8):
    E = fp8
    bad, uns = E.FP8_ERR_INVALID_ARG, E.FP8_ERR_UNSUPPORTED

    def fwd(gr=None, **kw):
        a = dict(M=64, N=64, K=64, x=A, x_dtype=0, ldx=64, w=A, w_dtype=0, ldw=64, hist_len=4, ring_x=A, ring_w=A + 256,
                 x8=A, ldx8=64, w8=A, ldw8=64, sx_out=A, sw_out=A, y=A, ldy=64)
        a.update(kw)
        gs = groups(fp8, **(dict(stride_b=0, scale_b_step=0) | (gr or {})))
        return fp8._lib.fp8_linear_grouped_forward(ctypes.byref(fp8.LinearFwdArgs(**a)), ctypes.byref(gs), None)

    def bwd(gr=None, **kw):
        a = dict(M=64, N=64, K=64, g=A, g_dtype=0, ldg=64, fmt_g=1, hist_len=4, ring_g=A, g8=A, ldg8=64, sg_out=A, x8=A,
                 ldx8=64, sx=A, w8=A, ldw8=64, sw=A, need_dx=1, need_dw=1, dx=A, lddx=64, dw=A, lddw=64)
        a.update(kw)
        gs = groups(fp8, **(dict(stride_b=0, scale_b_step=0) | (gr or {})))
        return fp8._lib.fp8_linear_grouped_backward(ctypes.byref(fp8.LinearBwdArgs(**a)), ctypes.byref(gs), None)

    for f in (fwd, bwd):
        assert f(dict(groups=-1)) == bad and f(dict(offsets=None)) == bad
        assert f(dict(stride_b=64)) == bad and f(dict(stride_d=64)) == bad
        assert f(dict(groups=2000)) == E.FP8_ERR_TOO_LARGE
        assert f(M=-1) == bad and f(N=1 << 31) == bad
    assert fp8._lib.fp8_linear_grouped_forward(None, None, None) == bad
    assert fp8._lib.fp8_linear_grouped_backward(None, None, None) == bad
    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(ldy=63), dict(sx_out=None), dict(sw_out=None), dict(fmt_x=2),
               dict(x_dtype=9), dict(w_dtype=9), dict(ring_w=A), dict(ring_x=None), dict(hist_len=0),
               dict(x_dtype=3), dict(w_dtype=3), dict(x_dtype=4, x_scale_in=A)):
        assert fwd(**kw) == bad, kw
    assert fwd(dict(scale_b_step=1)) == bad                 # one ring, one scale
    assert fwd(bias=A) == uns and bwd(need_dbias=1) == uns
    for kw in (dict(g=None), dict(x8=None), dict(w8=None), dict(sx=None), dict(sw=None), dict(dx=None), dict(dw=None),
               dict(lddx=63), dict(lddw=63), dict(sg_out=None), dict(g_dtype=9), dict(g_dtype=4), dict(fmt_g=3),
               dict(ring_g=None)):
        assert bwd(**kw) == bad, kw
    a = dict(M=4, N=32, K=64, x=A, x_dtype=0, ldx=64, w8=A, ldw8=64, sw=A, x8=A, ldx8=64, sx_out=A, y=A, y_dtype=0, ldy=32)

    def lin(**kw):
        return fp8._lib.fp8_linear_int8_forward(ctypes.byref(fp8.LinearInt8Args(**(a | kw))), None)

    assert fp8._lib.fp8_linear_int8_forward(None, None) == bad
    for kw in (dict(x=None), dict(w8=None), dict(sw=None), dict(x8=None), dict(sx_out=None), dict(y=None), dict(x_dtype=3),
               dict(y_dtype=3), dict(ldy=31), dict(ldx=63), dict(ldw8=48), dict(M=-1)):
        assert lin(**kw) == bad, kw
    assert lin(K=131072, ldx=131072, ldx8=131072, ldw8=131072) == E.FP8_ERR_TOO_LARGE


def test_python_helpers_refuse(fp8):
    """Shapes and types are checked before any pointer is taken (CPU tensors: refused as such)."""
    x8, w8 = torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(2, 32, 16, dtype=torch.uint8)
    off, one = torch.tensor([0, 2, 4], dtype=torch.int32), torch.ones(1)
    for args in ((x8, w8, off.float(), one, one), (x8, w8[:1], off, one, one), (x8, w8[:, :, :8], off, one, one),
                 (x8.float(), w8, off, one, one), (x8, w8, off, torch.ones(2), one), (x8, w8, off, one, torch.ones(3)),
                 (x8, w8.transpose(1, 2), off, one, one), (x8, w8[:, ::2], off, one, one),
                 (x8, w8, torch.zeros(6, dtype=torch.int32)[::2], one, one), (x8, w8, off, one, one)):
        with pytest.raises(ValueError):
            fp8.grouped_mm(*args)
    with pytest.raises(ValueError):
        fp8.linear_int8(torch.zeros(2, 16), torch.zeros(8, 16), torch.ones(8))          # w8 not int8
    with pytest.raises(ValueError):
        fp8.linear_int8(torch.zeros(2, 16), torch.zeros(8, 16, dtype=torch.int8), torch.ones(7))
    with pytest.raises(ValueError):
        fp8.linear_int8(torch.zeros(2, 16), torch.zeros(8, 16, dtype=torch.int8), torch.ones(8))  # not on a GPU
