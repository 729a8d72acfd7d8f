"""The tiles of the grouped and int8 products (fp8_mm_grouped_plan, fp8_mm_int8_plan: host arithmetic only).  Every form
of tile there is has a shape of its own in grouped_forms.py; the GPU tests run those shapes, so that a change of the
rule shows here when it takes one of the forms out of their reach."""
import ctypes

import pytest

from grouped_forms import GROUPED, INT8, WEIGHT_GRADIENT

A = 0x100000  # a fake 16-byte aligned device address; nothing is dereferenced


@pytest.fixture(scope="module")
def fp8():
    import fp8_delayed_scaling_03_b200 as m
    return m


def up(v):
    return (v + 15) // 16 * 16


def int8_args(F, m, n, k, dtype=0, ldd=None, **kw):
    a = dict(m=m, n=n, k=k, a=A, lda=up(k), b=A, ldb=up(k), scale_a=A, scale_b=A, bias=None, bias_dtype=0, d=A,
             d_dtype=dtype, ldd=n if ldd is None else ldd)
    return F.MmInt8Args(**a | kw)


def grouped_args(F, rows, n, k, groups, mn=False, **kw):
    ldb = up(n) if mn else up(k)
    a = dict(m=rows, n=n, k=k, a=A, fmt_a=0, a_major=0, lda=up(k), b=A, fmt_b=0, b_major=int(mn), ldb=ldb, scale_a=A,
             scale_b=A, d=A, ldd=n)
    return F.MmArgs(**a | kw), F.FP8_RAGGED_M, F.Groups(groups, A, 0, (k if mn else n) * ldb, 0, 0)


def dw_args(F, rows, n, k, groups, extra=0):
    a = F.MmArgs(m=n, n=k, k=rows, a=A, fmt_a=1, a_major=1, lda=up(n), b=A, fmt_b=0, b_major=1, ldb=up(k), scale_a=A,
                 scale_b=A, d=A, ldd=k + extra)
    return a, F.FP8_RAGGED_K, F.Groups(groups, A, 0, 0, n * (k + extra), 0)


@pytest.mark.parametrize("form", list(INT8))
def test_int8_forms(fp8, form):
    for dtype in (0, 1, 2):
        p = fp8.fp8_mm_int8_plan(int8_args(fp8, *INT8[form], dtype))
        assert (p.tile_lanes, p.tile_cols, p.split) == form
        m, n, _ = INT8[form]
        assert p.max_tiles >= -(-m // p.tile_cols) * -(-n // p.tile_lanes)


@pytest.mark.parametrize("form", list(GROUPED))
def test_grouped_forms(fp8, form):
    for mn in (False, True):
        p = fp8.fp8_mm_grouped_plan(*grouped_args(fp8, *GROUPED[form], mn))
        assert (p.tile_lanes, p.tile_cols, p.split) == form


@pytest.mark.parametrize("case", WEIGHT_GRADIENT)
def test_weight_gradient_forms(fp8, case):
    form, counts, n, k, extra = case
    p = fp8.fp8_mm_grouped_plan(*dw_args(fp8, sum(counts), n, k, len(counts), extra))
    assert (p.tile_lanes, p.tile_cols) == form and p.split == 1
    assert p.max_tiles == len(counts) * -(-n // form[1]) * -(-k // form[0])


def test_every_form_of_a_random_walk_is_covered(fp8):
    """Forms that shapes drawn over the whole range take: each has its test shape."""
    import math
    import random
    rng = random.Random(7)

    def draw(low, high):
        return int(math.exp(rng.uniform(math.log(low), math.log(high + 1))))

    for _ in range(20000):
        m, n, k, e = draw(1, 9000), draw(1, 12000), draw(1, 12000), draw(1, 64)
        p = fp8.fp8_mm_int8_plan(int8_args(fp8, m, n, k))
        assert (p.tile_lanes, p.tile_cols, p.split) in INT8, (m, n, k)
        p = fp8.fp8_mm_grouped_plan(*grouped_args(fp8, m, n, k, e))
        assert (p.tile_lanes, p.tile_cols, p.split) in GROUPED, (m, n, k, e)
        p = fp8.fp8_mm_grouped_plan(*dw_args(fp8, m, n, k, e))
        assert (p.tile_lanes, p.tile_cols) in {c[0] for c in WEIGHT_GRADIENT} and p.split == 1, (m, n, k, e)


def test_validation(fp8):
    E, lib = fp8, fp8._lib
    info = fp8.GroupedPlanInfo()
    good = int8_args(fp8, 16, 32, 64)
    assert lib.fp8_mm_int8_plan(None, 148, ctypes.byref(info)) == E.FP8_ERR_INVALID_ARG
    assert lib.fp8_mm_int8_plan(ctypes.byref(good), 0, ctypes.byref(info)) == E.FP8_ERR_INVALID_ARG
    assert lib.fp8_mm_int8_plan(ctypes.byref(good), 148, None) == E.FP8_ERR_INVALID_ARG
    for kw, status in ((dict(lda=72), E.FP8_ERR_MISALIGNED), (dict(ldd=31), E.FP8_ERR_INVALID_ARG),
                       (dict(k=131072, lda=131072, ldb=131072), E.FP8_ERR_TOO_LARGE)):
        a = int8_args(fp8, 16, 32, 64)
        for name, v in kw.items():
            setattr(a, name, v)
        assert lib.fp8_mm_int8_plan(ctypes.byref(a), 148, ctypes.byref(info)) == status
    a, ragged, g = grouped_args(fp8, 16, 32, 64, 2)

    def plan(a=a, ragged=ragged, g=g, sms=148, out=info):
        return lib.fp8_mm_grouped_plan(None if a is None else ctypes.byref(a), ragged, None if g is None else ctypes.byref(g),
                                       sms, None if out is None else ctypes.byref(out))

    assert plan() == E.FP8_OK
    assert plan(a=None) == plan(g=None) == plan(sms=0) == plan(out=None) == plan(ragged=2) == E.FP8_ERR_INVALID_ARG
    assert plan(g=fp8.Groups(2000, A, 0, 0, 0, 0)) == E.FP8_ERR_TOO_LARGE
    forced = grouped_args(fp8, 16, 32, 64, 2, tile_cfg=1)[0]
    assert plan(a=forced) == E.FP8_ERR_UNSUPPORTED
    for args in (grouped_args(fp8, 0, 32, 64, 2), grouped_args(fp8, 16, 0, 64, 2), grouped_args(fp8, 16, 32, 64, 0)):
        p = fp8.fp8_mm_grouped_plan(*args)
        assert (p.tile_lanes, p.tile_cols, p.split, p.max_tiles) == (0, 0, 0, 0)
    p = fp8.fp8_mm_int8_plan(int8_args(fp8, 0, 32, 64))
    assert (p.tile_lanes, p.tile_cols, p.split, p.max_tiles) == (0, 0, 0, 0)
