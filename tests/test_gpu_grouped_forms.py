"""Every form of tile of the grouped and int8 products (single CTAs of 16 to 256 columns, clusters that share a
contraction, CTA pairs) against 64-bit products, at shapes that take it on this GPU by the library's own plan.

Tolerances, per element.  FP8: one bf16 rounding (2^-8 of the value) and fp32 accumulation, 2e-6 of the sum of the
products' magnitudes.  Integers: the sum is exact; three roundings to fp32 and a fourth for the bias (2^-24 each),
then one to the output type, half its step."""
import numpy as np
import pytest
import torch

import fp8_delayed_scaling_03_b200 as F
from grouped_forms import GROUPED, INT8, WEIGHT_GRADIENT

pytestmark = pytest.mark.gpu

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
NAN = 0x7F   # a NaN code in both formats


def up(v):
    return (v + 15) // 16 * 16


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def codes(shape, dtype, seed):
    """fp8 codes of normal values, rows padded to 16 with NaN codes."""
    v = torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda") * 3.0
    buf = torch.full((*shape[:-1], up(shape[-1])), NAN, dtype=torch.uint8, device="cuda")
    buf[..., :shape[-1]] = v.to(dtype).view(torch.uint8)
    return buf[..., :shape[-1]]


def value(c, dtype):
    return c.contiguous().view(dtype).double()


def scales(n, seed, low=0.5, high=30.0):
    return torch.rand(n, generator=torch.Generator().manual_seed(seed)).mul(high - low).add(low).cuda()


def assert_close(got, want, mags, what):
    tol = want.abs() * 2.0 ** -8 + mags * 2e-6
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.numel(), bad.nonzero()[:5].tolist())


def ragged(rows, groups, seed):
    """Uneven group sizes, some of them none."""
    share = np.random.RandomState(seed).rand(groups) ** 2
    share[1::7] = 0.0
    return np.random.RandomState(seed + 1).multinomial(rows, share / share.sum())


@pytest.mark.parametrize("major", ["K", "MN"])
@pytest.mark.parametrize("form", list(GROUPED))
def test_grouped(form, major):
    rows, n, k, groups = GROUPED[form]
    edge = 1 if rows > 2 else 0                   # a row of no group before the first, one behind the last
    counts = ragged(rows - 2 * edge, groups, 3)
    mn = major == "MN"
    x8, w8 = codes((rows, k), E4M3, 1), codes((groups, k, n) if mn else (groups, n, k), E4M3, 2)
    x8[:edge], x8[rows - edge:] = NAN, NAN
    sx, sw = scales(1, 3), scales(groups, 4)
    off = torch.tensor(np.concatenate([[edge], edge + np.cumsum(counts)]), dtype=torch.int64, device="cuda")
    y = torch.full((rows, n), 7.0, dtype=torch.bfloat16, device="cuda")
    a = F.MmArgs(rows, n, k, x8.data_ptr(), 0, 0, x8.stride(0), w8.data_ptr(), 0, int(mn), w8.stride(1), sx.data_ptr(),
                 sw.data_ptr(), None, 0, None, y.data_ptr(), n, 0, None, 0)
    p = F.fp8_mm_grouped_plan(a, F.FP8_RAGGED_M, F.Groups(groups, off.data_ptr(), 1, w8.stride(0), 0, 1), sms())
    assert (p.tile_lanes, p.tile_cols, p.split) == form
    F.grouped_mm(x8, w8, off, sx, sw, y=y, w_major=F.FP8_MN_MAJOR if mn else F.FP8_K_MAJOR)
    at = edge
    for e, m in enumerate(counts):
        x, w, s = value(x8[at:at + m], E4M3), value(w8[e], E4M3), float(sx) * float(sw[e])
        w = w if mn else w.t()
        assert_close(y[at:at + m], x @ w / s, x.abs() @ w.abs() / s, (form, e))
        at += m
    assert bool((y[:edge] == 7.0).all()) and bool((y[rows - edge:] == 7.0).all())
    again = F.grouped_mm(x8, w8, off, sx, sw, w_major=F.FP8_MN_MAJOR if mn else F.FP8_K_MAJOR)
    assert torch.equal(again[edge:rows - edge], y[edge:rows - edge])
    assert F.fp8_get_device_status() == 0


@pytest.mark.parametrize("fmt_g", [F.FP8_E5M2, F.FP8_E4M3])
@pytest.mark.parametrize("case", range(len(WEIGHT_GRADIENT)))
def test_weight_gradient(case, fmt_g):
    """Groups that end inside a k-block, with NaN codes before the first and behind the last; the gap behind each row
    of D stays as it was."""
    form, counts, n, k, extra = WEIGHT_GRADIENT[case]
    rows, groups, ld, front = sum(counts), len(counts), k + extra, 3
    g_type = E5M2 if fmt_g == F.FP8_E5M2 else E4M3
    x8, g8 = codes((rows + 8, k), E4M3, 5), codes((rows + 8, n), g_type, 6)
    for t in (x8, g8):
        t[:front], t[front + rows:] = NAN, NAN
    sx, sg = scales(1, 8), scales(1, 9)
    off = torch.tensor(np.concatenate([[front], front + np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    buf = torch.full((groups, n, ld), 3.0, dtype=torch.bfloat16, device="cuda")
    a = F.MmArgs(n, k, rows + 8, g8.data_ptr(), fmt_g, 1, g8.stride(0), x8.data_ptr(), 0, 1, x8.stride(0), sg.data_ptr(),
                 sx.data_ptr(), None, 0, None, buf.data_ptr(), ld, 0, None, 0)
    gr = F.Groups(groups, off.data_ptr(), 0, 0, n * ld, 0)
    p = F.fp8_mm_grouped_plan(a, F.FP8_RAGGED_K, gr, sms())
    assert (p.tile_lanes, p.tile_cols) == form
    for _ in range(2):
        F.fp8_mm_grouped(a, F.FP8_RAGGED_K, gr, buf.device)
    at, s = front, float(sg) * float(sx)
    for e, m in enumerate(counts):
        x, g = value(x8[at:at + m], E4M3), value(g8[at:at + m], g_type)
        assert_close(buf[e, :, :k], g.t() @ x / s, g.abs().t() @ x.abs() / s, (case, e, m))
        at += m
    assert bool((buf[:, :, k:] == 3.0).all())
    assert F.fp8_get_device_status() == 0


def test_one_group_of_nan_rows_stays_out_of_the_others_pairs():
    """On CTA pairs: NaN codes of one group change that group's gradient alone, though k-blocks hold rows of both."""
    form, counts, n, k, _ = WEIGHT_GRADIENT[2]
    rows, off = sum(counts), torch.tensor([0, *np.cumsum(counts)], dtype=torch.int32, device="cuda")
    x8, g8, sx, sg = codes((rows, k), E4M3, 1), codes((rows, n), E5M2, 2), scales(1, 3), scales(1, 4)
    w8 = torch.zeros(len(counts), n, up(k), dtype=torch.uint8, device="cuda")[:, :, :k]

    def dw():
        fwd = F.ForwardResult(None, x8, w8, sx, sx, None, None)
        return F.grouped_linear_backward(g8, fwd, off, None, need_dx=False, g_scale_in=sg).dw

    clean = dw()
    x8[396:1196], g8[396:1196] = NAN, NAN   # group 2: its neighbours' k-blocks run into it
    got = dw()
    assert bool(got[2].isnan().all())
    assert all(torch.equal(got[e], clean[e]) for e in (0, 1, 3, 4))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("form", list(INT8))
def test_int8(form, dtype):
    m, n, k = INT8[form]
    gen = torch.Generator(device="cuda").manual_seed(1)
    a = torch.randint(-128, 128, (m, up(k)), dtype=torch.int8, generator=gen, device="cuda")[:, :k]
    b = torch.randint(-128, 128, (n, up(k)), dtype=torch.int8, generator=gen, device="cuda")[:, :k]
    sa, sb = scales(m, 3, 1e-4, 0.02), scales(n, 4, 1e-4, 0.02)
    bias = torch.randn(n, generator=torch.Generator().manual_seed(5)).cuda()
    # sums below 2^53: exact in 64 bits
    s = (a.double() @ b.double().t()) * sa.double()[:, None] * sb.double()
    eps = torch.finfo(dtype).eps / 2
    for extra, with_bias in ((0, True), (3, False), (8, True)):   # row pitches of each store path
        buf = torch.full((m, n + extra), 5.0, dtype=dtype, device="cuda")
        args = F.MmInt8Args(m, n, k, a.data_ptr(), a.stride(0), b.data_ptr(), b.stride(0), sa.data_ptr(), sb.data_ptr(),
                            bias.data_ptr() if with_bias else None, F.FP8_DT_FP32, buf.data_ptr(), F._dtype_code(buf),
                            n + extra)
        p = F.fp8_mm_int8_plan(args, sms())
        if extra == 0:
            assert (p.tile_lanes, p.tile_cols, p.split) == form
        F.fp8_mm_int8(args, buf.device)
        want = s + bias.double() if with_bias else s
        tol = want.abs() * eps * (1 + 1e-6) + s.abs() * 3.01 * 2.0 ** -24 + want.abs() * 2.0 ** -24 + \
            torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
        bad = ~((buf[:, :n].double() - want).abs() <= tol)
        assert not bad.any(), (form, dtype, extra, int(bad.sum()), bad.nonzero()[:5].tolist())
        assert bool((buf[:, n:] == 5.0).all())
    assert F.fp8_get_device_status() == 0
