"""The row quantize to 8-bit integers, the integer product with a scale per
token and per channel, and the linear of the two, against exact integers and
64-bit arithmetic.

Tolerance of a product, per element: the integer sum is exact; its conversion
and the two scalings round to fp32 three times and the bias adds a fourth
(each half a step, 2^-24 of the value it rounds), then one rounding to the
output type, half its step."""
import numpy as np
import pytest
import torch

import fp8_delayed_scaling_03_b200 as F

pytestmark = pytest.mark.gpu

WIDE = [torch.bfloat16, torch.float16, torch.float32]


def int8_codes(rows, cols, seed, ld=None, junk=99):
    gen = torch.Generator().manual_seed(seed)
    ld = (cols + 15) // 16 * 16 if ld is None else ld
    buf = torch.full((rows, ld), junk, dtype=torch.int8)
    buf[:, :cols] = torch.randint(-128, 128, (rows, cols), generator=gen).to(torch.int8)
    return buf.cuda()[:, :cols]


def scales(n, seed):
    return (torch.rand(n, generator=torch.Generator().manual_seed(seed)) * 0.02 + 1e-4).cuda()


def product(a, b, sa, sb, bias, d, k=None):
    args = F.MmInt8Args(a.shape[0], b.shape[0], a.shape[1] if k is None else k, a.data_ptr(), a.stride(0),
                        b.data_ptr(), b.stride(0), sa.data_ptr(), sb.data_ptr(),
                        bias.data_ptr() if bias is not None else None, F._dtype_code(bias) if bias is not None else 0,
                        d.data_ptr(), F._dtype_code(d), d.stride(0))
    F.fp8_mm_int8(args, d.device)
    return d


def exact_sum(a, b):
    return a.double() @ b.double().t()   # whole numbers below 2^53: exact


def assert_close(got, want, scaled, dtype, what=""):
    """scaled: |sum * sa * sb|, what the three fp32 roundings are relative to."""
    tol = want.abs() * (torch.finfo(dtype).eps / 2) * (1 + 1e-6) + scaled.abs() * 3.01 * 2.0 ** -24 + want.abs() * 2.0 ** -24
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    bad = ~((got.double() - want).abs() <= tol + tiny)
    assert not bad.any(), (what, int(bad.sum()), bad.numel(), bad.nonzero()[:5].tolist())


@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 33, 64, 100, 129, 256, 300])
@pytest.mark.parametrize("n,k", [(128, 128), (77, 64), (1000, 40), (16, 1), (129, 513), (640, 2048), (4096, 1500)])
def test_product(m, n, k):
    a, b, sa, sb = int8_codes(m, k, 1), int8_codes(n, k, 2), scales(m, 3), scales(n, 4)
    s = exact_sum(a, b) * sa.double()[:, None] * sb.double()
    for i, dtype in enumerate(WIDE):
        bias = torch.randn(n, generator=torch.Generator().manual_seed(5)).to(WIDE[(i + m) % 3]).cuda() if (m + i) % 2 else None
        y = product(a, b, sa, sb, bias, torch.empty(m, n, dtype=dtype, device="cuda"))
        assert_close(y, s if bias is None else s + bias.double(), s, dtype, (m, n, k, dtype))
    assert F.fp8_get_device_status() == 0


def test_large_product():
    """Sizes that fill the GPU: tiles on pairs of SMs, the last of them partial in every direction."""
    m, n, k = 1061, 5013, 400
    a, b, sa, sb = int8_codes(m, k, 1), int8_codes(n, k, 2), scales(m, 3), scales(n, 4)
    s = exact_sum(a, b) * sa.double()[:, None] * sb.double()
    for dtype in WIDE:
        y = product(a, b, sa, sb, None, torch.empty(m, n, dtype=dtype, device="cuda"))
        assert_close(y, s, s, dtype, dtype)
    one_a, one_b = torch.ones(m, device="cuda"), torch.ones(n, device="cuda")
    assert torch.equal(product(a, b, one_a, one_b, None, torch.empty(m, n, device="cuda")).double(), exact_sum(a, b))


def test_sums_are_exact_integers():
    """Scales of one, fp32 output: whole sums below 2^24 come out exactly, the extreme codes among them."""
    for m, n, k in ((3, 50, 900), (40, 130, 1000)):
        a, b = int8_codes(m, k, 1), int8_codes(n, k, 2)
        a[0], b[0], b[1] = -128, -128, 127
        one_a, one_b = torch.ones(m, device="cuda"), torch.ones(n, device="cuda")
        y = product(a, b, one_a, one_b, None, torch.empty(m, n, device="cuda"))
        assert torch.equal(y.double(), exact_sum(a, b))
    # the longest contraction, every product the largest: 2^31 - 2^14 in int32
    k = F.FP8_MAX_INT8_K
    a = torch.full((2, k + 1), -128, dtype=torch.int8, device="cuda")[:, :k]
    b = torch.full((20, k + 1), -128, dtype=torch.int8, device="cuda")[:, :k]
    y = product(a, b, torch.ones(2, device="cuda"), torch.ones(20, device="cuda"), None, torch.empty(2, 20, device="cuda"))
    assert bool((y == float(np.float32(k * 16384))).all())


def reference_codes(x):
    """(codes, scale) from the definition: 64-bit quotients of fp32 values, whose rounding crosses no border."""
    v = x.double().cpu()
    amax = v.abs().amax(1)
    bad = ~torch.isfinite(v).all(1)
    top = torch.where((amax > 0) & ~bad, amax, torch.ones_like(amax))
    q = torch.round(torch.where(bad[:, None], torch.zeros_like(v), v) * 127.0 / top[:, None])
    s = torch.where(amax > 0, amax.float() / torch.tensor(127.0), torch.ones(len(v)))
    return q.to(torch.int8), torch.where(bad, torch.full_like(s, float("nan")), s)


def check_quantize(x, ld_out=None):
    rows, cols = x.shape
    ld = (cols + 15) // 16 * 16 if ld_out is None else ld_out
    buf = torch.full((rows, ld), 55, dtype=torch.int8, device="cuda")
    scale = torch.full((rows + 1,), -3.0, device="cuda")
    F.quantize_int8(x, buf[:, :cols], scale[:rows])
    q, s = reference_codes(x)
    assert torch.equal(buf[:, :cols].cpu(), q)
    assert torch.equal(scale[:rows].cpu().view(torch.int32)[~s.isnan()], s.view(torch.int32)[~s.isnan()])
    assert torch.equal(scale[:rows].cpu().isnan(), s.isnan()) and float(scale[rows]) == -3.0
    end = (cols + 15) // 16 * 16
    assert bool((buf[:, cols:end] == 0).all()) and bool((buf[:, end:] == 55).all())


@pytest.mark.parametrize("dtype", WIDE)
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 15), (9, 16), (17, 300), (8, 1024), (5, 1025), (3, 4096), (2, 11008),
                                       (2, 16384), (2, 16385), (1, 40000)])
def test_quantize(dtype, rows, cols):
    gen = torch.Generator().manual_seed(rows * cols)
    x = (torch.randn(rows, cols, generator=gen) * torch.exp(torch.randn(rows, 1, generator=gen) * 3)).to(dtype)
    check_quantize(x.cuda())
    # rows that 16-byte loads cannot address, and a wider output pitch
    buf = torch.full((rows, cols + 3), 3e4, dtype=dtype)
    buf[:, :cols] = x
    check_quantize(buf.cuda()[:, :cols], (cols + 15) // 16 * 16 + 32)


@pytest.mark.parametrize("dtype", WIDE)
def test_quantize_borders_and_special_rows(dtype):
    """Values exactly on the border of two codes go to the even one, their fp32 neighbours to either side; rows of
    zeros, of the smallest and largest values, with NaN and infinities."""
    half = torch.arange(-126.5, 127.0, 1.0, dtype=torch.float64)
    rows = []
    for top in (127.0, 254.0, 127.0 * 2.0 ** -20, 127.0 * 2.0 ** 8):   # the border k + 0.5 is exact in every type
        v = (half * (top / 127.0)).to(dtype)
        rows.append(torch.cat([v, torch.tensor([top], dtype=dtype)]))
    if dtype == torch.float32:
        for top in (127.0, 1.1, 3e38, 2e-38):
            v = (half * (top / 127.0)).float()
            for to in (np.inf, -np.inf):
                w = torch.from_numpy(np.nextafter(v.numpy(), np.float32(to)))
                rows.append(torch.cat([w, torch.tensor([top])]))
    f = torch.finfo(dtype)
    least = f.smallest_normal * f.eps
    n = len(half) + 1
    zero = torch.zeros(n, dtype=dtype)
    rows += [zero, -zero]
    for fill in ([least], [-least, 3 * least, 100 * least], [f.max, -f.max, f.max / 3], [float("nan")], [1.0, float("inf")],
                 [float("-inf"), 2.0], [f.smallest_normal, f.smallest_normal / 2]):
        r = zero.clone()
        r[5:5 + len(fill)] = torch.tensor(fill, dtype=dtype)
        rows.append(r)
    check_quantize(torch.stack(rows).cuda())


@pytest.mark.parametrize("dtype", WIDE)
@pytest.mark.parametrize("M,N,K", [(1, 256, 512), (5, 77, 100), (64, 1000, 784), (257, 144, 96)])
def test_linear(dtype, M, N, K):
    """The serving path: weights quantized once by channel, inputs within the call."""
    gen = torch.Generator().manual_seed(M)
    x = torch.randn(M, K, generator=gen).to(dtype).cuda()
    w = (torch.randn(N, K, generator=gen) / K ** 0.5).cuda()
    bias = torch.randn(N, generator=gen).bfloat16().cuda()
    w8, sw = F.quantize_int8(w)
    r = F.linear_int8(x, w8, sw, bias=bias)
    q, s = reference_codes(x)
    assert torch.equal(r.x8.cpu(), q) and torch.equal(r.sx.cpu(), s) and r.y.dtype == dtype
    y = exact_sum(r.x8, w8) * s.cuda().double()[:, None] * sw.double()
    assert_close(r.y, y + bias.double(), y, dtype)
    # against the linear of the unquantized operands: each factor is off by at most half a step
    step = (s.cuda().double()[:, None] / 2) * w.double().abs().sum(1) + x.double().abs().sum(1)[:, None] * (sw.double() / 2) + \
        K * s.cuda().double()[:, None] * sw.double() / 4
    want = x.double() @ w.double().t() + bias.double()
    assert bool(((r.y.double() - want).abs() <= step + want.abs() * torch.finfo(dtype).eps + 1e-5).all())
    x8, sx = torch.empty(M, (K + 15) // 16 * 16, dtype=torch.int8, device="cuda")[:, :K], torch.empty(M, device="cuda")
    for given in (dict(x8=x8), dict(sx=sx), dict(x8=x8, sx=sx)):   # the caller's buffers
        o = F.linear_int8(x, w8, sw, bias=bias, **given)
        assert torch.equal(o.y, r.y) and torch.equal(o.x8, r.x8) and torch.equal(o.sx, r.sx)
        assert ("x8" not in given or o.x8 is x8) and ("sx" not in given or o.sx is sx)
    other = F.linear_int8(x, w8, sw, out_dtype=torch.float32)
    assert other.y.dtype == torch.float32
    assert_close(other.y, y, y, torch.float32)


def test_trained_experts_served_in_integers():
    """The two operators together: an expert layer's forward and backward, a step on its weights by that gradient, then
    the same experts served in 8-bit integers, group by group, against 64-bit products of the updated weights."""
    c, N, K = [30, 0, 75, 7], 192, 128
    rows, E = sum(c), len(c)
    off = torch.tensor([0, *np.cumsum(c)], dtype=torch.int32, device="cuda")
    gen = torch.Generator().manual_seed(8)
    x = torch.randn(rows, K, generator=gen).bfloat16().cuda()
    w = (torch.randn(E, N, K, generator=gen) / 12).bfloat16().cuda()
    rings = [F.ScaleRing(4) for _ in range(3)]
    for _ in range(2):
        f = F.grouped_linear_forward(x, w, off, rings[0], rings[1])
        b = F.grouped_linear_backward(f.y, f, off, rings[2])     # the gradient of sum(y^2) / 2
        w = (w.float() - 0.01 * b.dw.float()).bfloat16()
    at = 0
    for e, m in enumerate(c):
        w8, sw = F.quantize_int8(w[e])
        r = F.linear_int8(x[at:at + m], w8, sw)
        xe, we = x[at:at + m].double(), w[e].double()
        want = xe @ we.t()
        # each factor is off by at most half a step of its scale, then one rounding to bf16
        s = r.sx.double()[:, None]
        off_by = s / 2 * we.abs().sum(1) + xe.abs().sum(1)[:, None] * sw.double() / 2 + K * s * sw.double() / 4
        assert bool(((r.y.double() - want).abs() <= off_by + (want.abs() + off_by) * 2.0 ** -8 + 1e-6).all()), e
        at += m
    assert F.fp8_get_device_status() == 0


def test_bad_rows_give_nan_rows_only():
    x = torch.randn(20, 64, generator=torch.Generator().manual_seed(1)).cuda()
    w8, sw = F.quantize_int8(torch.randn(48, 64, generator=torch.Generator().manual_seed(2)).cuda())
    clean = F.linear_int8(x, w8, sw).y
    x[3, 5], x[7, 0], x[11] = float("nan"), float("inf"), 0.0
    y = F.linear_int8(x, w8, sw).y
    live = torch.ones(20, dtype=torch.bool, device="cuda")
    live[[3, 7, 11]] = False
    assert torch.equal(y[live], clean[live])
    assert bool(y[3].isnan().all()) and bool(y[7].isnan().all()) and bool((y[11] == 0).all())


def test_empty_sizes():
    """No rows, no channels, or an empty contraction, where the bias alone is the result."""
    w8, sw = F.quantize_int8(torch.randn(48, 64).cuda())
    r = F.linear_int8(torch.empty(0, 64, device="cuda"), w8, sw)
    assert r.y.shape == (0, 48) and r.x8.shape == (0, 64) and r.sx.shape == (0,)
    assert F.linear_int8(torch.empty(5, 0, device="cuda"), w8[:, :0], sw).x8.shape == (5, 0)
    assert F.linear_int8(torch.ones(3, 64, device="cuda"), w8[:0], sw[:0]).y.shape == (3, 0)
    bias = torch.randn(48).bfloat16().cuda()
    none = torch.empty(48, 0, dtype=torch.int8, device="cuda")
    nans = torch.full((5,), float("nan"), device="cuda")
    r = F.linear_int8(torch.empty(5, 0, device="cuda"), none, sw, bias=bias, sx=nans)
    assert torch.equal(r.y, bias.float().expand(5, 48)) and bool(nans.isnan().all())
    assert bool((F.linear_int8(torch.empty(5, 0, device="cuda"), none, sw, sx=nans).y == 0).all())


def test_strided_outputs_capture_and_streams():
    """Outputs with a pitch; two captured linears that share the input, replayed with new inputs; a side stream."""
    gen = torch.Generator().manual_seed(1)
    M, N, K = 37, 200, 256
    x = torch.randn(M, K, generator=gen).bfloat16().cuda()
    ws = [F.quantize_int8(torch.randn(N, K, generator=gen).cuda()) for _ in range(2)]
    want = [F.linear_int8(x, *w).y for w in ws]
    for ld in (208, 203, 200):
        buf = torch.full((M, ld), 5.0, dtype=torch.bfloat16, device="cuda")
        F.linear_int8(x, *ws[0], y=buf[:, :N])
        assert torch.equal(buf[:, :N], want[0]) and bool((buf[:, N:] == 5.0).all())
    outs = [torch.empty_like(want[0]) for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for w, o in zip(ws, outs):
            F.linear_int8(x, *w, y=o)
    for scale in (1.0, 3.0, 0.25):
        x.mul_(scale)
        graph.replay()
        want = [F.linear_int8(x, *w).y for w in ws]
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = F.linear_int8(x, *ws[1]).y
    side.synchronize()
    assert torch.equal(y, want[1])
    assert F.fp8_get_device_status() == 0
