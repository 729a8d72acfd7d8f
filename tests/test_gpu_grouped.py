"""FP8 products grouped by expert with ragged sizes against 64-bit products of
the decoded operands, group by group.

Tolerance, per element: one bf16 rounding, half a step of the value (2^-8 of
it), plus what fp32 accumulation may lose, 2e-6 of the sum of the products'
magnitudes -- the bound the library's GEMM tests use."""
import numpy as np
import pytest
import torch

import fp8_delayed_scaling_03_b200 as F

pytestmark = pytest.mark.gpu

TYPES = {F.FP8_E4M3: torch.float8_e4m3fn, F.FP8_E5M2: torch.float8_e5m2}


def codes(rows, cols, fmt, seed, ld=None, junk=0x7F, batch=None):
    """[rows, cols] (or [batch, rows, cols]) fp8 codes of normal values; the padding of a row holds NaN codes."""
    gen = torch.Generator().manual_seed(seed)
    shape = (rows, cols) if batch is None else (batch, rows, cols)
    v = torch.randn(shape, generator=gen) * 3.0
    ld = (cols + 15) // 16 * 16 if ld is None else ld
    buf = torch.full((*shape[:-1], ld), junk, dtype=torch.uint8)
    buf[..., :cols] = v.to(TYPES[fmt]).view(torch.uint8)
    return buf.cuda()[..., :cols]


def value(c, fmt):
    return c.contiguous().view(TYPES[fmt]).double()


def offsets_of(counts, first=0, dtype=torch.int32):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(counts)]), dtype=dtype, device="cuda")


def scales(n, seed):
    return (torch.rand(n, generator=torch.Generator().manual_seed(seed)) * 30 + 0.5).cuda()


def assert_close(got, want, mags, what):
    tol = want.abs() * 2.0 ** -8 + mags * 2e-6
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.numel(), float((err / tol.clamp_min(1e-300)).max()),
                           bad.nonzero()[:5].tolist())


COUNTS = {
    "one_row": [1],
    "decode": [1, 0, 2, 0, 0, 1, 0, 3],
    "all_empty": [0, 0, 0],
    "ragged": [37, 0, 128, 129, 1, 255, 16, 300],
    "one_takes_all": [0, 0, 515, 0],
    "many": [(7 * i) % 23 for i in range(100)],
    "whole_tiles": [256, 256, 512],
}


@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("n,k", [(128, 128), (272, 200), (77, 64), (1000, 40), (16, 1), (129, 513)])
@pytest.mark.parametrize("fmt_x,fmt_w,major", [(0, 0, "K"), (1, 0, "MN"), (0, 1, "K")])
def test_forward_and_dx(counts, n, k, fmt_x, fmt_w, major):
    c = COUNTS[counts]
    front, behind = (3, 5) if counts in ("ragged", "decode") else (0, 0)
    rows, groups = front + sum(c) + behind, len(c)
    x8 = codes(rows, k, fmt_x, 1)
    w8 = codes(n, k, fmt_w, 2, batch=groups) if major == "K" else codes(k, n, fmt_w, 2, batch=groups)
    off = offsets_of(c, front, torch.int64 if counts == "many" else torch.int32)
    sx, sw = scales(1, 3), scales(groups if counts != "whole_tiles" else 1, 4)
    y = torch.full((max(rows, 1), n), 7.0, dtype=torch.bfloat16, device="cuda")[:rows]
    out = F.grouped_mm(x8, w8, off, sx, sw, y=y, fmt_x=fmt_x, fmt_w=fmt_w,
                       w_major=F.FP8_K_MAJOR if major == "K" else F.FP8_MN_MAJOR)
    assert out is y and F.fp8_get_device_status() == 0
    at = front
    for e, m in enumerate(c):
        x, w = value(x8[at:at + m], fmt_x), value(w8[e], fmt_w)
        w = w if major == "K" else w.t()
        s = float(sx) * float(sw[e % sw.numel()])
        assert_close(y[at:at + m], x @ w.t() / s, x.abs() @ w.abs().t() / s, (counts, e))
        at += m
    assert bool((y[:front] == 7.0).all()) and bool((y[at:] == 7.0).all())  # rows of no group


@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("n,k", [(128, 128), (272, 200), (77, 64), (1000, 40), (16, 1), (129, 513)])
@pytest.mark.parametrize("fmt_g", [1, 0])
def test_weight_gradient(counts, n, k, fmt_g):
    c = COUNTS[counts]
    front, behind = (3, 5) if counts in ("ragged", "decode") else (0, 0)
    rows, groups = front + sum(c) + behind, len(c)
    x8, g8 = codes(rows, k, 0, 5), codes(rows, n, fmt_g, 6)
    if front:  # NaN codes in rows of no group stay out of every gradient
        x8[:front], x8[rows - behind:], g8[:front] = 0x7F, 0x7F, 0x7F
    off = offsets_of(c, front)
    fwd = F.ForwardResult(None, x8, codes(n, k, 0, 7, batch=groups), scales(1, 8), scales(1, 9), None, None)
    sg = scales(1, 10)
    b = F.grouped_linear_backward(g8, fwd, off, None, fmt_g=fmt_g, need_dx=False, g_scale_in=sg)
    assert b.dx is None and F.fp8_get_device_status() == 0
    assert b.sg is sg and b.amax_g is None   # a pre-quantized g's scale is the caller's
    at = front
    for e, m in enumerate(c):
        x, g = value(x8[at:at + m], 0), value(g8[at:at + m], fmt_g)
        s = float(sg) * float(fwd.sx)
        assert_close(b.dw[e], g.t() @ x / s, g.abs().t() @ x.abs() / s, (counts, e))
        at += m


@pytest.mark.parametrize("c,n,k", [([300, 0, 129, 515, 256], 4112, 144), ([257] * 9, 2049, 100), ([1000, 40, 160], 5000, 520),
                                   ([700, 333, 1, 0, 130], 4096, 1)])
def test_large_products(c, n, k):
    """Groups and widths that fill the GPU: tiles on pairs of SMs, forward, dX and dW."""
    rows, groups = sum(c), len(c)
    off = offsets_of(c)
    x8, w8, g8 = codes(rows, k, 0, 1), codes(n, k, 0, 2, batch=groups), codes(rows, n, 1, 3)
    sx, sw, sg = scales(1, 4), scales(groups, 5), scales(1, 6)
    y = F.grouped_mm(x8, w8, off, sx, sw)
    b = F.grouped_linear_backward(g8, F.ForwardResult(None, x8, w8, sx, sw, None, None), off, None, g_scale_in=sg)
    # dX with the operands' roles exchanged, so that its width is the large one too
    t8 = w8.transpose(1, 2).contiguous()
    tp = torch.zeros(groups, k, (n + 15) // 16 * 16, dtype=torch.uint8, device="cuda")
    tp[:, :, :n] = t8
    wide = F.grouped_mm(x8, tp[:, :, :n], off, sx, sw, w_major=F.FP8_MN_MAJOR)
    at = 0
    for e, m in enumerate(c):
        x, w, g = value(x8[at:at + m], 0), value(w8[e], 0), value(g8[at:at + m], 1)
        s, sd, sdw = float(sx) * float(sw[e]), float(sg) * float(sw[e]), float(sg) * float(sx)
        assert_close(y[at:at + m], x @ w.t() / s, x.abs() @ w.abs().t() / s, ("y", e))
        assert torch.equal(wide[at:at + m], y[at:at + m])
        assert_close(b.dx[at:at + m], g @ w / sd, g.abs() @ w.abs() / sd, ("dx", e))
        assert_close(b.dw[e], g.t() @ x / sdw, g.abs().t() @ x.abs() / sdw, ("dw", e))
        at += m
    assert F.fp8_get_device_status() == 0


@pytest.mark.parametrize("n,k", [(300, 100), (1300, 84), (2049, 128), (260, 1000), (128, 1100)])
def test_weight_gradient_of_many_groups(n, k):
    """More tiles than SMs, most of few columns or rows: 256 columns on one CTA, the last tiles narrower than one chunk
    of 128; groups without rows have a zero gradient; NaN codes of the neighbours stay out."""
    c = [0, 90, 1, 33, 128, 0, 97, 257, 160, 5] * 5
    rows = sum(c) + 4
    x8, g8, off = codes(rows, k, 0, 5), codes(rows, n, 1, 6), offsets_of(c, 2)
    x8[:2], x8[rows - 2:], g8[:2], g8[rows - 2:] = 0x7F, 0x7F, 0x7F, 0x7F
    fwd = F.ForwardResult(None, x8, codes(n, k, 0, 7, batch=len(c)), scales(1, 8), scales(1, 9), None, None)
    sg = scales(1, 10)
    b = F.grouped_linear_backward(g8, fwd, off, None, need_dx=False, g_scale_in=sg)
    at = 2
    for e, m in enumerate(c):
        x, g = value(x8[at:at + m], 0), value(g8[at:at + m], 1)
        s = float(sg) * float(fwd.sx)
        assert_close(b.dw[e], g.t() @ x / s, g.abs().t() @ x.abs() / s, (e, m))
        at += m
    assert F.fp8_get_device_status() == 0


@pytest.mark.parametrize("c", [[1], [1, 0, 2, 0, 0, 1, 0, 3], [40, 0, 20], [64], [33], [0, 0, 5]])
@pytest.mark.parametrize("n,k", [(130, 1024), (400, 1100), (24, 8192), (1000, 2050)])
@pytest.mark.parametrize("major", ["K", "MN"])
def test_few_tiles_and_long_contractions(c, n, k, major):
    """Launches of a few tiles, whose k-blocks several CTAs share: the same result every time."""
    rows, groups = sum(c), len(c)
    x8 = codes(rows, k, 0, 1)
    w8 = codes(n, k, 0, 2, batch=groups) if major == "K" else codes(k, n, 0, 2, batch=groups)
    off, sx, sw = offsets_of(c), scales(1, 3), scales(groups, 4)
    y = F.grouped_mm(x8, w8, off, sx, sw, w_major=F.FP8_K_MAJOR if major == "K" else F.FP8_MN_MAJOR)
    at = 0
    for e, m in enumerate(c):
        x, w = value(x8[at:at + m], 0), value(w8[e], 0)
        w = w if major == "K" else w.t()
        s = float(sx) * float(sw[e])
        assert_close(y[at:at + m], x @ w.t() / s, x.abs() @ w.abs().t() / s, (c, e))
        at += m
    for _ in range(3):
        again = F.grouped_mm(x8, w8, off, sx, sw, w_major=F.FP8_K_MAJOR if major == "K" else F.FP8_MN_MAJOR)
        assert torch.equal(again, y)
    assert F.fp8_get_device_status() == 0


@pytest.mark.parametrize("small", [True, False])
def test_neighbours_nans_stay_out(small):
    """NaN codes in one group change that group's results alone, though its rows share tiles and k-blocks with others'."""
    c = [5, 33, 70, 129]
    rows, n, k = sum(c), 144 if small else 5120, 96
    off = offsets_of(c)
    x8, g8, w8 = codes(rows, k, 0, 1), codes(rows, n, 1, 2), codes(n, k, 0, 3, batch=len(c))
    sx, sw, sg = scales(1, 4), scales(1, 5), scales(1, 6)

    def both():
        y = F.grouped_mm(x8, w8, off, sx, sw)
        b = F.grouped_linear_backward(g8, F.ForwardResult(None, x8, w8, sx, sw, None, None), off, None, g_scale_in=sg)
        return y.clone(), b.dx.clone(), b.dw.clone()

    clean = both()
    x8[38:108], g8[38:108] = 0x7F, 0x7F  # group 2
    y, dx, dw = both()
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[38:108] = False
    assert torch.equal(y[keep], clean[0][keep]) and torch.equal(dx[keep], clean[1][keep])
    assert bool(y[~keep].isnan().all()) and bool(dx[~keep].isnan().all()) and bool(dw[2].isnan().all())
    for e in (0, 1, 3):
        assert torch.equal(dw[e], clean[2][e])


def test_one_group_equals_fp8_mm():
    """The same products as fp8_mm's, forward, dX and dW."""
    M, N, K = 300, 400, 528
    x8, w8, g8 = codes(M, K, 0, 1), codes(N, K, 0, 2, batch=1), codes(M, N, 1, 3)
    sx, sw, sg = scales(1, 4), scales(1, 5), scales(1, 6)
    off = offsets_of([M])
    y = F.grouped_mm(x8, w8, off, sx, sw)
    b = F.grouped_linear_backward(g8, F.ForwardResult(None, x8, w8, sx, sw, None, None), off, None, g_scale_in=sg)
    want = [torch.empty_like(t) for t in (y, b.dx, b.dw[0])]
    K_, MN = F.FP8_K_MAJOR, F.FP8_MN_MAJOR
    F.fp8_mm(M, N, K, x8, 0, K_, x8.stride(0), w8, 0, K_, w8.stride(1), sx, sw, want[0], N, tile_cfg=1)
    F.fp8_mm(M, K, N, g8, 1, K_, g8.stride(0), w8, 0, MN, w8.stride(1), sg, sw, want[1], K, tile_cfg=1)
    F.fp8_mm(N, K, M, g8, 1, MN, g8.stride(0), x8, 0, MN, x8.stride(0), sg, sx, want[2], K, tile_cfg=1)
    for got, ref in zip((y, b.dx, b.dw[0]), want):
        # both round one fp32 sum to bf16; the sums' orders may differ, so the results by a step
        assert bool(((got.double() - ref.double()).abs() <= ref.double().abs() * 2.0 ** -7 + 1e-6).all())


def test_strided_and_unaligned_outputs():
    """Row pitches above the width, and rows that 16-byte stores cannot address: bytes past n stay."""
    c, n, k = [70, 3, 140], 152, 96
    rows = sum(c)
    off = offsets_of(c)
    x8, w8 = codes(rows, k, 0, 1, ld=144), codes(n, k, 0, 2, ld=112, batch=3)
    sx, sw = scales(1, 3), scales(3, 4)
    want = F.grouped_mm(x8, w8, off, sx, sw)
    for ld, start in ((160, 0), (155, 0), (168, 1), (168, 8)):
        buf = torch.full((rows * ld + 64,), 5.0, dtype=torch.bfloat16, device="cuda")
        y = buf[start:start + rows * ld].view(rows, ld)[:, :n]
        F.grouped_mm(x8, w8, off, sx, sw, y=y)
        assert torch.equal(y, want), (ld, start)
        y.fill_(5.0)
        assert bool((buf == 5.0).all()), (ld, start)


@pytest.mark.parametrize("bad", [[0, 90, 40, 200], [-7, 50, 60, 200], [0, 50, 60, 5000], [150, 120, 90, 20]])
def test_bad_offsets_stay_inside_the_buffers(bad):
    """Offsets that fall or leave the buffer are clamped: group e is [v(e), v(e + 1)) with v the running maximum of the
    clamped offsets.  Nothing outside y is touched."""
    rows, n, k = 200, 144, 64
    x8, w8, sx, sw = codes(rows, k, 0, 1), codes(n, k, 0, 2, batch=3), scales(1, 3), scales(3, 4)
    buf = torch.full((rows + 300, n), 5.0, dtype=torch.bfloat16, device="cuda")
    y = buf[150:150 + rows]
    F.grouped_mm(x8, w8, torch.tensor(bad, dtype=torch.int64, device="cuda"), sx, sw, y=y)
    v = np.maximum.accumulate(np.clip(bad, 0, rows))
    want = torch.full((rows, n), 5.0, dtype=torch.bfloat16, device="cuda")
    F.grouped_mm(x8, w8, torch.tensor(v, dtype=torch.int32, device="cuda"), sx, sw, y=want)
    assert torch.equal(y, want)
    assert bool((buf[:150] == 5.0).all()) and bool((buf[150 + rows:] == 5.0).all())
    assert F.fp8_get_device_status() == 0


@pytest.mark.parametrize("E,top", [(1024, 1), (1000, 5)])
def test_many_groups(E, top):
    counts = np.random.RandomState(E).randint(0, top + 1, E)
    rows, n, k = int(counts.sum()), 48, 32
    x8, w8, sx, sw = codes(rows, k, 0, 1), codes(n, k, 0, 2, batch=E), scales(1, 3), scales(E, 4)
    y = F.grouped_mm(x8, w8, offsets_of(counts), sx, sw)
    e = torch.from_numpy(np.repeat(np.arange(E), counts)).cuda()
    x, w = value(x8, 0), value(w8, 0)
    s = (float(sx) * sw[e].double())[:, None]
    assert_close(y, torch.einsum("rk,rnk->rn", x, w[e]) / s, torch.einsum("rk,rnk->rn", x.abs(), w[e].abs()) / s, E)


@pytest.mark.parametrize("wide", [torch.bfloat16, torch.float16, torch.float32])
def test_linear_training_steps(wide):
    """Two delayed-scaling steps of an expert layer through the public calls: codes, scales and rings equal the
    quantize's own, products equal 64-bit ones of those codes."""
    c, N, K = [40, 0, 131, 9], 208, 144
    rows, E = sum(c), len(c)
    off = offsets_of(c)
    gen = torch.Generator().manual_seed(3)
    rings = [F.ScaleRing(4) for _ in range(3)]
    alone = [F.ScaleRing(4) for _ in range(3)]
    for step in range(2):
        x = (torch.randn(rows, K, generator=gen) * (1 + step)).to(wide).cuda()
        w = (torch.randn(E, N, K, generator=gen) / 12).to(wide).cuda()
        g = (torch.randn(rows, N, generator=gen) * 1e-3).to(wide).cuda()
        f = F.grouped_linear_forward(x, w, off, rings[0], rings[1])
        b = F.grouped_linear_backward(g, f, off, rings[2])
        for t, fmt, ring, code, scale, amax in ((x, 0, alone[0], f.x8, f.sx, f.amax_x),
                                                (w.view(E * N, K), 0, alone[1], f.w8.reshape(E * N, K), f.sw, f.amax_w),
                                                (g, 1, alone[2], b.g8, b.sg, b.amax_g)):
            want, want_amax, want_scale = F.quantize(t, fmt, ring)
            assert torch.equal(code, want) and torch.equal(scale, want_scale) and torch.equal(amax, want_amax)
        for mine, theirs in zip(rings, alone):
            assert torch.equal(mine.words(), theirs.words())
        at = 0
        for e, m in enumerate(c):
            xe, ge, we = value(f.x8[at:at + m], 0), value(b.g8[at:at + m], 1), value(f.w8[e], 0)
            sx, sw, sg = float(f.sx), float(f.sw), float(b.sg)
            assert_close(f.y[at:at + m], xe @ we.t() / (sx * sw), xe.abs() @ we.abs().t() / (sx * sw), ("y", e))
            assert_close(b.dx[at:at + m], ge @ we / (sg * sw), ge.abs() @ we.abs() / (sg * sw), ("dx", e))
            assert_close(b.dw[e], ge.t() @ xe / (sg * sx), ge.abs().t() @ xe.abs() / (sg * sx), ("dw", e))
            at += m
    assert F.fp8_get_device_status() == 0


def test_linear_current_scaling_and_prequantized():
    """No rings (scales from the tensors' own amax); then fp8 operands with one weight scale per expert."""
    c, N, K = [17, 60], 96, 80
    rows, E = sum(c), len(c)
    off = offsets_of(c)
    gen = torch.Generator().manual_seed(4)
    x = torch.randn(rows, K, generator=gen).bfloat16().cuda()
    w = torch.randn(E, N, K, generator=gen).bfloat16().cuda()
    f = F.grouped_linear_forward(x, w, off, None, None)
    assert float(f.amax_x) == float(x.abs().max()) and float(f.amax_w) == float(w.abs().max())
    assert float(f.sx) == pytest.approx(448.0 / float(f.amax_x), rel=1e-6)
    sw = scales(E, 5)
    p = F.grouped_linear_forward(f.x8, f.w8, off, None, None, x_scale_in=f.sx, w_scale_in=sw)
    assert torch.equal(p.sw, sw) and torch.equal(p.sx, f.sx) and float(p.amax_x) == 0.0 and float(p.amax_w) == 0.0
    assert torch.equal(p.y, F.grouped_mm(f.x8, f.w8, off, f.sx, sw))
    # only one operand quantized
    h = F.grouped_linear_forward(x, f.w8, off, None, None, w_scale_in=sw)
    assert torch.equal(h.y, p.y)
    # no rows: the snapshot of the scales is still taken
    z = F.grouped_linear_forward(f.x8[:0], f.w8, offsets_of([0, 0]), None, None, x_scale_in=f.sx, w_scale_in=sw)
    assert z.y.shape == (0, N) and torch.equal(z.sw, sw) and float(z.amax_w) == 0.0


def test_gradients_against_differences():
    """The gradients of sum(y * h) with exactly representable operands: y is linear in each weight and each input, so a
    difference over a step that fp8 holds exactly gives the derivative."""
    c, N, K = [6, 0, 11], 32, 48
    rows = sum(c)
    off = offsets_of(c)
    gen = torch.Generator().manual_seed(6)
    grid = lambda *s: torch.randint(-3, 4, s, generator=gen).float()  # noqa: E731
    x, w, h = grid(rows, K), grid(3, N, K), grid(rows, N)
    one = torch.ones(1, device="cuda")

    def code(t, fmt):
        return t.to(TYPES[fmt]).view(torch.uint8).cuda().contiguous()

    def loss(x, w):
        y = F.grouped_mm(code(x, 0), code(w, 0), off, one, one)   # small whole sums: exact in bf16
        return float((y.double().cpu() * h.double()).sum())

    fwd = F.ForwardResult(None, code(x, 0), code(w, 0), one, one, None, None)
    b = F.grouped_linear_backward(code(h, 1), fwd, off, None, g_scale_in=one)
    base = loss(x, w)
    for r, k in ((0, 0), (5, 47), (6, 13), (16, 31)):
        y = x.clone()
        y[r, k] += 1.0
        assert loss(y, w) - base == float(b.dx[r, k])
    for e, n, k in ((0, 0, 0), (0, 31, 47), (1, 3, 3), (2, 16, 20)):
        v = w.clone()
        v[e, n, k] += 1.0
        assert loss(x, v) - base == float(b.dw[e, n, k])


def test_capture_streams_and_repeats():
    """Two calls captured into graphs on a side stream and replayed, with new offsets written between replays; results
    equal the eager ones bit for bit."""
    n, k, rows = 272, 320, 400
    x8, w8, sx, sw, sg = codes(rows, k, 0, 1), codes(n, k, 0, 2, batch=3), scales(1, 3), scales(3, 4), scales(1, 5)
    g8 = codes(rows, n, 1, 6)
    fwd = F.ForwardResult(None, x8, w8, sx, sw, None, None)
    off = offsets_of([100, 100, 200])
    y, dx = torch.zeros(rows, n, dtype=torch.bfloat16, device="cuda"), torch.zeros(rows, k, dtype=torch.bfloat16, device="cuda")
    dw = torch.zeros(3, n, k, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        F.grouped_mm(x8, w8, off, sx, sw, y=y)
    side.synchronize()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    with torch.cuda.graph(graphs[0]):
        F.grouped_mm(x8, w8, off, sx, sw, y=y)
    with torch.cuda.graph(graphs[1]):
        F.grouped_linear_backward(g8, fwd, off, None, g_scale_in=sg, dx=dx, dw=dw)
    for counts in ([100, 100, 200], [0, 399, 1], [133, 0, 267], [0, 0, 0]):
        new = offsets_of(counts)
        off.copy_(new)
        for t in (y, dx, dw):
            t.zero_()
        for gr in graphs:
            gr.replay()
        want = F.grouped_linear_backward(g8, fwd, new, None, g_scale_in=sg, dx=torch.zeros_like(dx))
        ref = F.grouped_mm(x8, w8, new, sx, sw, y=torch.zeros_like(y))
        torch.cuda.synchronize()
        assert torch.equal(y, ref) and torch.equal(dx, want.dx) and torch.equal(dw, want.dw)
    assert F.fp8_get_device_status() == 0


def test_calls_in_flight_together():
    """Two captured graphs and eager calls of other sizes on three streams at once, grouped and int8, with no
    synchronize between them: each result equals the call's own, run alone, bit for bit."""
    def operands(seed, rows, n, k, counts):
        gen = torch.Generator().manual_seed(seed)
        x8, w8, g8 = codes(rows, k, 0, seed), codes(n, k, 0, seed + 1, batch=len(counts)), codes(rows, n, 1, seed + 2)
        sx, sw, sg, off = scales(1, seed + 3), scales(len(counts), seed + 4), scales(1, seed + 5), offsets_of(counts)
        x = torch.randn(rows, k, generator=gen).bfloat16().cuda()
        q = torch.randint(-127, 128, (n, (k + 15) // 16 * 16), dtype=torch.int8, generator=gen).cuda()[:, :k]
        qs = torch.rand(n, generator=gen).cuda()
        outs = [torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
                for shape in ((rows, n), (rows, k), (len(counts), n, k), (rows, n))]

        def run():
            F.grouped_mm(x8, w8, off, sx, sw, y=outs[0])
            F.grouped_linear_backward(g8, F.ForwardResult(None, x8, w8, sx, sw, None, None), off, None, g_scale_in=sg,
                                      dx=outs[1], dw=outs[2])
            F.linear_int8(x, q, qs, y=outs[3])
        return outs, run

    sets = [operands(1, 40, 272, 1040, [7, 0, 33]), operands(20, 900, 520, 384, [300, 1, 599]),
            operands(40, 3, 1511, 1000, [1, 1, 1])]
    want = []
    for outs, run in sets:
        run()
        torch.cuda.synchronize()
        want.append([o.clone() for o in outs])
    graphs = []
    for _, run in sets[:2]:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            run()
    for outs, _ in sets:
        for o in outs:
            o.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(30):
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
        with torch.cuda.stream(streams[2]):
            sets[2][1]()
    torch.cuda.synchronize()
    for (outs, _), ref in zip(sets, want):
        assert all(torch.equal(o, r) for o, r in zip(outs, ref))
    assert F.fp8_get_device_status() == 0


def test_empty_contraction():
    """k = 0: the groups' rows are zero, whatever the scales, the others stay."""
    off = torch.tensor([1, 3, 3, 40], dtype=torch.int32, device="cuda")
    nan = torch.full((1,), float("nan"), device="cuda")
    for n in (32, 33, 5000):
        y = torch.full((50, n), 7.0, dtype=torch.bfloat16, device="cuda")
        F.grouped_mm(torch.empty(50, 0, dtype=torch.uint8, device="cuda"),
                     torch.empty(3, n, 0, dtype=torch.uint8, device="cuda"), off, nan, nan, y=y)
        assert bool((y[1:40] == 0).all()) and bool((y[:1] == 7).all()) and bool((y[40:] == 7).all())


def test_one_weight_for_all_groups():
    """stride_b 0: every group uses the same weight, with scales of their own."""
    c, n, k = [40, 0, 90], 176, 112
    rows = sum(c)
    x8, w8, sx, sw, off = codes(rows, k, 0, 1), codes(n, k, 0, 2), scales(1, 3), scales(3, 4), offsets_of(c)
    y = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
    a = F.MmArgs(rows, n, k, x8.data_ptr(), 0, 0, x8.stride(0), w8.data_ptr(), 0, 0, w8.stride(0), sx.data_ptr(),
                 sw.data_ptr(), None, 0, None, y.data_ptr(), n, 0, None, 0)
    F.fp8_mm_grouped(a, F.FP8_RAGGED_M, F.Groups(3, off.data_ptr(), 0, 0, 0, 1), y.device)
    three = torch.zeros(3, n, w8.stride(0), dtype=torch.uint8, device="cuda")
    three[:, :, :k] = w8
    assert torch.equal(y, F.grouped_mm(x8, three[:, :, :k], off, sx, sw))


def test_weight_gradient_scales_and_pitches():
    """Through the C entry: one scale per group, and D with a row pitch and a gap between the groups."""
    c, n, k = [33, 0, 64, 7], 130, 72
    rows, ld, gap = sum(c), 80, 130 * 80 + 48
    x8, g8, sg, sx, off = codes(rows, k, 0, 1), codes(rows, n, 1, 2), scales(1, 3), scales(4, 4), offsets_of(c)
    buf = torch.full((4 * gap,), 3.0, dtype=torch.bfloat16, device="cuda")
    a = F.MmArgs(n, k, rows, g8.data_ptr(), 1, 1, g8.stride(0), x8.data_ptr(), 0, 1, x8.stride(0), sg.data_ptr(),
                 sx.data_ptr(), None, 0, None, buf.data_ptr(), ld, 0, None, 0)
    F.fp8_mm_grouped(a, F.FP8_RAGGED_K, F.Groups(4, off.data_ptr(), 0, 0, gap, 1), buf.device)
    at = 0
    for e, m in enumerate(c):
        x, g, s = value(x8[at:at + m], 0), value(g8[at:at + m], 1), float(sg) * float(sx[e])
        d = buf[e * gap:e * gap + n * ld].view(n, ld)
        assert_close(d[:, :k], g.t() @ x / s, g.abs().t() @ x.abs() / s, e)
        assert bool((d[:, k:] == 3.0).all()) and bool((buf[e * gap + n * ld:(e + 1) * gap] == 3.0).all())
        at += m


def test_weights_and_gradients_past_31_bits():
    """Weights of more than 2^31 bytes, and a weight gradient of more than 2^31 elements."""
    E, n, k = 9, 16384, 16640
    assert E * n * k > 2 ** 31
    c = [3, 0, 40, 1, 0, 0, 2, 0, 18]
    rows = sum(c)
    off = offsets_of(c)
    w8 = torch.randint(0, 0x40, (E, n, k), dtype=torch.uint8, device="cuda")
    x8, g8, sx, sg = codes(rows, k, 0, 1), codes(rows, n, 1, 2), scales(1, 3), scales(1, 4)
    b = F.grouped_linear_backward(g8, F.ForwardResult(None, x8, w8, sx, sx, None, None), off, None, g_scale_in=sg)
    y = F.grouped_mm(x8, w8, off, sx, sx)
    e = 8
    x, g, w = value(x8[46:], 0), value(g8[46:], 1), value(w8[e], 0)
    s, sd, sdw = float(sx) ** 2, float(sg) * float(sx), float(sg) * float(sx)
    assert_close(y[46:], x @ w.t() / s, x.abs() @ w.abs().t() / s, "y")
    assert_close(b.dx[46:], g @ w / sd, g.abs() @ w.abs() / sd, "dx")
    at = slice(n - 300, n)
    assert_close(b.dw[e, at], g[:, at].t() @ x / sdw, g[:, at].abs().t() @ x.abs() / sdw, "dw")
    assert bool((b.dw[7, at] == 0).all())


def test_column_offsets_past_31_bits():
    """Rows of y beyond 2^31 elements."""
    n, k, rows = 11008, 16, 200_000
    assert rows * n > 2 ** 31
    x8 = torch.randint(0, 0x40, (rows, k), dtype=torch.uint8, device="cuda")
    w8 = codes(n, k, 0, 2, batch=2)
    sx, sw = scales(1, 3), scales(2, 4)
    off = torch.tensor([0, 150_000, rows], dtype=torch.int64, device="cuda")
    y = F.grouped_mm(x8, w8, off, sx, sw)
    for r0, e in ((0, 0), (149_900, 0), (150_000, 1), (rows - 100, 1)):
        x, w = value(x8[r0:r0 + 100], 0), value(w8[e], 0)
        s = float(sx) * float(sw[e])
        assert_close(y[r0:r0 + 100], x @ w.t() / s, x.abs() @ w.abs().t() / s, r0)
