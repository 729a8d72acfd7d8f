"""The grouped linears with some operands quantized beforehand and the others into the caller's own buffers: forward,
then the backward on what the forward returned, against 64-bit products of the codes in those results.

Tolerance, per element: one bf16 rounding (2^-8 of the value) and fp32 accumulation, 2e-6 of the products' magnitudes."""
import itertools

import pytest
import torch

import fp8_delayed_scaling_03_b200 as F

pytestmark = pytest.mark.gpu


def decoded(codes, dtype):
    return codes.contiguous().view(dtype).double()


def assert_close(got, want, mags, what):
    assert bool(((got.double() - want).abs() <= want.abs() * 2.0 ** -8 + mags * 2e-6).all()), what


@pytest.mark.parametrize("x_codes,w_codes,g_codes", list(itertools.product((False, True), repeat=3)))
def test_backward_multiplies_by_the_codes_of_the_forward(x_codes, w_codes, g_codes):
    counts, N, K = [20, 0, 43], 80, 112
    rows, E = sum(counts), len(counts)
    off = torch.tensor([0, 20, 20, 63], dtype=torch.int32, device="cuda")
    gen = torch.Generator().manual_seed(11)
    x = torch.randn(rows, K, generator=gen).bfloat16().cuda()
    w = (torch.randn(E, N, K, generator=gen) / 10).bfloat16().cuda()
    g = (torch.randn(rows, N, generator=gen) * 1e-2).bfloat16().cuda()
    kw, bkw = {}, {}
    if x_codes:
        x, _, kw["x_scale_in"] = F.quantize(x, F.FP8_E4M3, None)
    else:   # the caller's buffers hold NaN codes until the call
        kw["x8"] = torch.full((rows, K), 0x7F, dtype=torch.uint8, device="cuda")
    if w_codes:
        w, _, kw["w_scale_in"] = F.quantize(w.view(E * N, K), F.FP8_E4M3, None)
        w = w.reshape(E, N, K)
    else:
        kw["w8"] = torch.full((E, N, K), 0x7F, dtype=torch.uint8, device="cuda")
    if g_codes:
        g, _, bkw["g_scale_in"] = F.quantize(g, F.FP8_E5M2, None)
    else:
        bkw["g8"] = torch.full((rows, N), 0x7F, dtype=torch.uint8, device="cuda")
    f = F.grouped_linear_forward(x, w, off, None, None, **kw)
    b = F.grouped_linear_backward(g, f, off, None, **bkw)
    for mine, operand, buffer, is_codes in ((f.x8, x, kw.get("x8"), x_codes), (f.w8, w, kw.get("w8"), w_codes),
                                            (b.g8, g, bkw.get("g8"), g_codes)):
        assert mine.data_ptr() == (operand if is_codes else buffer).data_ptr()
    sx, sw, sg = float(f.sx), float(f.sw), float(b.sg)
    at = 0
    for e, m in enumerate(counts):
        xe, we = decoded(f.x8[at:at + m], torch.float8_e4m3fn), decoded(f.w8[e], torch.float8_e4m3fn)
        ge = decoded(b.g8[at:at + m], torch.float8_e5m2)
        assert_close(f.y[at:at + m], xe @ we.t() / (sx * sw), xe.abs() @ we.abs().t() / (sx * sw), ("y", e))
        assert_close(b.dx[at:at + m], ge @ we / (sg * sw), ge.abs() @ we.abs() / (sg * sw), ("dx", e))
        assert_close(b.dw[e], ge.t() @ xe / (sg * sx), ge.abs().t() @ xe.abs() / (sg * sx), ("dw", e))
        at += m
    assert F.fp8_get_device_status() == 0
