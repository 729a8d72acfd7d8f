"""Operands of linear_forward / linear_backward that come as fp8 codes: their scales, checked before any pointer is
taken, and (on a GPU) the codes that the results hold."""
import pytest
import torch


@pytest.fixture(scope="module")
def fp8():
    import fp8_delayed_scaling_03_b200 as m
    return m


def test_scales_of_codes_are_fp32(fp8):
    """The kernels read a scale as one fp32 word: another type would be read as another number, an empty tensor past
    its end."""
    x, w, g = (torch.zeros(s, dtype=torch.uint8) for s in ((4, 16), (32, 16), (4, 32)))
    one = torch.ones(1)
    fwd = fp8.ForwardResult(None, x, w, one, one, one, one)
    for bad in (torch.ones(1, dtype=torch.float64), torch.ones(1, dtype=torch.bfloat16), torch.ones(0)):
        with pytest.raises(ValueError, match="x_scale_in"):
            fp8.linear_forward(x, w, None, None, x_scale_in=bad, w_scale_in=one)
        with pytest.raises(ValueError, match="w_scale_in"):
            fp8.linear_forward(x, w, None, None, x_scale_in=one, w_scale_in=bad)
        with pytest.raises(ValueError, match="g_scale_in"):
            fp8.linear_backward(g, fwd, None, g_scale_in=bad)


@pytest.mark.gpu
def test_results_hold_the_codes_that_were_multiplied(fp8):
    """A buffer passed for the codes of an operand that is codes already is not written: the results hold the operand's
    own, and the backward equals the one of a forward without the buffers, bit for bit."""
    M, N, K = 96, 128, 64
    gen = torch.Generator().manual_seed(2)
    x8, _, sx = fp8.quantize(torch.randn(M, K, generator=gen).bfloat16().cuda(), fp8.FP8_E4M3, None)
    w8, _, sw = fp8.quantize(torch.randn(N, K, generator=gen).bfloat16().cuda(), fp8.FP8_E4M3, None)
    g8, _, sg = fp8.quantize(torch.randn(M, N, generator=gen).bfloat16().cuda(), fp8.FP8_E5M2, None)

    def buffer(*shape):
        return torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda")   # NaN codes

    results = []
    for fkw, bkw in (({}, {}), (dict(x8=buffer(M, K), w8=buffer(N, K)), dict(g8=buffer(M, N)))):
        f = fp8.linear_forward(x8, w8, None, None, x_scale_in=sx, w_scale_in=sw, **fkw)
        b = fp8.linear_backward(g8, f, None, g_scale_in=sg, need_dbias=True, **bkw)
        assert torch.equal(f.x8, x8) and torch.equal(f.w8, w8) and torch.equal(b.g8, g8)
        results.append((f.y, b.dx, b.dw, b.dbias))
    for got, want in zip(*results):
        assert torch.equal(got, want) and not bool(got.isnan().any())
