"""Operands of linear_forward / linear_backward that come as fp8 codes: the codes that the results hold (on a GPU)."""
import pytest
import torch


@pytest.fixture(scope="module")
def fp8():
    import fp8_delayed_scaling_03_b200 as m
    return m


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
