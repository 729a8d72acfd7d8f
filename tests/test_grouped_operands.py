"""Operands of the grouped helpers that come as fp8 codes, refused or accepted before anything is enqueued (CPU
tensors: a call whose operands are in order is refused for its device, and for nothing before that)."""
import pytest
import torch

NOT_ON_GPU = "expected CUDA tensors"
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


@pytest.fixture(scope="module")
def fp8():
    import fp8_delayed_scaling_03_b200 as m
    return m


def operands():
    one = torch.ones(1)
    return dict(x=torch.zeros(4, 16, dtype=torch.uint8), w=torch.zeros(2, 32, 16, dtype=torch.uint8),
                g=torch.zeros(4, 32, dtype=torch.uint8), off=torch.tensor([0, 2, 4], dtype=torch.int32), one=one)


def forward(fp8, o, x=None, w=None, **kw):
    kw = dict(x_scale_in=o["one"], w_scale_in=o["one"]) | kw
    return fp8.grouped_linear_forward(o["x"] if x is None else x, o["w"] if w is None else w, o["off"], None, None, **kw)


def backward(fp8, o, g=None, **kw):
    fwd = fp8.ForwardResult(None, o["x"], o["w"], o["one"], o["one"], None, None)
    return fp8.grouped_linear_backward(o["g"] if g is None else g, fwd, o["off"], None, **dict(g_scale_in=o["one"]) | kw)


def test_a_buffer_for_codes_that_are_there_already_is_refused(fp8):
    """An operand that comes as codes is used in place.  A buffer for its codes would never be written, and a backward
    pass that took it from the result would multiply by what it happens to hold."""
    o = operands()
    for kw in (dict(x8=torch.zeros(4, 16, dtype=torch.uint8)), dict(w8=torch.zeros(2, 32, 16, dtype=torch.uint8)),
               dict(x=o["x"].view(E4M3), x8=torch.zeros(4, 16, dtype=torch.uint8)),
               dict(x8=torch.zeros(4, 32, dtype=torch.uint8)[:, :16]), dict(x8=o["w"][0, :4])):
        with pytest.raises(ValueError, match="already fp8 codes"):
            forward(fp8, o, **kw)
    for kw in (dict(), dict(g=o["g"].view(E5M2))):
        with pytest.raises(ValueError, match="already fp8 codes"):
            backward(fp8, o, g8=torch.zeros(4, 32, dtype=torch.uint8), **kw)


def test_the_operand_itself_as_its_buffer_is_accepted(fp8):
    o = operands()
    xf = o["x"].view(E4M3)
    for kw in (dict(x8=o["x"]), dict(w8=o["w"]), dict(x8=o["x"], w8=o["w"]), dict(x=xf, x8=o["x"]), dict(x=xf, x8=xf),
               dict(x8=o["x"][:, :])):
        with pytest.raises(ValueError, match=NOT_ON_GPU):
            forward(fp8, o, **kw)
    for kw in (dict(g8=o["g"]), dict(g=o["g"].view(E5M2), g8=o["g"]), dict()):
        with pytest.raises(ValueError, match=NOT_ON_GPU):
            backward(fp8, o, **kw)


def test_buffers_of_operands_quantized_here(fp8):
    """Shape and type of the buffers for a wide operand's codes."""
    o = operands()
    x, w, g = torch.zeros(4, 16), torch.zeros(2, 32, 16), torch.zeros(4, 32)
    with pytest.raises(ValueError, match=NOT_ON_GPU):
        forward(fp8, o, x=x, w=w, x8=o["x"], w8=o["w"])
    with pytest.raises(ValueError, match=NOT_ON_GPU):
        backward(fp8, o, g=g, g8=o["g"])


def test_scales_of_codes_are_one_fp32_value(fp8):
    """The kernels read a scale as one fp32 word: another type would be read as another number, an empty tensor past
    its end."""
    o = operands()
    bad = (torch.ones(1, dtype=torch.float64), torch.ones(1, dtype=torch.bfloat16), torch.ones(2), torch.ones(0),
           torch.ones(1, dtype=torch.int32))
    for s in bad:
        with pytest.raises(ValueError, match="x_scale_in"):
            forward(fp8, o, x_scale_in=s)
        with pytest.raises(ValueError, match="g_scale_in"):
            backward(fp8, o, g_scale_in=s)
    for s in (torch.ones(()), torch.ones(1, 1), torch.ones(4)[2:3]):
        with pytest.raises(ValueError, match=NOT_ON_GPU):
            forward(fp8, o, x_scale_in=s)
        with pytest.raises(ValueError, match=NOT_ON_GPU):
            backward(fp8, o, g_scale_in=s)
    # a wide operand's scale comes from its ring or its amax: what is passed is not read
    with pytest.raises(ValueError, match=NOT_ON_GPU):
        forward(fp8, o, x=torch.zeros(4, 16), x_scale_in=bad[0])
