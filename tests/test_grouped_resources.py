"""The grouped and 8-bit integer kernels as ptxas reports them for sm_100a (nvcc only, no GPU): no build spills, and
every build of the product keeps within the registers that one CTA an SM leaves its threads."""
import re

import pytest

from test_kernel_resources import ptxas_report


@pytest.fixture(scope="module")
def products():
    return {n: r for n, r in ptxas_report("grouped.cu").items() if "grouped_kernel" in n}


def test_products(products):
    assert len(products) == 14  # fp8 and int8 (three outputs): single, pair, split; the weight gradient: single, pair
    for name, res in products.items():
        assert res["spill"] == 0, (name, res)
        ragged_k = re.search(r"grouped_kernelILb[01]ELb([01])", name).group(1) == "1"
        threads = 352 if ragged_k else 320
        assert res["regs"] * threads <= 65536, (name, res)


def test_row_quantize():
    kernels = ptxas_report("quantize_int8.cu")
    assert len(kernels) == 3
    for name, res in kernels.items():
        assert res["spill"] == 0 and res["regs"] * 512 <= 65536, (name, res)
