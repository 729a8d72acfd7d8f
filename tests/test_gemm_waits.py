"""Give-up path of the GEMM kernels (their source; no GPU is made to wait): bulk loads that are under way when a wait
gives up land in shared memory that the block still owns."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_a_block_that_gave_up_outlives_its_copies():
    text = open(os.path.join(ROOT, "fp8_delayed_scaling_03_b200", "csrc", "gemm.cu")).read()
    text = re.sub(r"//[^\n]*", "", text)
    end = text[text.rindex("else cta_sync();"):text.index("int pair_capacity_impl")]
    assert "settle_copies(abort_flag)" in end
    # the pair's issuer waits for both blocks' loads: the other block has to know that it gave up
    issuer = text[text.index("} else if (warp == 1) {"):text.index("float4* const part_row")]
    assert re.search(r"kPair && \*abort_flag\)\s*st_cluster_u32\(mapa_shared\(smem_u32\(const_cast<const int\*>\(abort_flag\)\), 1\), 1u\)",
                     issuer)
