"""What no run can show: orderings that the memory model asks for, read in the source."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_attention_kv_csa_gb300", "csrc")


def test_space_of_the_sums_goes_to_the_async_proxy_behind_a_fence():
    """The attention's prefix sums lie where TMA later writes tiles: every thread has its proxy fence between its last use
    of them and the block barrier before the first copy."""
    with open(os.path.join(CSRC, "csa_latent_mma.cu")) as f:
        kernel = re.sub(r"//[^\n]*", "", f.read())
    kernel = kernel[kernel.index("latent_mma_kernel(const AttnParams"):]
    sums = kernel[kernel.index("int *items"):kernel.index("if (warp < kSoftWarps)")]
    end = sums.rindex("__syncthreads();")
    last_use = max(sums.rindex(w) for w in ("items[", "kept[", "fact("))
    assert last_use < sums.index("fence_async_smem();", last_use) < end
