"""What reading the source of the 4-bit cache's kernels has to show."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "lsh_sampled_sparse_gb300", "csrc")


def test_dependent_kernels_of_the_4_bit_cache_make_no_non_coherent_load():
    """A kernel launched as a dependent begins before its predecessor has written positions, lengths,
    queries or rows; a non-coherent load promises that nobody writes them during its life."""
    with open(os.path.join(CSRC, "mp_kv4.cu")) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert code.count("launch_dependent(") == 4
    assert "__ldg(" not in code and ".global.nc" not in code and "__restrict__" not in code
    kernels = re.findall(r"__global__.*?\n}\n", code, re.S)
    assert len(kernels) == 4 and all("wait_for_predecessor();" in k for k in kernels)
