"""barrier.cluster in its aligned form needs every thread of a warp to arrive together.
After code in which threads take their own ways only a block barrier ahead of it makes
sure of that: each cluster barrier of the step's kernels has one."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "cross_entropy_rl_gb300", "csrc")


@pytest.mark.parametrize("name", ["embed_kernels.cu", "policy_kernels.cu", "grad_kernels.cu"])
def test_a_block_barrier_ahead_of_each(name):
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    ahead = re.findall(r"([^;{}]*;)\s*(?:if \([^()]*\)\s*)?cluster_barrier\(\);", code)
    assert len(ahead) == code.count("cluster_barrier();") > 0
    assert [a.strip() for a in ahead] == ["__syncthreads();"] * len(ahead)
