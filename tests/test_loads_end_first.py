"""A CTA must not end while a load into its shared memory is in flight, also after one of its
bounded waits ran out: the producers of the 4-bit product and of the GEMM on CTA pairs keep a
record of their loads and wait for them, with a limit, before they leave, whichever warp
gave up."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "cross_entropy_rl_gb300", "csrc")


def block_end(text, at):
    """Index behind the block that opens at or after `at`."""
    at = text.index("{", at) + 1
    depth = 1
    while depth:
        depth += {"{": 1, "}": -1}.get(text[at], 0)
        at += 1
    return at


@pytest.mark.parametrize("source,kernel,waits", [
    ("fp4_gemm.cu", "few_kernel", ["wait_for_loads(bars.full, issued"]),
    ("fp4_gemm.cu", "pair_kernel", ["wait_for_loads(bars.landed, issued",
                                    "if (leader) wait_for_pair_loads(bars.full, issued"]),
    ("gemm_tc.cu", "gemm_pair_kernel", ["if (leader) wait_for_pair_loads(bars->full, issued"]),
])
def test_producers_wait_for_their_loads(source, kernel, waits):
    with open(os.path.join(CSRC, source)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    start = re.search(r"\b%s\(const __grid_constant__" % kernel, code).end()
    start = code.index("if (warp == 0) {", start)
    producer = code[start:block_end(code, start)]
    at = re.search(r"\b(for|while) \([^{]*\{", producer)
    loads = producer[at.start():block_end(producer, at.start())]
    rest = producer[at.start() + len(loads):]
    # every stage that the loop loads is recorded, ahead of the step to the next
    assert re.search(r"\w*load\w*(<[^()]*>)?\(", loads)
    assert [x.strip() for x in re.findall(r"(.*);\s*if \(\+\+stage == ", loads)] == ["issued.add(stage, phase)"]
    # and waited for behind the loop, outside of what runs after a time-out alone
    gave_up = rest.index("if (!ok)")
    always = re.sub(r"\s+", " ", rest[:gave_up] + rest[block_end(rest, gave_up):])
    for wait in waits:
        assert wait in always
