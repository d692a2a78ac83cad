"""A CTA must not end while a load into its shared memory is in flight, also after one of its
bounded waits ran out: the producers of the 4-bit product keep a record of their loads and
wait for them, with a limit, before they leave, whichever warp gave up."""
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


@pytest.mark.parametrize("kernel,barriers", [("few_kernel", ["full"]), ("pair_kernel", ["landed", "full"])])
def test_producers_wait_for_their_loads(kernel, barriers):
    with open(os.path.join(CSRC, "fp4_gemm.cu")) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    start = code.index(kernel + "(const __grid_constant__")
    start = code.index("if (warp == 0) {", start)
    producer = code[start:block_end(code, start)]
    loads = producer[producer.index("for ("):]
    rest = loads[block_end(loads, 0):]
    loads = loads[:block_end(loads, 0)]
    # every stage that the loop loads is recorded, ahead of the step to the next
    assert len(re.findall(r"tma_load_2d(?:_pair)?\(", loads)) == 2
    assert re.search(r"issued\.add\(stage, phase\);\s*if \(\+\+stage == ", loads)
    # and waited for behind the loop, outside of what runs after a time-out alone
    gave_up = rest.index("if (!ok)")
    always = rest[:gave_up] + rest[block_end(rest, gave_up):]
    for name in barriers:
        assert re.search(r"wait_for_loads\(bars\.%s, issued, P\.wait_ns\)" % name, always)
