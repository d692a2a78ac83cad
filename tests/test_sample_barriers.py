"""The length of the list of tokens is read by all threads of a block, and the outcome decides
which barriers they meet: nobody may clear it between another thread's read and a barrier."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "cross_entropy_rl_gb300", "csrc")


def code():
    with open(os.path.join(CSRC, "sample_kernels.cu")) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def body(name):
    text = code()
    start = re.search(r"\b%s\([^()]*\)\s*(?:const\s*)?\{" % name, text).end()
    depth, at = 1, start
    while depth:
        depth += {"{": 1, "}": -1}.get(text[at], 0)
        at += 1
    return text[start:at]


def test_what_follows_an_overflow_leaves_the_length_alone():
    # both run between the read of the length and the next barrier
    assert "n_list" not in body("start_min") and "n_list" not in body("start_wide")


def test_a_barrier_ahead_of_each_clearing():
    for name in ("run", "find_piece"):
        text = body(name)
        clears = [m.start() for m in re.finditer(r"sh\.n_list = 0;", text)]
        assert len(clears) == 1
        read = max([m.start() for m in re.finditer(r"\w+ = sh\.n_list;", text) if m.start() < clears[0]],
                   default=0)
        assert re.search(r"__syncthreads\(\);|block_sum\(", text[read:clears[0]])
