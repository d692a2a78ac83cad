"""A 4-bit matrix made from stored buffers, taken back before any other call of the process."""
import subprocess
import sys

import pytest

CODE = """
import torch
import cross_entropy_rl_gb300 as ll
L = ll.load()
q = ll.FP4Matrix(torch.zeros(4, L.ll_fp4_row_bytes(64), dtype=torch.uint8),
                 torch.zeros(L.ll_fp4_scale_bytes(4, 64, 0), dtype=torch.uint8), None, 64)
try:
    %s
except ll.LLError as e:  # host memory: refused by the C ABI, so the binding let it through
    assert e.status in (1, 6), e
    print("refused")
"""


@pytest.mark.parametrize("call", ["ll.fp4_dequantize(q)", "ll.fp4_dequantize(q, torch.bfloat16)",
                                  "ll.fp4_linear(q, q)", "ll.fp4_quantize(torch.zeros(4, 64))"])
def test_first_call(call):
    from cross_entropy_rl_gb300 import build as B
    B.build()
    r = subprocess.run([sys.executable, "-c", CODE % call], capture_output=True, text=True, cwd=B.ROOT,
                       timeout=600)
    assert r.returncode == 0 and r.stdout.strip() == "refused", r.stderr
