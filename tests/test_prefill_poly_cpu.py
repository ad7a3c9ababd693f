"""The prompts' kernel and the others have the same softplus polynomial (CPU)."""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "linear_attention_speculative_kda_gb300", "csrc")


def coefficients(name, function):
    text = open(os.path.join(CSRC, name)).read()
    body = re.search(function + r".*?constexpr float c\[10\] = \{(.*?)\};", text, re.S).group(1)
    return [float.fromhex(x.strip().rstrip("f")) for x in body.split(",")]


def test_one_polynomial():
    want = coefficients("kda_device.cuh", r"float softplus\(float x\) \{")
    assert len(want) == 10
    assert coefficients("kda_prefill.cu", r"Poly softplus_poly\(\) \{") == want
