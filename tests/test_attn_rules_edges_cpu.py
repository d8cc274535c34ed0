"""The arithmetic of attention's rules, without a GPU."""
import os
import re

import numpy as np

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "int4_gathered_expert_gb300", "csrc")


def test_the_caps_polynomial_by_itself():
    """tanh(u) / u up to u = 1 by the kernels' factors in 64 bits: as near as their comment says, 4.1e-9 and 5.4e-9 of
    itself (a degree of 7 in u^2 that begins with 1 can come to 4.05e-9)."""
    src = open(os.path.join(CSRC, "e0_attn.cuh")).read()
    body = src[src.index("tanh_of(int i)"):]
    c = [np.float64(np.float32(x)) for x in re.findall(r"[?:] (-?\d+\.\d+)f", body[:body.index("}")])]
    assert len(c) == 8
    u = np.linspace(1e-3, 1, 100001)
    p = np.polynomial.polynomial.polyval(u * u, c)
    want = np.tanh(u) / u
    assert np.abs(p - want).max() < 4.15e-9 and np.abs(p / want - 1).max() < 5.45e-9
