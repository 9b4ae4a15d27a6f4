"""The selective scan's log1p polynomial, read from the kernel source: s P(s^2) with s = e / (2 + e) against log1p(e)
over e in (0, 1], in fp32 Horner form as the kernel evaluates it. Five roundings of at most half a step (the
quotient, its square, the last two multiply-adds, the product) and the polynomial's own 4.1e-9 stay below 5 * 2^-24.
"""
import os
import re

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_log1p_polynomial():
    src = open(os.path.join(ROOT, "test_sequence_layers_amd", "csrc", "scan.hip")).read()
    m = re.search(r"kLog1pP\[(\d+)\]\s*=\s*\{([^}]*)\}", src)
    c = [np.float32(v.strip().rstrip("f")) for v in m.group(2).split(",")]
    assert len(c) == int(m.group(1))
    e = np.concatenate([np.exp(-np.linspace(0, 80, 200001)), np.linspace(1e-6, 1, 200001)]).astype(np.float32)
    s = (e / (np.float32(2) + e)).astype(np.float32)
    q = s * s
    p = np.full_like(q, c[-1])
    for v in c[-2::-1]:  # (a fused multiply-add rounds once: the product is exact in float64)
        p = (p.astype(np.float64) * q + np.float64(v)).astype(np.float32)
    got, ref = (s * p).astype(np.float64), np.log1p(e.astype(np.float64))
    assert np.abs(got / ref - 1).max() < 5 * 2.0 ** -24
