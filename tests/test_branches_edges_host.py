"""Edges of the operators for several continuations of a sequence that need no GPU."""
import os
import re

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "dynamic_sparsity_approximate_amd", "csrc")


def test_the_largest_logits_exponential_stays_near_one():
    """What the selection's reading kernel computes for a wave's largest logit, in the kernel's own steps: up to the
    size at which it stops to, that is between 1/4 and 4; at 1e10 it would overflow."""
    with open(os.path.join(SRC, "beam.hip")) as f:
        found = re.search(r"bool has_power\(float top\) { return fabsf\(top\) <= 0x1p(\d+)f; }", f.read())
    limit = 2.0 ** int(found.group(1))
    hi, lo = np.float32(1.4426950408889634), np.float32(1.925963033500995e-8)
    assert abs(float(hi) + float(lo) - np.log2(np.e)) < 2.0 ** -50

    def exponent(top):
        top = top.astype(np.float32)
        c = (top * hi).astype(np.float64)  # rounded to fp32
        # an fma: a product of 48 bits and its difference are exact in 64
        rest = (top.astype(np.float64) * float(hi) - c).astype(np.float32)
        return (top.astype(np.float64) * float(lo) + rest).astype(np.float32)

    rng = np.random.default_rng(1)
    tops = np.concatenate([limit * (1 - rng.random(100000) * 0.75), limit * 2.0 ** -rng.uniform(0, 60, 100000), [limit]])
    assert np.abs(exponent(np.concatenate([tops, -tops]))).max() < 2.0
    assert np.abs(exponent(np.array([1e10, -1e10]))).max() > 128.0
