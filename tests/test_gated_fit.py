"""The polynomial behind gelu's normal distribution, from its source (CPU only): the coefficients as
they are stored, in fp32, against the function that they stand for."""
import math
import os
import re

from fp4_communication_compression_amd import _build

TEXT = open(os.path.join(_build.HERE, "csrc", "fp4q_act.h")).read()
# what the comment says of it, over 0 <= x <= 30 (e^(-x^2 / 2) is below 2^-126 from 13.3 on)
OFF, END = 4.8e-8, 30.0


def test_normal_distribution():
    """P(-x) = t Q(t) e^(-x^2 / 2), t = 1 / (1 + c x): of Q the relative error in 64 bits."""
    found = re.search(r"constexpr float kQ\[\] = \{([^}]*)\}", TEXT).group(1)
    q = [float.fromhex(v.strip().rstrip("f")) for v in found.split(",")]
    c = float(re.search(r"fmaf\(([0-9.]+)f, fabsf\(g\), 1\.0f\)", TEXT).group(1))
    assert len(q) == 10 and abs(c - 0.45 / math.sqrt(2)) < 1e-15
    worst = 0.0
    for i in range(60001):
        x = END * i / 60000
        t, value = 1 / (1 + c * x), 0.0
        for v in reversed(q):
            value = value * t + v
        want = 0.5 * math.erfc(x / math.sqrt(2)) * math.exp(x * x / 2)
        worst = max(worst, abs(value * t / want - 1))
    assert 0.95 * OFF < worst <= OFF, worst
    assert "%.1fe-8" % (OFF * 1e8) in TEXT
