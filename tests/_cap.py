"""The forms in which the attention kernels cap a score (csrc/rx_rules.cuh), one
fp32 operation at a time, with the coefficients of the source.  For the tests of
the error that include/rx.h states."""
import os
import re

import numpy as np

F = np.float32
LOG2E = F(1.4426950408889634)
SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "prefix_shared_kv_radixattention_gb300", "csrc",
                      "rx_rules.cuh")


def coefficients(name):
    """P: tanh y = y P(y^2) up to 1, Q: up to 3/8."""
    with open(SOURCE) as f:
        m = re.search(r"static const \w+ " + name + r"\[\d\] = \{([^}]*)\}", f.read())
    return [float(x.rstrip("f")) for x in m.group(1).replace(" ", "").split(",")]


def fma(a, b, c):
    return (np.asarray(a, np.float64) * np.asarray(b, np.float64) + np.asarray(c, np.float64)).astype(F)


class Cap:
    """As make_rules fills it in; x: the products q . k (fp32), results in log2 units less the base."""

    def __init__(self, cap, scale=0.125, fixed=None):
        self.cap, self.sl2 = F(cap), F(F(scale) * LOG2E)
        self.c2 = F(self.cap * LOG2E)
        self.fixed = bool(self.c2 <= F(72.2)) if fixed is None else fixed
        self.base = F(min(self.c2, F(100) - self.c2)) if self.fixed else F(0)
        self.scale = float(F(scale))

    def true(self, x):
        """cap tanh(s / cap), in 64 bits."""
        s = np.asarray(x, np.float64) * self.scale
        return float(self.cap) * np.tanh(s / float(self.cap))

    def near_in_range(self):
        """Whether make_rules leaves the form of degree 7 on: its coefficients within fp32's normal range."""
        k1 = float(self.sl2) / float(self.c2)
        return all(2e-38 < abs(q * float(self.c2) * k1 ** (2 * i + 1)) < 1e18 for i, q in enumerate(coefficients("Q")))

    def near(self, x):
        k1 = float(self.sl2) / float(self.c2)
        c, out = float(self.c2) * k1, []
        for q in coefficients("Q"):
            out.append(F(q * c))
            c *= k1 * k1
        z = F(x) * F(x)
        r = fma(out[3], z, out[2])
        r = fma(r, z, out[1])
        r = fma(r, z, out[0])
        return fma(r, x, -self.base)

    def poly(self, x):
        c = [F(F(p) * self.c2) for p in coefficients("P")]
        y = F(x) * F(self.sl2 * F(F(1) / self.c2))
        z = y * y
        r = fma(c[6], z, c[5])
        for i in range(4, -1, -1):
            r = fma(r, z, c[i])
        return fma(r, y, -self.base)

    def exponential(self, x, exp_off=0.0, rcp_off=0.0):
        """exp_off, rcp_off: how far the approximations are off, relative to their values."""
        with np.errstate(over="ignore"):
            e = np.exp2((F(x) * F(self.sl2 * F(F(2) / self.cap))).astype(np.float64)) * (1 + exp_off)
        e = (np.minimum(e, 3e38).astype(F) + F(1)).astype(F)
        r = (1.0 / e.astype(np.float64) * (1 + rcp_off)).astype(F)
        return fma(r, F(-2) * self.c2, self.c2 - self.base)

    def score(self, out):
        """Natural units, the base put back exactly."""
        return (np.asarray(out, np.float64) + float(self.base)) / float(LOG2E)
