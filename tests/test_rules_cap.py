"""The error of a capped score that include/rx.h states, on the CPU: the kernels'
forms in fp32, an operation at a time, against cap tanh(s / cap) in 64 bits."""
import numpy as np
import pytest

from tests._cap import F, Cap, coefficients

# The special-function units: 2^x off by at most 2^-22 of its value, 1/x by 2^-23 (the PTX documentation).
EXP, RCP = 2.0 ** -22, 2.0 ** -23
CAPS = [1e-3, 0.7, 1.0, 5.0, 20.0, 30.0, 40.0, 50.0, 51.0, 80.0, 1e3, 1e6]


def test_the_fits():
    """What the comments beside the coefficients say."""
    for name, top, off in (("P", 1.0, 2.6e-8), ("Q", 0.375, 1.1e-8)):
        y = np.linspace(0, top, 200001)
        c = [float(F(x)) if name == "P" else x for x in coefficients(name)]    # Q is held in 64 bits
        worst = np.abs(y * sum(k * (y * y) ** i for i, k in enumerate(c)) - np.tanh(y)).max()
        assert 0.9 * off < worst <= off


@pytest.mark.parametrize("scale", [0.125, 128 ** -0.5, 3.0])
@pytest.mark.parametrize("slopes", [False, True])     # with slopes there is no fixed base
@pytest.mark.parametrize("cap", CAPS)
def test_forms_stay_within_the_stated_error(cap, slopes, scale):
    c = Cap(cap, scale, False if slopes else None)
    assert c.fixed == (cap <= 50.0 and not slopes)
    for form, top in ((c.near, 0.375), (c.poly, 1.0)):
        if form == c.near and not c.near_in_range():
            continue
        x = (np.linspace(-top, top, 40001) * cap / c.scale).astype(F)
        t = c.true(x)
        assert (np.abs(c.score(form(x)) - t) <= 2.0 ** -21 * np.abs(t) + 2.0 ** -24 * cap).all()
    x = (np.concatenate([np.linspace(-4, 4, 40001), np.geomspace(4, 1e4, 999), -np.geomspace(4, 1e4, 999)]) * cap / c.scale).astype(F)
    for s in (-1, 1):
        assert np.abs(c.score(c.exponential(x, s * EXP, s * RCP)) - c.true(x)).max() <= 5 * 2.0 ** -23 * cap


def test_the_fixed_base_keeps_weights_in_range():
    """2^-100 to 2^45 for every cap that has one."""
    for cap in np.linspace(1e-3, 50.0, 400):
        c = Cap(cap)
        if c.fixed:
            assert -float(c.c2) - float(c.base) >= -100.0 and float(c.c2) - float(c.base) <= 45.0
