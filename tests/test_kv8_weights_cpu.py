"""How far the 8-bit verify's weights are off on their way to the tensor cores: P is rounded to f16 and
cut into three e5m2 parts (upper bytes of f16: cut, cut, rounded).  Every f16 value is tried."""
import numpy as np


def parts_of(x):
    """The sum of the three parts of f16 values x >= 0, exact in float64."""
    total = np.zeros(x.shape)
    rest = x.copy()
    for part in range(3):
        bits = rest.view(np.uint16) + np.uint16(0x80 if part == 2 else 0)
        cut = (bits & np.uint16(0xff00)).view(np.float16)
        total += cut.astype(np.float64)
        rest = (rest.astype(np.float64) - cut.astype(np.float64)).astype(np.float16)   # exact
    return total


def test_weights_are_within_the_stated_bound():
    x = np.arange(0, 0x7800 + 1, dtype=np.uint16).view(np.float16)     # 0 .. 2^15
    v = x.astype(np.float64)
    got = parts_of(x)
    step = np.diff(v)
    low = v - np.concatenate([[0], step]) / 2                          # what rounds to x lies in [low, high]
    high = v + np.concatenate([step, [0]]) / 2
    worst = 0.0
    for p in (low, v, high):
        err = np.abs(got - p)
        # (small ones: half a step of e5m2's subnormals, 2^-16, and half of one of f16's, 2^-24)
        assert (err <= 1.1 * 2.0 ** -9 * p + 2.0 ** -17 + 2.0 ** -25).all()
        big = p >= 2.0 ** -5
        worst = max(worst, float((err[big] / p[big]).max() * 2 ** 9))
    assert 1.09 < worst < 1.1                                          # (1.094, just below 1.1426 * 2^e)


def test_the_bound_is_what_the_header_states():
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "include", "vegas.h")) as f:
        text = " ".join(f.read().replace("*", " ").split())
    assert "within 1.1 2^-9 of each" in text
    assert "1.01 2^-28 of the row's largest" in text    # (which is 2^11 or more: 2^-17 + 2^-25 < 1.01 2^-17)
