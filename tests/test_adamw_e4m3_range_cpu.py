"""The 8-bit moments' rule for small elements of a block, in the oracle's own arithmetic."""
import numpy as np
import pytest

from oracle import moe_oracle as O


def _stored(val, bits, rounded):
    scale = np.repeat(np.abs(val).reshape(-1, 256).max(1) / 448.0, 256)
    a = np.where(scale > 0, np.abs(val) / np.where(scale > 0, scale, 1.0), 0.0)
    return np.sign(val) * scale * rounded(np.minimum(a, 448.0), bits)[0]


@pytest.mark.parametrize("S", [100.0, 1.0, 0.1])
@pytest.mark.parametrize("ratio", [1e-4, 1e-5, 1e-6])
def test_no_element_moves_far_beyond_the_rate(S, ratio):
    # Constant gradients: a first moment of at most ceil(x) codes over a root of at least max(1, floor(x)), and
    # at least sqrt(1/2) where the code is 1 and x below it: 2 lr at most, 8% more where the block's largest
    # code, a rounding below 448, falls to 416
    n, lr, betas = 2048, 1e-4, (0.9, 0.999)
    g = np.full(n, S * ratio)
    g[::256] = S
    p, m, r, worst = np.zeros(n), np.zeros(n), np.zeros(n), 0.0
    for t in range(1, 301):
        q, m, v = O.adamw(p, g, m, r * r, t, lr, betas, 1e-8, 0.0)
        worst, p = max(worst, np.abs(q - p).max() / lr), q
        bits = O.rounding_bits(9, t, 0, n)
        m, r = _stored(m, bits & 0xFFFF, O.e4m3_round), _stored(np.sqrt(v), bits >> 16, O.e4m3_round_root)
    assert worst <= 2.0 * 1.08


def test_a_root_keeps_the_smallest_code_unless_it_is_zero():
    a = np.array([0.0, 1e-30, 1e-4, 2.0 ** -9, 2.0 ** -9 * 1.5, 1.0, 448.0])
    for bits in (0, 0x7FFF, 0xFFFF):
        want, room = O.e4m3_round(a, np.full(7, bits))
        got, same = O.e4m3_round_root(a, np.full(7, bits))
        assert got[0] == 0.0 and np.all(got[1:3] == 2.0 ** -9)
        assert np.array_equal(got[3:], want[3:]) and np.array_equal(room, same)
