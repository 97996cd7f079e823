"""Per-pair stretching by the pair's number (PI_ROPE_YARN_INDEX), on the host."""

import math
import os

import numpy as np
import pytest

from activation_sparse_predictor_amd import binding as B
from activation_sparse_predictor_amd import runtime as R
from oracle import draft as O

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libpi.so not built")


@pytest.mark.parametrize("rot", [2, 26, 64, 128, 256])
@pytest.mark.parametrize("base,factor,trained", [(10000.0, 8.0, 4096.0), (5e5, 32.0, 8192.0), (100.0, 1.0, 4096.0), (1e4, 4.0, 5.0), (10.0, 2.0, 1e9)])
@pytest.mark.parametrize("slow,fast", [(1.0, 32.0), (0.0, 4.0), (2.5, 2.6)])
def test_against_the_oracle(rot, base, factor, trained, slow, fast):
    freqs, gain = B.pi_rope_frequencies(rot, base, B.PI_ROPE_YARN_INDEX, factor, trained, slow, fast)
    want, g = O.frequencies(rot, base, "yarn-index", factor, trained, slow, fast)
    # 2 ulp a power, and three roundings more; a blend of two values of one sign loses nothing
    assert np.allclose(freqs, want, rtol=1e-13, atol=0) and gain == np.float32(g)
    own = base ** (-2.0 * np.arange(rot // 2) / rot)
    assert np.all(freqs <= own * (1 + 1e-13)) and np.all(freqs >= own / factor * (1 - 1e-13))


def test_the_blend():
    """128 dimensions, base 10^4, 4096 tokens: pairs 20.95 and 45.03 turn 32 times and once, so the blend falls from pair 20
    to pair 46: what is left of the own frequency at factor 8 is 1 - 7/8 (m - 20) / 26."""
    freqs, _ = B.pi_rope_frequencies(128, 1e4, B.PI_ROPE_YARN_INDEX, 8.0, 4096.0, 1.0, 32.0)
    own = 1e4 ** (-np.arange(64) / 64)
    for r, at in ((32, 20.95), (1, 45.03)):
        assert 64 * math.log(4096 / (2 * math.pi * r)) / math.log(1e4) == pytest.approx(at, abs=0.01)
    left = freqs / own
    assert np.allclose(left[:21], 1.0) and np.allclose(left[46:], 1 / 8)
    for m in (28, 33, 38):
        assert left[m] == pytest.approx(1 - 7 / 8 * (m - 20) / 26, rel=1e-12)
    assert np.allclose(left[[28, 33, 38]], [0.730769, 0.5625, 0.394231], rtol=0, atol=1e-6)   # 19/26, 9/16, 41/104
    other, _ = B.pi_rope_frequencies(128, 1e4, B.PI_ROPE_YARN, 8.0, 4096.0, 1.0, 32.0)   # by turns: another model's
    assert 2.2 < np.max(freqs / other) < 2.4


@pytest.mark.parametrize("args", [(8, 1e4, 5, 0.5, 4096.0, 1.0, 32.0), (8, 1e4, 5, 2.0, 0.0, 1.0, 32.0), (8, 1e4, 5, 2.0, 4096.0, 32.0, 32.0),
                                  (8, 1e4, 5, 2.0, 4096.0, -1.0, 32.0), (8, 1e4, 6, 2.0, 4096.0, 1.0, 32.0)])
def test_refused(args):
    with pytest.raises(B.PiError) as e:
        B.pi_rope_frequencies(*args)
    assert e.value.status == B.PI_ERR_INVALID_ARG


def test_plan():
    plan = R.rope(128, scaling="yarn-index", factor=8.0, device="cpu")
    freqs, gain = O.frequencies(128, 1e4, "yarn-index", 8.0)
    got = [t % 2 ** 64 / 2.0 ** 64 for t in plan["turns"].tolist()]
    assert np.allclose(got, freqs / (2 * math.pi), rtol=1e-12) and plan["gain"] == pytest.approx(gain)
