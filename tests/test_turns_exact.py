"""pi_rope_turns against rationals: the nearest 2^-64 of a turn, at every size of frequency."""

import os
import random
import struct

import numpy as np
import pytest

from activation_sparse_predictor_amd import binding as B
from oracle import draft as O

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libpi.so not built")


def near(f, steps):
    return struct.unpack("d", struct.pack("q", struct.unpack("q", struct.pack("d", f))[0] + steps))[0]


def test_to_the_nearest():
    rng = random.Random(3)
    tau = 6.283185307179586
    f = [0.0, 5e-324, 2.0 ** -1022, 2.0 ** -80, 2.0 ** -64, 2.0 ** -62, 1e-18, 1e-4, 1.0, 7.0, 100.0, 999999.7, 2.0 ** 20,
         near(2.0 ** 20, -1), 2.0 ** 19 + 0.5]
    f += [near(tau * k, s) for k in (1, 2, 3, 1000, 166886) for s in (-1, 0, 1)]   # around whole turns
    f += [near(tau * 2.0 ** -65 * k, s) for k in (1, 3, 5) for s in (-1, 0, 1)]    # around halves of a unit
    f += [10000.0 ** (-2 * m / 128) for m in range(64)] + [5e5 ** (-2 * m / 26) for m in range(13)]
    f += [rng.random() * 2.0 ** rng.randint(-90, 20) for _ in range(2000)]
    got = B.pi_rope_turns(np.array(f))
    assert [int(t) for t in got] == [O.turns(x) for x in f]
