"""The split of drafted rows' attention over workgroups (att_plan in attend.hpp): a model of its rule in
fp32, with the kernels' own att_piece and slots, never asks for more slots than the workspace has."""

from __future__ import annotations

import numpy as np
import pytest

from tests.test_kv_plan import host_program

F = np.float32


@pytest.fixture(scope="module")
def slots(tmp_path_factory):
    return int(host_program(tmp_path_factory.mktemp("plan"), 'printf("%d\\n", kAttSlots);')[0])


def piece(want, least):
    return least if want < F(least) else int(want) + 1 if want < F(16777216) else 16777216


def pieces(rt, tiles, c):
    return rt * -(-tiles // c)


def choose(rt, tiles, n_kv, target, at_once, least, slots):
    """C, for items rt of each sequence's tiles (single kernel of few items: at_once 0)."""
    room = F(target) / F(n_kv)
    total = F(np.sum(rt.astype(F) * tiles.astype(F), dtype=F))
    c = piece(total / room * F(1.001), least)
    once = F(at_once) / F(n_kv) if at_once else room
    if len(rt) > 64 or rt.sum() > once:
        return c

    def fit(c, most):
        for _ in range(24):
            if F(pieces(rt, tiles, c).sum()) <= most:
                break
            c += c // 16 + 1
        return c

    wish = total / once * F(1.001)
    c = fit(piece(wish, least), once)
    if at_once and F(c) > F(1.5) * wish and c > 32:
        twice = min(F(2) * once, F(slots) / F(n_kv))
        shorter = fit(piece(F(0.5) * wish, least), twice)
        if 2 * (shorter + 8) < c + 8:
            c = shorter
    return c


# (workgroups of the work, of the chip, rows an item, least tiles): prompt.hip by head width, attend.hip by waves
KERNELS = [(512, 768, 128, 8), (512, 512, 128, 8), (256, 256, 64, 8), (512, 0, 16, 4), (256, 0, 16, 4)]


@pytest.mark.parametrize("target,at_once,rows,least", KERNELS)
def test_slots_suffice(slots, target, at_once, rows, least):
    """Random batches, and alike ones around the places where one turn of pieces becomes two."""
    rng = np.random.default_rng(target + at_once + rows)
    most = turns = 0
    for i in range(20000):
        n_kv = int(rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 8, 12, 16, 28, 40, 56, 71, 128, 1024]))
        n_seq = int(rng.choice([rng.integers(1, 13), rng.integers(1, 65), rng.integers(1, 65), rng.integers(60, 200)]))
        group = int(rng.choice([1, 2, 3, 8, 16, 64, 71]))
        n = rng.integers(1, 257) if rng.random() < 0.4 else rng.integers(0, 257, n_seq)
        n = np.broadcast_to(np.asarray(n), (n_seq,))
        ctx = np.exp(rng.uniform(0, np.log(rng.choice([64, 4096, 131072, 2 ** 24])), n_seq)).astype(np.int64)
        if rng.random() < 0.5:
            ctx[:] = ctx[0] - (rng.integers(0, 65, n_seq) if rng.random() < 0.5 else 0)
        ctx = np.maximum(ctx, 0)
        rt = -(-n * group // rows)
        tiles = np.maximum(-(-ctx // 64) + np.minimum(-(-n // 64), 4), 1)
        if rt.sum() == 0:
            continue
        c = choose(rt, tiles, n_kv, target, at_once, least, slots)
        ns = -(-tiles // c)
        held = int((rt * ns)[ns > 1].sum()) * n_kv
        most = max(most, held)
        turns += at_once > 0 and int((rt * ns).sum()) * n_kv > at_once >= int(rt.sum()) * n_kv
        assert held <= slots, (i, held, n_kv, rt.tolist(), tiles.tolist(), c)
    assert most > slots // 4 and (turns > 0 or not at_once or 2 * at_once > 1.4 * slots)
