"""CPU tests of how a product is cut into tiles, on the library's own arithmetic: the plan of the host and the tile
counts, heights and columns that the kernel takes from the same functions."""
import ctypes
from collections import namedtuple

import numpy as np
import pytest

import int8_mixed_precision_outlier_b200 as L
from int8_mixed_precision_outlier_b200 import _build

PAIRS, L2 = 74, 126 << 20        # a B200: 148 SMs
RING_BYTES, BLOCK = 208 * 1024, 128
INVALID, ALIGNMENT, OK = -1, -2, 0

Plan = namedtuple("Plan", "H nN BT halves quarter b_rows KPB stages tiles drop")


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return L.load_library()


def plan(lib, S, N, K, E=None, gated=False, pairs=PAIRS, l2=L2):
    out = (ctypes.c_int64 * 10)()
    rc = lib.llmint8_product_plan_debug(S, N, K, E or 1, int(E is not None), int(gated), pairs, l2, out)
    assert rc == OK, (S, N, K, E, gated)
    return Plan(*out)


def tiles(lib, rows, most, quarter=8):
    """(tiles, rows of each, columns of the last one's products, quarters that a CTA copies for it)"""
    out = (ctypes.c_int32 * 4)()
    assert lib.llmint8_product_tiles_debug(rows, most, quarter, out) == OK
    return tuple(out)


def some_products(seed, count):
    """Sizes over the whole range that the entry points take: (S, N, K, E or None, gated)."""
    rng = np.random.default_rng(seed)
    log = lambda low, high: int(round(low * (high / low) ** rng.random()))  # noqa: E731
    for i in range(count):
        gated = bool(rng.random() < 0.4)
        N = 32 * log(1, 2000) if gated else log(1, 64000)
        E = None if rng.random() < 0.5 else log(1, 1024)
        K = 16 * log(1, 4096) if i % 2 else 128 * log(1, 512)
        yield log(1, 100000) if i % 10 else log(1, 2 ** 30), N, K, E, gated


def test_plans_fit_their_ring(lib):
    """Every stage fits, there are at least two, and the tiles cover the channels."""
    for S, N, K, E, gated in some_products(0, 4000):
        p = plan(lib, S, N, K, E, gated)
        what = (S, N, K, E, gated, p)
        assert p.stages >= 2 and p.KPB in (1, 2, 4), what
        assert p.stages * p.KPB * (p.H + p.b_rows * p.halves) * BLOCK <= RING_BYTES, what
        assert p.KPB == 1 or K % BLOCK == 0 and p.KPB <= K // BLOCK, what
        assert p.H % (32 if gated else 8) == 0 and 0 < p.H <= 128, what
        assert (p.nN - 1) * 2 * p.H < N <= p.nN * 2 * p.H, what
        assert p.BT % 16 == 0 and 16 <= p.BT <= 256, what
        assert p.halves == 1 or E is None and p.H == 128, what
        assert p.drop == (N * K * (E or 1) > L2), what


def test_copies_hold_every_height_of_a_tile(lib):
    """The quarters that a CTA copies hold its half of the tile's columns and stay inside the room of a k-block, whose
    rows come in swizzle groups of 8."""
    seen = set()
    for S, N, K, E, gated in some_products(1, 600):
        p = plan(lib, S, N, K, E, gated)
        if (p.BT, p.quarter, p.b_rows) in seen:
            continue
        seen.add((p.BT, p.quarter, p.b_rows))
        assert p.quarter % 8 == 0 and p.b_rows % 8 == 0
        for rows in range(1, p.BT + 1):
            count, per, columns, quarters = tiles(lib, rows, p.BT, p.quarter)
            assert count == 1 and rows <= per <= p.BT and rows <= columns <= 256
            assert columns // 2 <= quarters * p.quarter <= p.b_rows, (p, rows)
    assert len(seen) >= 8


def test_plans_count_enough_tiles(lib):
    """The launch is sized by an upper bound of the tiles: no division of the rows over the groups has more."""
    rng = np.random.default_rng(2)
    for S, N, K, E, gated in some_products(3, 400):
        p = plan(lib, S, N, K, E, gated)
        if E is None:
            count = tiles(lib, S, p.BT)[0]
            assert count % p.halves == 0
            assert count // p.halves * p.nN <= p.tiles
            continue
        for sizes in (rng.multinomial(S, np.full(E, 1 / E)), rng.multinomial(S, rng.dirichlet(np.full(E, 0.05)))):
            assert sum(tiles(lib, int(m), p.BT)[0] for m in sizes if m) * p.nN <= p.tiles


@pytest.mark.parametrize("most", range(32, 257, 32))
def test_tiles_cover_their_group(lib, most):
    """Equal to the rounding, none empty, none above `most`, up to the largest group."""
    rng = np.random.default_rng(most)
    ms = np.concatenate([np.arange(1, 3000), rng.integers(1, 2 ** 31 - 256, 500), 2 ** 31 - 256 - np.arange(300),
                         (rng.integers(1, 2 ** 22, 300) * most)[:, None].repeat(3, 1).ravel()
                         + np.tile([-1, 0, 1], 300)])
    for m in ms[ms <= 2 ** 31 - 257].tolist():
        count, per, columns, _ = tiles(lib, m, most)
        assert count == -(-m // most)
        assert per % 16 == 0 and 16 <= per <= most and per * (count - 1) < m <= per * count
        assert m - per * (count - 1) <= columns <= most


def test_columns_are_a_shape_of_the_pair_product(lib):
    """kind::i8 on a CTA pair takes N = 32, 64, ... 256 columns: every height of every tile, the last one's too."""
    for rows in range(1, 257):
        columns = tiles(lib, rows, 256)[2]
        assert columns % 32 == 0 and rows <= columns <= 256, rows
    for S, N, K, E, gated in some_products(4, 600):
        p = plan(lib, S, N, K, E, gated)
        assert p.BT % 32 == 0 and 32 <= p.BT <= 256
        for rows in {S if E is None else max(1, S // E), p.BT + 1, 3 * p.BT - 17}:
            _, per, columns, _ = tiles(lib, rows, p.BT)
            assert per % 32 == 0 and columns % 32 == 0, (p, rows)


def test_halves_have_rows(lib):
    """A tile of two halves is planned only where each half of each tile has rows."""
    cut = 0
    for S in list(range(200, 2600, 7)) + [2 ** 30 + 1, 2 ** 31 - 257]:
        for N in (8192, 13824, 18442):
            p = plan(lib, S, N, 4096)
            if p.halves == 2:
                cut += 1
                count, per, _, _ = tiles(lib, S, p.BT)
                assert count % 2 == 0 and per * (count - 1) < S and p.tiles == count // 2 * p.nN
    assert cut > 50


def test_which_plans_the_tested_shapes_take(lib):
    """Both kinds of tiles, both kinds of stages and both fates of the weights are among the shapes that run on the
    GPU: a change of the plan's constants may not take one of them away unseen."""
    halves = {s: plan(lib, *s[:3], gated=s[3]).halves for s in
              [(257, 13824, 2048, False), (270, 18944, 2064, True), (600, 9001, 4096, False),
               (513, 8192, 4112, True), (1051, 12297, 8064, False), (1213, 18442, 6160, False),
               (150, 40000, 128, False)]}
    assert halves[257, 13824, 2048, False] == 2 and halves[270, 18944, 2064, True] == 2
    assert halves[1051, 12297, 8064, False] == 2 and halves[1213, 18442, 6160, False] == 2
    assert halves[150, 40000, 128, False] == 1
    assert plan(lib, 64, 4096, 512).KPB == 2 and plan(lib, 16, 4096, 4096).KPB == 4 and plan(lib, 33, 257, 272).KPB == 1
    assert plan(lib, 16, 4096, 2048, E=16).drop == 1 and plan(lib, 16, 4096, 2048, E=8).drop == 0


def test_plan_refusals(lib):
    out = (ctypes.c_int64 * 10)()
    f = lambda S=4, N=64, K=64, E=1, grouped=0, gated=0, pairs=74, plan=out: lib.llmint8_product_plan_debug(  # noqa: E731
        S, N, K, E, grouped, gated, pairs, L2, plan)
    assert f() == OK and f(E=3, grouped=1) == OK
    assert f(S=0) == INVALID and f(N=0) == INVALID and f(K=8) == INVALID and f(K=72) == ALIGNMENT
    assert f(S=2 ** 31 - 256) == INVALID and f(N=2 ** 31 - 256) == INVALID and f(gated=1, N=48) == INVALID
    assert f(E=2) == INVALID and f(E=1025, grouped=1) == INVALID and f(pairs=0) == INVALID and f(plan=None) == INVALID
    t = (ctypes.c_int32 * 4)()
    g = lib.llmint8_product_tiles_debug
    assert g(0, 64, 8, t) == INVALID and g(2 ** 31, 64, 8, t) == INVALID and g(5, 24, 8, t) == INVALID
    assert g(5, 512, 8, t) == INVALID and g(5, 64, 0, t) == INVALID and g(5, 64, 8, None) == INVALID
