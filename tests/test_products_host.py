"""CPU tests of the products with token and channel scales and of the kernels around them: what the C entry points
refuse before they touch the device, what the Python binding refuses, and restatements in numpy of the kernels' index
arithmetic (group bounds, tiles, expert positions)."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import int8_mixed_precision_outlier_b200 as L
from int8_mixed_precision_outlier_b200 import _build


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return L.load_library()


A = ctypes.c_void_p(0x10000)        # aligned, never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10002)
INVALID, ALIGNMENT, OK = -1, -2, 0


def scaled(lib, Xq=A, sx=A, T=4, K=64, Wq=A, sw=A, bias=None, N=64, gated=0, Y=A, dtype=0):
    return lib.llmint8_scaled_matmul(Xq, sx, T, K, Wq, sw, bias, N, gated, Y, dtype, None)


def grouped(lib, S=4, K=64, offsets=A, E=2, Wq=A, N=64, gated=0, Y=A, dtype=0):
    return lib.llmint8_grouped_matmul(A, A, S, K, offsets, E, Wq, A, None, N, gated, Y, dtype, None)


def test_scaled_matmul_refusals(lib):
    assert scaled(lib, T=-1) == INVALID and scaled(lib, N=-1) == INVALID
    assert scaled(lib, T=1 << 31) == INVALID and scaled(lib, N=1 << 31) == INVALID
    assert scaled(lib, K=8) == INVALID and scaled(lib, K=0) == INVALID and scaled(lib, K=65552) == INVALID
    assert scaled(lib, K=72) == ALIGNMENT
    assert scaled(lib, dtype=3) == INVALID and scaled(lib, dtype=-1) == INVALID
    assert scaled(lib, gated=1, N=48) == INVALID and scaled(lib, gated=1, N=33) == INVALID
    for name in ("Xq", "sx", "Wq", "sw", "Y"):
        assert scaled(lib, **{name: None}) == INVALID, name
        assert scaled(lib, **{name: ODD}) == ALIGNMENT, name
    assert scaled(lib, bias=ODD) == ALIGNMENT
    assert scaled(lib, T=0, Xq=None, sx=None, Y=None) == OK and scaled(lib, N=0, Wq=None, sw=None, Y=None) == OK


def test_products_refuse_sizes_whose_tiles_pass_32_bits(lib):
    """The last tile of the channels ends up to 255 rows past N, the last tile of the tokens 255 past S."""
    last = (1 << 31) - 1
    assert scaled(lib, N=last - 255, K=16) == INVALID and scaled(lib, T=last - 255, K=16) == INVALID
    assert grouped(lib, N=last - 255, K=16) == INVALID and grouped(lib, S=last - 255, K=16) == INVALID


def test_grouped_matmul_refusals(lib):
    assert grouped(lib, E=0) == INVALID and grouped(lib, E=1025) == INVALID
    assert grouped(lib, offsets=None) == INVALID and grouped(lib, offsets=ODD) == ALIGNMENT
    assert grouped(lib, Wq=None) == INVALID and grouped(lib, Y=ODD) == ALIGNMENT
    assert grouped(lib, K=40) == ALIGNMENT and grouped(lib, gated=1, N=16) == INVALID
    assert grouped(lib, S=0, Y=None) == OK


def test_quantize_rows_refusals(lib):
    q = lambda X=A, dtype=0, T=4, K=64, pos=None, copies=0, S=4, Xq=A, sx=A: lib.llmint8_quantize_rows(  # noqa: E731
        X, dtype, T, K, pos, copies, S, Xq, sx, None)
    assert q(T=-1) == INVALID and q(K=8) == INVALID and q(K=65552) == INVALID and q(K=24) == ALIGNMENT
    assert q(dtype=7) == INVALID
    assert q(S=5) == INVALID                       # without positions Xq has X's rows
    assert q(pos=A, copies=0) == INVALID
    assert q(X=None) == INVALID and q(Xq=None) == INVALID and q(sx=None) == INVALID
    assert q(X=ODD) == ALIGNMENT and q(Xq=ODD) == ALIGNMENT and q(sx=ODD) == ALIGNMENT
    assert q(pos=ODD, copies=1) == ALIGNMENT
    assert q(T=0, S=0, X=None) == OK and q(pos=A, copies=2, S=0, Xq=None) == OK


def test_expert_positions_refusals(lib):
    f = lambda ids=A, size=8, T=4, k=2, E=8, pos=A, off=A: lib.llmint8_expert_positions(  # noqa: E731
        ids, size, T, k, E, pos, off, None)
    assert f(T=-1) == INVALID and f(k=0) == INVALID and f(E=0) == INVALID and f(E=1025) == INVALID
    assert f(size=2) == INVALID and f(T=1 << 30, k=2) == INVALID
    assert f(ids=None) == INVALID and f(pos=None) == INVALID and f(off=None) == INVALID
    assert f(ids=ctypes.c_void_p(0x10004)) == ALIGNMENT and f(pos=ODD) == ALIGNMENT and f(off=ODD) == ALIGNMENT


def test_expert_combine_refusals(lib):
    f = lambda Y=A, yd=0, S=8, N=64, pos=A, w=A, T=4, k=2, out=A, od=0: lib.llmint8_expert_combine(  # noqa: E731
        Y, yd, S, N, pos, w, T, k, out, od, None)
    assert f(T=-1) == INVALID and f(k=0) == INVALID and f(S=-1) == INVALID and f(N=-1) == INVALID
    assert f(yd=3) == INVALID and f(od=3) == INVALID
    assert f(Y=None) == INVALID and f(pos=None) == INVALID and f(w=None) == INVALID and f(out=None) == INVALID
    assert f(Y=ODD) == ALIGNMENT and f(out=ODD) == ALIGNMENT and f(pos=ODD) == ALIGNMENT and f(w=ODD) == ALIGNMENT
    assert f(T=0, pos=None, w=None, out=None) == OK and f(N=0, out=None) == OK


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 64)
    q, s = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
    off = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError, match="CUDA"):
        L.llmint8_quantize_rows(x)
    with pytest.raises(TypeError, match="CUDA"):
        L.llmint8_scaled_matmul(q, s, q, s)
    with pytest.raises(TypeError, match="CUDA"):
        L.llmint8_grouped_matmul(q, s, off, q[None], s[None])
    with pytest.raises(TypeError, match="CUDA"):
        L.llmint8_grouped_matmul(q, s, None, q[None], s[None])
    with pytest.raises(TypeError, match="CUDA"):
        L.llmint8_expert_positions(off[:2, None], 4)
    with pytest.raises(TypeError, match="CUDA"):
        L.llmint8_expert_combine(x, off[:, None], s[:3, None])
    with pytest.raises(TypeError, match="float16, bfloat16 or float32"):
        L.llmint8_quantize_rows(x.double())
    with pytest.raises(TypeError, match="int32 or int64"):
        L.llmint8_expert_positions(torch.zeros(2, 2), 4)


def test_import_on_a_torch_without_cuda():
    """Such a build has none of torch._C's CUDA functions: the package is imported, and what needs no GPU works."""
    code = ("import torch\n"
            "for name in [n for n in dir(torch._C) if n.startswith('_cuda_')]:\n"
            "    delattr(torch._C, name)\n"
            "import int8_mixed_precision_outlier_b200 as L\n"
            "assert 'llmint8_scaled_matmul' in L.header_functions()\n"
            "try:\n"
            "    L.llmint8_quantize_rows(torch.zeros(4, 64))\n"
            "except TypeError as e:\n"
            "    print('refused:', e)\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "refused: X must be a CUDA tensor" in r.stdout, r.stderr


def test_int8_experts_refuses_at_construction():
    """Shapes that no call could use are refused before anything is quantised."""
    for E in (0, 1025):
        with pytest.raises(ValueError, match="experts"):
            L.Int8Experts(torch.zeros(E, 32, 16), torch.zeros(E, 16, 16))
    for w1, w2 in [((2, 32, 24), (2, 16, 16)), ((2, 24, 16), (2, 16, 12))]:
        with pytest.raises(ValueError, match="multiples of 16"):
            L.Int8Experts(torch.zeros(w1), torch.zeros(w2))
    with pytest.raises(ValueError, match="W1 must be"):
        L.Int8Experts(torch.zeros(2, 32, 16), torch.zeros(3, 16, 16))


# ------------------------------------------------------------------ index arithmetic, restated

def scan_groups(offsets, S, BT, nN):
    """The bounds as the kernel clamps them, the cumulative tile counts, whether a bound was wrong."""
    off, cum, bad = [], [0], False
    prev = 0
    for i, o in enumerate(offsets):
        v = max(min(max(o, 0), S), prev)
        bad |= v != o
        off.append(v)
        if i:
            cum.append(cum[-1] + -(-(v - prev) // BT) * nN)
        prev = v
    return off, cum, bad


def token_tiles(m, BT):
    """ceil(m / BT) by a multiplication, as the kernel takes it."""
    shift = 31 + (BT - 1).bit_length()
    product = (m + BT - 1) * ((1 << shift) // BT + 1)
    assert product < 1 << 64
    return product >> shift


def tile_rows(m, mt, BT):
    if mt <= 1:
        return (m + 15) // 16 * 16
    share = int(np.float32(m) / np.float32(mt)) + 1
    per = min((share + 15) // 16 * 16, BT)
    return per + 16 if per * mt < m else per


@pytest.mark.parametrize("BT", range(16, 257, 16))
def test_tile_arithmetic(BT):
    """The quotient without a division is exact up to the largest m, and the tiles of a group cover it: equal to the
    rounding, none empty, none above BT."""
    rng = np.random.default_rng(BT)
    ms = np.concatenate([np.arange(1, 5000), rng.integers(1, 2 ** 31 - 256, 2000),
                         2 ** 31 - 256 - np.arange(600), (rng.integers(1, 2 ** 22, 500) * BT)[:, None].repeat(3, 1).ravel()
                         + np.tile([-1, 0, 1], 500)])
    for m in ms[ms <= 2 ** 31 - 256].tolist():
        mt = token_tiles(m, BT)
        assert mt == -(-m // BT)
        per = tile_rows(m, mt, BT)
        assert per % 16 == 0 and 16 <= per <= BT and per * mt >= m and per * (mt - 1) < m


def find_tile(off, cum, BT, w):
    E = len(cum) - 1
    block = sum((i + 1) * 32 < E and cum[min((i + 1) * 32, E)] <= w for i in range(32))
    lo = block * 32 + sum(block * 32 + i + 1 < E and cum[min(block * 32 + i + 1, E)] <= w for i in range(32))
    assert cum[lo] <= w < cum[lo + 1]
    begin, m = off[lo], off[lo + 1] - off[lo]
    mt = -(-m // BT)
    assert mt == token_tiles(m, BT)
    per = tile_rows(m, mt, BT)
    r = w - cum[lo]
    nt, i = r // mt, r % mt
    return lo, begin + i * per, min(per, m - i * per), nt


@pytest.mark.parametrize("BT", [16, 32, 48, 64, 128, 192, 256])
def test_tiles_cover_every_row_once(BT):
    rng = np.random.default_rng(BT)
    for trial in range(40):
        E = int(rng.choice([1, 2, 31, 32, 33, 64, 65, 70, 1024])) if trial % 4 == 0 else int(rng.integers(1, 70))
        sizes = rng.integers(0, rng.choice([2, 18, 300, 1100]), E) * (rng.random(E) < 0.7)
        lead, tail = int(rng.integers(0, 3)), int(rng.integers(0, 5))
        offsets = (lead + np.concatenate([[0], np.cumsum(sizes)])).tolist()
        S, nN = offsets[-1] + tail, int(rng.integers(1, 4))
        off, cum, bad = scan_groups(offsets, S, BT, nN)
        assert not bad and off == offsets
        seen = np.zeros((S, nN), int)
        for w in range(cum[-1]):
            e, m0, tok, nt = find_tile(off, cum, BT, w)
            assert 1 <= tok <= BT and off[e] <= m0 and m0 + tok <= off[e + 1] and 0 <= nt < nN
            seen[m0:m0 + tok, nt] += 1
        assert (seen[offsets[0]:offsets[-1]] == 1).all()
        assert not seen[:offsets[0]].any() and not seen[offsets[-1]:].any()


def test_tiles_of_two_halves_cover_every_row_once():
    """Where every half has rows (the others are not cut this way); the kernel finds the tile i // 2 and its halves."""
    cut = 0
    for S in list(range(257, 3000)) + [2 ** 31 - 257, 2 ** 30 + 1]:
        wide = (S + 511) // 512
        half = -(-S // (2 * wide)) + 15 & ~15
        assert half <= 256
        if (2 * wide - 1) * half >= S:
            continue
        cut += 1
        mt = token_tiles(S, half)
        per = tile_rows(S, mt, half)
        assert mt == 2 * wide and per <= half and per * mt >= S and per * (mt - 1) < S
    assert cut > 2000


@pytest.mark.parametrize("offsets", [[0, 5, 3, 9], [-4, 2, 2, 2], [0, 1 << 30, 4, 10], [7, 7, 2, 99], [3, 1, 0, -1]])
def test_wrong_bounds_stay_inside(offsets):
    S = 10
    off, cum, bad = scan_groups(offsets, S, 16, 2)
    assert bad and all(0 <= a <= b <= S for a, b in zip(off, off[1:]))
    for w in range(cum[-1]):
        _, m0, tok, _ = find_tile(off, cum, 16, w)
        assert 0 <= m0 and tok >= 1 and m0 + tok <= S


@pytest.mark.parametrize("S,E,ctas", [(1, 1, 1), (31, 3, 1), (1000, 7, 1), (5000, 64, 2), (40000, 300, 8), (0, 5, 1)])
def test_positions_by_parts_are_a_stable_sort(S, E, ctas):
    """Counts per run of choices, prefix sums over runs and experts, then positions in order: as the kernel does."""
    rng = np.random.default_rng(S + E)
    ids = rng.integers(-1, E + 1, S)
    warps = ctas * 32
    per = -(-(-(-S // warps)) // 32) * 32
    runs = [ids[w * per:(w + 1) * per] for w in range(warps)]
    assert sum(len(r) for r in runs) == S
    cnt = np.array([np.bincount(r[(r >= 0) & (r < E)], minlength=E) for r in runs])
    total = cnt.sum(0)
    first = np.cumsum(total) - total
    at = first + np.cumsum(cnt, 0) - cnt
    pos = []
    for w, r in enumerate(runs):
        for v in r:
            if 0 <= v < E:
                pos.append(at[w][v])
                at[w][v] += 1
            else:
                pos.append(-1)
    key = np.where((ids >= 0) & (ids < E), ids, E)
    order = np.argsort(key, kind="stable")
    want = np.empty(S, int)
    want[order] = np.where(key[order] < E, np.arange(S), -1)
    assert np.array_equal(np.array(pos, int), want)
