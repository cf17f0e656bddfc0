"""GPU tests of the products with token and channel scales, dense and grouped by expert, and of the row quantisation,
expert positions and combine, each against its definition in 64 bits.

Tolerances count the kernels' roundings.  u = 2^-24 is half a step of binary32, eps(t) / 2 half a step of the output
type.  The int32 sums are exact.
  z = fl(fl(fl(acc) sx) sw) [+ b]: at most 3 u |z0| before the bias (second-order terms: 3.1 u), u |z| for the addition;
  gate: with dg, du the errors of its arguments, |silu'| < 1.1; 2^h within 2 ulp (4 u), its correction, 1 + t, the
  reciprocal (1 ulp, 2 u) and two products one rounding each: dy <= 1.1 dg |u| + |silu(g)| du + 10 u |y|;
  the output's own rounding: eps / 2 |y|, or half the smallest subnormal step.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF_SUBNORMAL = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}
TYPES = [torch.float16, torch.bfloat16, torch.float32]


@pytest.fixture(scope="module")
def L():
    import int8_mixed_precision_outlier_b200 as lib
    lib.load_library()
    assert lib.llmint8_sync_status() == 0
    return lib


@pytest.fixture(autouse=True)
def no_fault(L):
    yield
    assert L.llmint8_sync_status() == 0


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def codes(g, *shape):
    return torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8)


def scales(g, mean, *shape):
    return (torch.rand(*shape, generator=g, device="cuda") + 0.5) * mean


def z_of(Xq, sx, Wq, sw, b):
    """z and the bound of its error, in float64 (the integer sums are below 2^53)."""
    z0 = (Xq.double() @ Wq.double().T) * sx.double()[:, None] * sw.double()
    z = z0 if b is None else z0 + b.double()
    return z, 3.1 * U * z0.abs() + (0 if b is None else U * z.abs() * 1.01)


def expected(Xq, sx, Wq, sw, b, gated, dtype):
    z, dz = z_of(Xq, sx, Wq, sw, b)
    y, dy = z, dz
    if gated:
        F = z.shape[1] // 2
        g, u, dg, du = z[:, :F], z[:, F:], dz[:, :F], dz[:, F:]
        s = g * torch.sigmoid(g)
        y = s * u
        dy = 1.1 * dg * u.abs() + s.abs() * du + 10 * U * y.abs()
    return y, dy + torch.finfo(dtype).eps / 2 * y.abs() * (1 + 2.0 ** -8) + HALF_SUBNORMAL[dtype]


def check(Y, y, tol, what=""):
    err = (Y.double() - y).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, first {bad.nonzero()[0].tolist()}, " \
                          f"largest error over its bound {(err / tol).max().item():.3g}"


def fenced(rows, cols, dtype):
    """An output with rows of a known pattern before and after it; returns it and the check of the fences."""
    pad = 64
    whole = torch.full(((rows + 2 * pad) * cols,), 777.0, dtype=dtype, device="cuda")
    inner = whole[pad * cols:(pad + rows) * cols].view(rows, cols)

    def untouched():
        assert (whole[:pad * cols] == 777).all() and (whole[(pad + rows) * cols:] == 777).all()
    return inner, untouched


# ------------------------------------------------------------------ dense product

DENSE = [(1, 8, 16), (1, 1, 16), (3, 100, 144), (16, 1000, 256), (17, 130, 128), (33, 257, 272), (64, 4096, 512),
         (65, 513, 640), (128, 384, 4096), (200, 1000, 1040), (256, 128, 128), (257, 300, 256), (511, 777, 1152),
         (1000, 2000, 512), (2, 19001, 128), (700, 5000, 384)]


@pytest.mark.parametrize("T,N,K", DENSE)
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_scaled_matmul(L, T, N, K, dtype):
    g = gen(T + N + K)
    Xq, Wq = codes(g, T, K), codes(g, N, K)
    sx, sw = scales(g, 0.01, T), scales(g, 0.01 / K ** 0.5, N)
    b = torch.randn(N, generator=g, device="cuda")
    for bias in (None, b):
        Y, untouched = fenced(T, N, dtype) if N % 8 == 0 else (torch.empty(T, N, dtype=dtype, device="cuda"), None)
        assert L.llmint8_scaled_matmul(Xq, sx, Wq, sw, bias=bias, Y=Y) is Y
        check(Y, *expected(Xq, sx, Wq, sw, bias, False, dtype), f"bias {bias is not None}")
        if untouched:
            untouched()


@pytest.mark.parametrize("T,F,K", [(1, 16, 16), (5, 48, 128), (16, 1008, 256), (31, 176, 400), (100, 512, 1024),
                                   (257, 336, 640), (600, 1040, 384)])
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_scaled_matmul_gated(L, T, F, K, dtype):
    g = gen(T + F + K)
    Xq, Wq = codes(g, T, K), codes(g, 2 * F, K)
    sx, sw = scales(g, 0.02, T), scales(g, 0.02 / K ** 0.5, 2 * F)
    b = torch.randn(2 * F, generator=g, device="cuda")
    for bias in (None, b):
        Y, untouched = fenced(T, F, dtype)
        L.llmint8_scaled_matmul(Xq, sx, Wq, sw, bias=bias, gated=True, Y=Y)
        check(Y, *expected(Xq, sx, Wq, sw, bias, True, dtype), f"bias {bias is not None}")
        untouched()


FEW_TILES = [(333, 13824, 144, False), (257, 9999, 256, False), (150, 40000, 128, False), (16, 40008, 1040, False),
              (500, 19968, 272, True), (1111, 8000, 640, False), (47, 64000, 512, True),
              (257, 13824, 2048, False), (270, 18944, 2064, True), (600, 9001, 4096, False), (513, 8192, 4112, True)]


@pytest.mark.parametrize("T,N,K,gated", FEW_TILES)
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_scaled_matmul_of_a_few_tiles_per_sm(L, T, N, K, gated, dtype):
    """One to four tiles for each pair of SMs; tiles of two halves, full and ragged, with and without a K tail."""
    g = gen(T + N)
    Xq, Wq = codes(g, T, K), codes(g, N, K)
    sx, sw = scales(g, 0.01, T), scales(g, 0.001, N)
    b = torch.randn(N, generator=g, device="cuda")
    Y, untouched = fenced(T, N // 2 if gated else N, dtype)
    L.llmint8_scaled_matmul(Xq, sx, Wq, sw, b, gated=gated, Y=Y)
    check(Y, *expected(Xq, sx, Wq, sw, b, gated, dtype))
    untouched()


def test_scaled_matmul_is_exact_on_integers(L):
    """Unit scales, float32 output: the int32 sums themselves, at codes of the largest magnitudes and the largest K
    (sums up to 2^30 round to binary32 once)."""
    for T, N, K, lo in [(7, 40, 1024, -127), (3, 24, 65536, -128), (130, 72, 65536, -128)]:
        g = gen(K + T)
        Xq, Wq = codes(g, T, K), codes(g, N, K)
        Xq[0], Wq[0], Wq[1] = lo, lo, 127
        one = torch.ones(max(T, N), device="cuda")
        Y = L.llmint8_scaled_matmul(Xq, one[:T].contiguous(), Wq, one[:N].contiguous(), dtype=torch.float32)
        want = (Xq.double() @ Wq.double().T).float()
        assert torch.equal(Y, want)


@pytest.mark.parametrize("T,N,K", [(33, 24000, 65520), (300, 4000, 65520), (1, 40000, 16400), (600, 9001, 16384)])
def test_tiles_of_many_laps_of_the_ring(L, T, N, K):
    """Up to 512 stages a tile and several tiles a pair of SMs: every warp goes round the ring of stages with the one
    that moves it on.  Unit scales, the sums themselves."""
    g = gen(K + N)
    Xq, Wq = codes(g, T, K), codes(g, N, K)
    one = torch.ones(max(T, N), device="cuda")
    Y = L.llmint8_scaled_matmul(Xq, one[:T].contiguous(), Wq, one[:N].contiguous(), dtype=torch.float32)
    x = Xq.double()
    for n0 in range(0, N, 4000):
        assert torch.equal(Y[:, n0:n0 + 4000], (x @ Wq[n0:n0 + 4000].double().T).float())


@pytest.mark.parametrize("call", ["scaled", "int32"])
def test_a_call_longer_than_the_wait_limit_is_no_timeout(L, call):
    """The limit bounds each wait: a product of milliseconds whose steps take microseconds runs under a limit of one
    millisecond."""
    g = gen(40)
    T, N, K = 65536, 16384, 4096
    Xq, Wq, one = codes(g, T, K), codes(g, N, K), torch.ones(T, device="cuda")
    sw = one[:N].contiguous()
    run = (lambda: L.llmint8_scaled_matmul(Xq, one, Wq, sw, dtype=torch.float32)) if call == "scaled" else \
        (lambda: L.llmint8_int8_gemm_i32(Xq, Wq))
    want = run()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    L.llmint8_set_wait_limit_ns(1_000_000)
    try:
        begin.record()
        Y = run()
        end.record()
        assert L.llmint8_sync_status() == 0
    finally:
        L.llmint8_set_wait_limit_ns(2_000_000_000)
    assert begin.elapsed_time(end) > 1.5 and torch.equal(Y, want)


def test_scaled_matmul_agrees_with_the_int32_product(L):
    g = gen(5)
    Xq, Wq = codes(g, 190, 1024), codes(g, 320, 1024)
    acc = L.llmint8_int8_gemm_i32(Xq, Wq)
    one = torch.ones(320, device="cuda")
    assert torch.equal(L.llmint8_scaled_matmul(Xq, one[:190].contiguous(), Wq, one, dtype=torch.float32), acc.float())


def test_nan_scale_stays_in_its_row(L):
    g = gen(9)
    Xq, Wq = codes(g, 40, 128), codes(g, 96, 128)
    sx, sw = scales(g, 0.01, 40), scales(g, 0.01, 96)
    sx[17] = float("nan")
    for gated in (False, True):
        Y = L.llmint8_scaled_matmul(Xq, sx, Wq, sw, gated=gated)
        assert Y[17].isnan().all() and not Y[:17].isnan().any() and not Y[18:].isnan().any()


def test_gate_at_large_arguments(L):
    """silu of large arguments of both signs: 0 or the argument, never a NaN."""
    K = 128
    Xq = torch.full((1, K), 127, dtype=torch.int8, device="cuda")
    Wq = torch.full((32, K), 127, dtype=torch.int8, device="cuda")
    Wq[1:16:2] = -127
    one = torch.ones(32, device="cuda")
    Y = L.llmint8_scaled_matmul(Xq, one[:1].contiguous(), Wq, one, gated=True, dtype=torch.float32)[0]
    z = float(K * 127 * 127)
    assert (Y[0::2] == z * z).all() and (Y[1::2] == 0).all()


def test_gate_over_its_whole_range(L):
    """silu at arguments from the smallest to the largest magnitude, infinite and NaN ones: the bound of the gate's
    own roundings, 0 where its value is above -88 * 2^-126, NaN where the formula has it."""
    g = torch.cat([torch.linspace(-90, 90, 20001), torch.logspace(-38, 38, 2001), -torch.logspace(-38, 38, 2001),
                   torch.tensor([0.0, 3.4e38, -3.4e38, float("inf"), float("nan")])]).float().cuda()
    T = g.numel()
    Xq = torch.zeros(T, 16, dtype=torch.int8, device="cuda")
    Xq[:, 0] = 1
    Wq = torch.zeros(32, 16, dtype=torch.int8, device="cuda")
    Wq[:16, 0], sw = 1, torch.ones(32, device="cuda")
    b = torch.cat([torch.zeros(16), torch.full((16,), 3.0)]).cuda()
    Y = L.llmint8_scaled_matmul(Xq, g, Wq, sw, bias=b, gated=True, dtype=torch.float32)[:, 0]
    d = g.double()
    y = 3 * d * torch.sigmoid(d)
    # The reciprocal is flushed where 1 + e^-g > 2^126, that is g < -126 ln 2 = -87.3365; at and below -87.33 the
    # value itself is at most 87.33 e^-87.33 = 87.9 * 2^-126 (|g| e^g falls as g does), flushed or not.
    small = (d < -87.33) & (d.isfinite())
    assert (Y[small].abs() <= 3 * 88 * 2.0 ** -126).all()
    assert Y[-2].isnan() and Y[-1].isnan()      # an infinite scale: the value channel's sum is 0 * inf
    rest = ~small & d.isfinite() & (y.abs() <= 3.4e38)
    check(Y[rest], y[rest], 11 * U * y[rest].abs() + 2.0 ** -126)
    assert (Y[d.isfinite() & (y > 3.41e38)] == float("inf")).all()


@pytest.mark.parametrize("u", [1.0, 2.0 ** 100, -3e38])
def test_gate_where_its_reciprocal_is_subnormal(L, u):
    """silu(g) u for g from -110 to -80, where 1 / (1 + e^-g) leaves binary32's normal range at -87.34 but silu(g) u
    need not: 10 u of the value, and a step of e^g where that is subnormal (2^-149, for its own rounding and the
    correction's, half a step each), times |g u|, half a step of g e^g (2^-150 |u|) and of the output."""
    g = torch.cat([torch.linspace(-110, -80, 30001), torch.linspace(-88, -87, 5001)]).float().cuda()
    Xq = torch.zeros(g.numel(), 16, dtype=torch.int8, device="cuda")
    Xq[:, 0] = 1
    Wq = torch.zeros(32, 16, dtype=torch.int8, device="cuda")
    Wq[:16, 0], one = 1, torch.ones(32, device="cuda")
    b = torch.cat([torch.zeros(16), torch.full((16,), u)]).cuda()
    Y = L.llmint8_scaled_matmul(Xq, g, Wq, one, bias=b, gated=True, dtype=torch.float32)
    d, v = g.double(), float(b[-1])
    y = (v * d * torch.sigmoid(d))[:, None].expand(-1, 16)
    tol = 10 * U * y.abs() + ((d.abs() * 2.0 ** -149 + 2.0 ** -150) * abs(v))[:, None] * (1 + 2.0 ** -20) + 2.0 ** -150
    check(Y, y, tol)
    if abs(v) > 1:
        assert (Y[(d > -95)] != 0).all()


# ------------------------------------------------------------------ grouped product

GROUPS = [([1], 64, 128), ([3, 0, 5], 100, 144), ([0, 0, 7, 0], 40, 16), ([16, 17, 15, 1, 0, 33], 257, 272),
          ([300, 2, 0, 65], 384, 512), ([1] * 50, 72, 256), ([0] * 40 + [513] + [0] * 30 + [40], 200, 384),
          ([128, 256, 257, 511], 1000, 640), ([20] * 8, 2048, 1024), ([2, 1, 0, 1, 3] * 6, 4096, 512)]


@pytest.mark.parametrize("sizes,N,K", GROUPS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_grouped_matmul(L, sizes, N, K, gated, dtype):
    """Ragged and empty groups, rows before the first and behind the last that have to stay as they were."""
    N = (N + 31) // 32 * 32 if gated else N
    g = gen(sum(sizes) + N + K)
    E, lead, tail = len(sizes), 3, 5
    S = lead + sum(sizes) + tail
    bounds = lead + np.concatenate([[0], np.cumsum(sizes)])
    offsets = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    Xq, Wq = codes(g, S, K), codes(g, E, N, K)
    sx, sw = scales(g, 0.02, S), scales(g, 0.02 / K ** 0.5, E, N)
    b = torch.randn(E, N, generator=g, device="cuda")
    No = N // 2 if gated else N
    for bias in (None, b):
        Y = torch.full((S, No), 555.0, dtype=dtype, device="cuda")
        L.llmint8_grouped_matmul(Xq, sx, offsets, Wq, sw, bias=bias, gated=gated, Y=Y)
        assert (Y[:lead] == 555).all() and (Y[S - tail:] == 555).all()
        for e in range(E):
            lo, hi = bounds[e], bounds[e + 1]
            if hi > lo:
                check(Y[lo:hi], *expected(Xq[lo:hi], sx[lo:hi], Wq[e], sw[e], None if bias is None else bias[e], gated,
                                          dtype), f"group {e}")


# ------------------------------------------------------------------ weights beyond L2, tiles of two halves in a row

def plan(L, S, N, K, E=None, gated=False):
    """(halves of a tile, tiles, weights leave L2 first) as the call on this device plans them."""
    import ctypes
    props = torch.cuda.get_device_properties(0)
    out = (ctypes.c_int64 * 10)()
    assert L.load_library().llmint8_product_plan_debug(S, N, K, E or 1, int(E is not None), int(gated),
                                                       props.multi_processor_count // 2, props.L2_cache_size, out) == 0
    return out[3], out[8], out[9]


def just_beyond_l2(K, E=1):
    """The fewest channels, a multiple of 32 and some, with which the weights are more than L2 holds."""
    return (torch.cuda.get_device_properties(0).L2_cache_size // (E * K) // 32 + 1) * 32


@pytest.mark.parametrize("T,K,gated,halves", [(1, 4096, False, 1), (16, 4080, True, 1), (150, 4096, True, 1),
                                              (256, 2736, False, 1), (270, 4096, False, 2), (270, 4080, True, 2),
                                              (300, 8192, False, 2), (600, 4096, False, 1)])
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_scaled_matmul_with_weights_beyond_l2(L, T, K, gated, halves, dtype):
    """Weights that one tile alone reads leave L2 first; calls one after the other, and where several tiles share them."""
    N = just_beyond_l2(K) + (0 if gated else 9)
    planned, _, first_out = plan(L, T, N, K, gated=gated)
    assert planned == halves and first_out == 1
    g = gen(T + N)
    Xq, Wq = codes(g, T, K), codes(g, N, K)
    sx, sw = scales(g, 0.02, T), scales(g, 0.02 / K ** 0.5, N)
    b = torch.randn(N, generator=g, device="cuda")
    y, tol = expected(Xq, sx, Wq, sw, b, gated, dtype)
    for _ in range(2):
        Y = torch.empty(T, N // 2 if gated else N, dtype=dtype, device="cuda")
        L.llmint8_scaled_matmul(Xq, sx, Wq, sw, bias=b, gated=gated, Y=Y)
        check(Y, y, tol)


@pytest.mark.parametrize("K", [2048, 2032])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_grouped_matmul_with_weights_beyond_l2(L, K, gated, dtype):
    """Groups of one tile, whose weights leave L2 first, beside groups of several and empty ones; rows before and
    behind them."""
    sizes = [0, 1, 20, 700, 0, 33, 260, 5, 64, 0, 0, 513, 16, 17, 1, 0]
    E, lead, tail = len(sizes), 2, 7
    N = just_beyond_l2(K, E)
    bounds = lead + np.concatenate([[0], np.cumsum(sizes)])
    S = int(bounds[-1]) + tail
    assert plan(L, S, N, K, E, gated)[2] == 1
    g = gen(K + gated)
    Xq, Wq = codes(g, S, K), codes(g, E, N, K)
    sx, sw = scales(g, 0.02, S), scales(g, 0.02 / K ** 0.5, E, N)
    b = torch.randn(E, N, generator=g, device="cuda")
    offsets = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    Y = torch.full((S, N // 2 if gated else N), 555.0, dtype=dtype, device="cuda")
    L.llmint8_grouped_matmul(Xq, sx, offsets, Wq, sw, bias=b, gated=gated, Y=Y)
    assert (Y[:lead] == 555).all() and (Y[S - tail:] == 555).all()
    for e in range(E):
        lo, hi = bounds[e], bounds[e + 1]
        if hi > lo:
            check(Y[lo:hi], *expected(Xq[lo:hi], sx[lo:hi], Wq[e], sw[e], b[e], gated, dtype), f"group {e}")


@pytest.mark.parametrize("T,N,K,gated", [(1051, 12297, 8064, False), (1051, 12288, 8064, True),
                                         (1500, 18944, 8192, False), (1500, 18944, 8192, True),
                                         (1051, 12297, 8080, False)])
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_tiles_of_two_halves_one_after_the_other(L, T, N, K, gated, dtype):
    """Two and three such tiles a pair: the products wait for both accumulators, and the ring goes on from tile to
    tile."""
    halves, tiles, _ = plan(L, T, N, K, gated=gated)
    assert halves == 2 and tiles > 1.9 * (torch.cuda.get_device_properties(0).multi_processor_count // 2)
    g = gen(T + N)
    Xq, Wq = codes(g, T, K), codes(g, N, K)
    sx, sw = scales(g, 0.02, T), scales(g, 0.02 / K ** 0.5, N)
    b = torch.randn(N, generator=g, device="cuda")
    Y, untouched = fenced(T, N // 2 if gated else N, dtype)
    L.llmint8_scaled_matmul(Xq, sx, Wq, sw, b, gated=gated, Y=Y)
    check(Y, *expected(Xq, sx, Wq, sw, b, gated, dtype))
    untouched()


def test_grouped_matmul_of_one_group_is_the_dense_product(L):
    g = gen(3)
    Xq, Wq = codes(g, 77, 256), codes(g, 320, 256)
    sx, sw = scales(g, 0.01, 77), scales(g, 0.01, 320)
    offsets = torch.tensor([0, 77], dtype=torch.int32, device="cuda")
    assert torch.equal(L.llmint8_grouped_matmul(Xq, sx, offsets, Wq[None], sw[None]),
                       L.llmint8_scaled_matmul(Xq, sx, Wq, sw))


def test_grouped_matmul_of_many_groups(L):
    """The most experts the library takes, few of them with rows."""
    E, N, K = L.MAX_EXPERTS, 24, 64
    g = gen(8)
    sizes = np.zeros(E, int)
    sizes[[0, 31, 32, 500, 1022, 1023]] = [2, 1, 3, 20, 1, 4]
    bounds = np.concatenate([[0], np.cumsum(sizes)])
    Xq, Wq = codes(g, bounds[-1], K), codes(g, E, N, K)
    sx, sw = scales(g, 0.01, int(bounds[-1])), scales(g, 0.01, E, N)
    Y = L.llmint8_grouped_matmul(Xq, sx, torch.tensor(bounds, dtype=torch.int32, device="cuda"), Wq, sw)
    for e in np.nonzero(sizes)[0]:
        lo, hi = bounds[e], bounds[e + 1]
        check(Y[lo:hi], *expected(Xq[lo:hi], sx[lo:hi], Wq[e], sw[e], None, False, torch.float16), f"group {e}")


@pytest.mark.parametrize("bounds", [[0, 5, 3, 9], [-4, 2, 2, 2], [0, 1 << 30, 4, 10], [7, 7, 2, 99], [3, 1, 0, -1]])
def test_wrong_offsets_are_reported_and_stay_inside(L, bounds):
    g = gen(1)
    Xq, Wq = codes(g, 10, 64), codes(g, 3, 40, 64)
    sx, sw = scales(g, 0.01, 10), scales(g, 0.01, 3, 40)
    Y, untouched = fenced(10, 40, torch.float16)
    L.llmint8_grouped_matmul(Xq, sx, torch.tensor(bounds, dtype=torch.int32, device="cuda"), Wq, sw, Y=Y)
    assert L.llmint8_sync_status() == -1 and L.llmint8_sync_status() == 0
    untouched()


# ------------------------------------------------------------------ row quantisation

def quantized(X):
    """The definition: s = fl32(max|x| / 127), code = rint_even(fl32(x / s)), in float64 with those two roundings."""
    x = X.double()
    s = (x.abs().amax(1) / 127).float()
    q = torch.where(s[:, None] > 0, (x / s.double()[:, None]).float().double(), torch.zeros_like(x))
    return q.round().clamp(-127, 127).to(torch.int8), s


def rows(g, T, K, dtype):
    X = torch.randn(T, K, generator=g, device="cuda") * 10 ** (4 * torch.rand(T, 1, generator=g, device="cuda") - 2)
    X[:, torch.randint(0, K, (3,), generator=g, device="cuda")] *= 20
    return X.to(dtype)


@pytest.mark.parametrize("T,K", [(1, 16), (3, 48), (70, 256), (5, 4096), (9, 5120), (4, 8192), (2, 16400), (3, 65536),
                                 (2000, 128)])
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_quantize_rows(L, T, K, dtype):
    X = rows(gen(T + K), T, K, dtype)
    Xq, s = L.llmint8_quantize_rows(X)
    q0, s0 = quantized(X)
    assert torch.equal(s, s0) and torch.equal(Xq, q0)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_quantize_rows_at_its_edges(L, dtype):
    """Zero rows, exact ties, values next to ties, the type's largest and smallest magnitudes, subnormal scales."""
    K = 256
    f = torch.finfo(dtype)
    X = torch.zeros(12, K, device="cuda", dtype=torch.float64)
    half = torch.arange(K, device="cuda", dtype=torch.float64) % 127 + 0.5
    X[1, :], X[1, 0] = half, 127                       # s = 1: ties
    X[2, :], X[2, 0] = -half, 127
    X[3, :], X[3, 0] = half / 64, 127 / 64
    X[4, 5] = f.max
    X[5, :] = f.max
    X[6, 7] = f.smallest_normal
    X[7, 7] = -torch.finfo(dtype).smallest_normal * f.eps   # the smallest subnormal
    X[8, :] = f.smallest_normal * f.eps * (torch.arange(K, device="cuda") % 100)
    X[9, :] = f.smallest_normal * (1 + torch.arange(K, device="cuda") % 130) / 8
    X[10, :] = torch.nextafter(half.float(), torch.full_like(half, 1e9).float()).double()
    X[10, 0] = 127
    X[11, :] = -0.0
    X = X.to(dtype)
    Xq, s = L.llmint8_quantize_rows(X)
    q0, s0 = quantized(X)
    assert torch.equal(s, s0) and torch.equal(Xq, q0)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("K", [64, 16384])
def test_quantize_rows_with_values_that_are_not_finite(L, dtype, K):
    X = rows(gen(K), 6, K, dtype)
    X[1, 3], X[2, K - 1], X[3, 0], X[4, 5], X[4, 6] = float("nan"), float("inf"), float("-inf"), float("nan"), float("inf")
    Xq, s = L.llmint8_quantize_rows(X)
    assert s[1:5].isnan().all() and not Xq[1:5].any()
    q0, s0 = quantized(X[[0, 5]])
    assert torch.equal(s[[0, 5]], s0) and torch.equal(Xq[[0, 5]], q0)


@pytest.mark.parametrize("T,k,K,E", [(1, 1, 16, 1), (40, 2, 128, 4), (33, 8, 400, 16), (300, 3, 5120, 8), (10, 4, 32768, 8)])
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_quantize_rows_to_positions(L, T, k, K, E, dtype):
    g = gen(T * k + K)
    X = rows(g, T, K, dtype)
    ids = torch.randint(-1, E, (T, k), generator=g, device="cuda")
    positions, offsets = L.llmint8_expert_positions(ids, E)
    Xq = torch.full((T * k, K), 99, dtype=torch.int8, device="cuda")
    s = torch.full((T * k,), -3.0, device="cuda")
    L.llmint8_quantize_rows(X, positions, Xq, s)
    q0, s0 = quantized(X)
    at = positions.reshape(-1).long()
    row = torch.arange(T, device="cuda").repeat_interleave(k)[at >= 0]
    at = at[at >= 0]
    assert torch.equal(Xq[at], q0[row]) and torch.equal(s[at], s0[row])
    n = int(offsets[-1])
    assert (Xq[n:] == 99).all() and (s[n:] == -3).all()


def test_positions_outside_are_reported_and_stay_inside(L):
    X = rows(gen(2), 4, 64, torch.float16)
    pos = torch.tensor([[0, 3], [1 << 30, -1], [2, -7], [6, 1]], dtype=torch.int32, device="cuda")
    whole = torch.full((6 + 64, 64), 99, dtype=torch.int8, device="cuda")
    s = torch.full((6,), -3.0, device="cuda")
    L.llmint8_quantize_rows(X, pos, whole[32:38], s)
    assert L.llmint8_sync_status() == -1
    q0, _ = quantized(X)
    assert torch.equal(whole[32:36], q0[[0, 3, 2, 0]])
    assert (whole[:32] == 99).all() and (whole[36:] == 99).all() and (s[4:] == -3).all()
    Y = torch.randn(6, 64, device="cuda")
    out = L.llmint8_expert_combine(Y, pos, torch.ones(4, 2, device="cuda"))
    assert L.llmint8_sync_status() == -1 and L.llmint8_sync_status() == 0
    assert torch.equal(out, torch.stack([Y[0] + Y[3], torch.zeros(64, device="cuda"), Y[2], Y[1]]))


@pytest.mark.parametrize("call", ["scaled", "int32"])
def test_a_recorded_argument_does_not_slow_the_next_calls(L, call):
    """A position outside stays recorded until the status is read; the products in between run as ever.  After a wait
    that ran out each would stay 20 us longer, for copies that may still be landing: 100 calls are 2 ms apart then, and
    a quarter of that is allowed for the clocks."""
    g = gen(12)
    Xq, Wq, one = codes(g, 256, 256), codes(g, 256, 256), torch.ones(256, device="cuda")
    acc = torch.empty(256, 256, dtype=torch.int32, device="cuda")
    Y = torch.empty(256, 256, device="cuda")
    run = (lambda: L.llmint8_scaled_matmul(Xq, one, Wq, one, Y=Y)) if call == "scaled" else \
        (lambda: L.llmint8_int8_gemm_i32(Xq, Wq, acc))
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(100):
            run()

    def ms():
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        times = []
        for _ in range(7):
            begin.record()
            graph.replay()
            end.record()
            torch.cuda.synchronize()
            times.append(begin.elapsed_time(end))
        return sorted(times)[3]
    clear = ms()
    pos = torch.full((1, 1), -9, dtype=torch.int32, device="cuda")
    L.llmint8_expert_combine(torch.ones(1, 8, device="cuda"), pos, torch.ones(1, 1, device="cuda"))
    recorded = ms()
    assert L.llmint8_sync_status() == -1
    assert recorded < clear + 0.5, (clear, recorded)


# ------------------------------------------------------------------ expert positions

@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 8), (7, 3, 5), (512, 2, 8), (1000, 4, 64), (4097, 1, 3),
                                   (9000, 8, 128), (5000, 2, 1024), (40000, 6, 256), (3, 50, 2)])
@pytest.mark.parametrize("itype", [torch.int32, torch.int64], ids=str)
def test_expert_positions(L, T, k, E, itype):
    g = gen(T + k + E)
    ids = torch.randint(-2, E + 2, (T, k), generator=g, device="cuda", dtype=itype)
    if itype == torch.int64:
        ids[0, 0] = (1 << 40) + 1        # only its low half would name an expert
    positions, offsets = L.llmint8_expert_positions(ids, E)
    flat = ids.reshape(-1).cpu().numpy()
    key = np.where((flat >= 0) & (flat < E), flat, E)
    order = np.argsort(key, kind="stable")
    want = np.empty(flat.size, np.int64)
    want[order] = np.where(key[order] < E, np.arange(flat.size), -1)
    assert np.array_equal(positions.reshape(-1).cpu().numpy(), want)
    assert np.array_equal(offsets.cpu().numpy(), np.searchsorted(key[order], np.arange(E + 1)))


def test_expert_positions_of_one_expert_or_none(L):
    ids = torch.zeros(3000, 2, dtype=torch.int64, device="cuda")
    positions, offsets = L.llmint8_expert_positions(ids + 5, 7)
    assert torch.equal(positions.reshape(-1).cpu(), torch.arange(6000, dtype=torch.int32))
    assert offsets.tolist() == [0] * 6 + [6000, 6000]
    positions, offsets = L.llmint8_expert_positions(ids - 1, 7)
    assert (positions == -1).all() and not offsets.any()
    positions, offsets = L.llmint8_expert_positions(ids[:0], 7)
    assert positions.shape == (0, 2) and not offsets.any()


# ------------------------------------------------------------------ combine

@pytest.mark.parametrize("T,k,N", [(1, 1, 1), (5, 2, 64), (33, 8, 1000), (300, 3, 257), (70, 1, 5120), (20, 6, 8)])
@pytest.mark.parametrize("itype", TYPES, ids=str)
@pytest.mark.parametrize("otype", TYPES, ids=str)
def test_expert_combine(L, T, k, N, itype, otype):
    """Sums of k terms in binary32: each product is fused (no rounding of its own), k roundings of partial sums that
    are at most the sum of magnitudes."""
    g = gen(T + k + N)
    Y = torch.randn(T * k, N, generator=g, device="cuda").to(itype)
    w = torch.rand(T, k, generator=g, device="cuda") - 0.3
    ids = torch.randint(-1, 4, (T, k), generator=g, device="cuda")
    ids[0] = -1
    positions, offsets = L.llmint8_expert_positions(ids, 4)
    Y[int(offsets[-1]):] = float("nan")  # rows that no position names
    out = L.llmint8_expert_combine(Y, positions, w, dtype=otype)
    there = positions >= 0
    terms = torch.where(there[:, :, None], Y[positions.clamp(min=0).long()].double() * w[:, :, None].double(), 0.0)
    y = terms.sum(1)
    tol = k * U * 1.01 * terms.abs().sum(1) + torch.finfo(otype).eps / 2 * 1.01 * y.abs() + HALF_SUBNORMAL[otype]
    check(out, y, tol)
    assert not out[0].any()


# ------------------------------------------------------------------ together

def mixture(L, X, ids, weights, W1, W2, positions=None):
    """The experts' layer by its parts: W1 = (codes [E, 2 F, K], scales), W2 = (codes [E, N, F], scales)."""
    positions, offsets = L.llmint8_expert_positions(ids, W1[0].shape[0])
    Xq, sx = L.llmint8_quantize_rows(X, positions)
    H = L.llmint8_grouped_matmul(Xq, sx, offsets, *W1, gated=True, dtype=torch.float32)
    Hq, sh = L.llmint8_quantize_rows(H)
    Y = L.llmint8_grouped_matmul(Hq, sh, offsets, *W2, dtype=torch.float32)
    return L.llmint8_expert_combine(Y, positions, weights, dtype=X.dtype), (Xq, sx, H, Hq, sh, Y, positions, offsets)


@pytest.mark.parametrize("T,k,E,K,F", [(1, 2, 8, 256, 128), (37, 2, 4, 128, 208), (300, 4, 16, 512, 256)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=str)
def test_a_mixture_of_experts(L, T, k, E, K, F, dtype):
    """Router's ids to output: each stage against its definition on the inputs that it got."""
    g = gen(T + K)
    X = torch.randn(T, K, generator=g, device="cuda").to(dtype)
    logits = torch.randn(T, E, generator=g, device="cuda")
    top, ids = logits.topk(k, 1)
    weights = torch.softmax(top, 1)
    if T > 30:
        ids[5:9] = -1
    W1 = (codes(g, E, 2 * F, K), scales(g, 0.02 / K ** 0.5, E, 2 * F))
    W2 = (codes(g, E, K, F), scales(g, 0.02 / F ** 0.5, E, K))
    out, (Xq, sx, H, Hq, sh, Y, positions, offsets) = mixture(L, X, ids, weights, W1, W2)
    bounds = offsets.tolist()
    q0, s0 = quantized(X)
    at = positions.reshape(-1).long()
    row = torch.arange(T, device="cuda").repeat_interleave(k)[at >= 0]
    assert torch.equal(Xq[at[at >= 0]], q0[row]) and torch.equal(sx[at[at >= 0]], s0[row])
    n = bounds[-1]
    for e in range(E):
        lo, hi = bounds[e], bounds[e + 1]
        if hi > lo:
            check(H[lo:hi], *expected(Xq[lo:hi], sx[lo:hi], W1[0][e], W1[1][e], None, True, torch.float32), f"H {e}")
            check(Y[lo:hi], *expected(Hq[lo:hi], sh[lo:hi], W2[0][e], W2[1][e], None, False, torch.float32), f"Y {e}")
    qh, s = quantized(H[:n])
    assert torch.equal(Hq[:n], qh) and torch.equal(sh[:n], s)
    there = positions >= 0
    terms = torch.where(there[:, :, None], Y[positions.clamp(min=0).long()].double() * weights[:, :, None].double(), 0.0)
    y = terms.sum(1)
    check(out, y, k * U * 1.01 * terms.abs().sum(1) + torch.finfo(dtype).eps / 2 * 1.01 * y.abs() + HALF_SUBNORMAL[dtype])


def test_a_mixture_replayed_from_a_graph(L):
    """Captured once, replayed on new inputs in the same buffers, equal to the direct calls bit for bit."""
    g = gen(77)
    T, k, E, K, F = 50, 2, 8, 256, 128
    W1 = (codes(g, E, 2 * F, K), scales(g, 0.02 / K ** 0.5, E, 2 * F))
    W2 = (codes(g, E, K, F), scales(g, 0.02 / F ** 0.5, E, K))
    X = torch.randn(T, K, generator=g, device="cuda").half()
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda")
    w = torch.rand(T, k, generator=g, device="cuda")
    mixture(L, X, ids, w, W1, W2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = mixture(L, X, ids, w, W1, W2)
    for seed in range(3):
        g2 = gen(seed)
        X.copy_(torch.randn(T, K, generator=g2, device="cuda").half())
        ids.copy_(torch.randint(-1, E, (T, k), generator=g2, device="cuda"))
        graph.replay()
        graph.replay()
        direct, _ = mixture(L, X, ids, w, W1, W2)
        assert torch.equal(out, direct)


def test_calls_on_two_streams(L):
    """Two streams at once, with outputs that the calls allocate themselves."""
    g = gen(4)
    Xq, Wq = codes(g, 300, 1024), codes(g, 2048, 1024)
    sx, sw = scales(g, 0.01, 300), scales(g, 0.01, 2048)
    few = Xq[:5].contiguous()
    want, want_few = L.llmint8_scaled_matmul(Xq, sx, Wq, sw), L.llmint8_scaled_matmul(few, sx[:5].contiguous(), Wq, sw)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    sx5 = sx[:5].contiguous()
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        got.append((L.llmint8_scaled_matmul(Xq, sx, Wq, sw, stream=a), want))
        got.append((L.llmint8_scaled_matmul(few, sx5, Wq, sw, stream=b), want_few))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in got)


def test_weights_quantised_by_the_call_before(L):
    """The product after the kernel that writes its weights and the one that writes its activations, repeatedly and
    with the int32 product between: nothing may read the weights before they are there."""
    g = gen(6)
    W = torch.randn(2, 4096, 2048, generator=g, device="cuda").half()
    X = torch.randn(4, 2048, generator=g, device="cuda").half()
    q, s = zip(*(quantized(W[i]) for i in range(2)))
    qx, s_x = quantized(X)
    want = [L.llmint8_scaled_matmul(qx, s_x, q[i], s[i]) for i in range(2)]
    acc = [L.llmint8_int8_gemm_i32(qx, q[i]) for i in range(2)]
    Wq, sw = torch.empty_like(q[0]), torch.empty_like(s[0])
    torch.cuda.synchronize()
    got = []
    for i in (0, 1) * 8:
        L.llmint8_quantize_rows(W[i], Xq=Wq, xscale=sw)
        Xq, sx = L.llmint8_quantize_rows(X)
        got.append((L.llmint8_scaled_matmul(Xq, sx, Wq, sw), want[i]))
        L.llmint8_quantize_rows(W[1 - i], Xq=Wq, xscale=sw)
        got.append((L.llmint8_scaled_matmul(Xq, sx, Wq, sw), want[1 - i]))
        L.llmint8_quantize_rows(W[i], Xq=Wq, xscale=sw)
        Xq, sx = L.llmint8_quantize_rows(X)
        got.append((L.llmint8_int8_gemm_i32(Xq, Wq), acc[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in got)


def test_two_captured_graphs_at_once(L):
    """Two graphs with the same layer in each, replayed on two streams at the same time."""
    g = gen(31)
    T, k, E, K, F = 120, 2, 4, 512, 256
    W1 = (codes(g, E, 2 * F, K), scales(g, 0.02 / K ** 0.5, E, 2 * F))
    W2 = (codes(g, E, K, F), scales(g, 0.02 / F ** 0.5, E, K))
    runs = []
    for _ in range(2):
        X = torch.randn(T, K, generator=g, device="cuda").half()
        ids = torch.randint(0, E, (T, k), generator=g, device="cuda")
        w = torch.rand(T, k, generator=g, device="cuda")
        want, _ = mixture(L, X, ids, w, W1, W2)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out, kept = mixture(L, X, ids, w, W1, W2)
        runs.append((graph, torch.cuda.Stream(), out, want, kept, X, ids, w))
    torch.cuda.synchronize()
    for _ in range(25):
        for graph, stream, *_ in runs:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, _, out, want, *_ in runs:
        assert torch.equal(out, want)


def test_offsets_past_32_bits(L):
    """Outputs, codes and inputs of more than 2^31 elements: the first and the last rows."""
    g = gen(1)
    T, N, K = 140000, 16384, 16
    ends = [0, 1, T // 2, T - 2, T - 1]
    Xq, Wq = codes(g, T, K), codes(g, N, K)
    sx, sw = scales(g, 0.02, T), scales(g, 0.02, N)
    Y = L.llmint8_scaled_matmul(Xq, sx, Wq, sw, dtype=torch.bfloat16)
    check(Y[ends], *expected(Xq[ends], sx[ends], Wq, sw, None, False, torch.bfloat16))
    q, s = L.llmint8_quantize_rows(Y)
    q0, s0 = quantized(Y[ends])
    assert torch.equal(q[ends], q0) and torch.equal(s[ends], s0)
    positions = torch.tensor([[T - 1, 0], [T - 2, T - 1]], dtype=torch.int32, device="cuda")
    out = L.llmint8_expert_combine(Y, positions, torch.ones(2, 2, device="cuda"), dtype=torch.float32)
    rows_ = Y[positions.long()].float()
    assert torch.equal(out, rows_[:, 0] + rows_[:, 1])
    q.zero_()
    at = torch.full((3, 1), T - 1, dtype=torch.int32, device="cuda") - torch.arange(3, dtype=torch.int32, device="cuda")[:, None]
    L.llmint8_quantize_rows(Y[:3].contiguous(), at, q, s)
    assert torch.equal(q[[T - 1, T - 2, T - 3]], quantized(Y[:3])[0]) and not q[: T - 3].any()


def test_more_than_2_30_rows(L):
    """One group of more than 2^30 rows, of which 160 at its start and its end hold something: twice its length and its
    rounded-up parts pass 32 bits."""
    g = gen(2)
    S, N, K = (1 << 30) + 4097, 16, 16
    some = torch.cat([torch.arange(80), torch.arange(S - 80, S)]).cuda()
    Xq = torch.zeros(S, K, dtype=torch.int8, device="cuda")
    Xq[some] = codes(g, 160, K)
    sx = torch.full((S,), 0.5, device="cuda")
    Wq, sw = codes(g, 1, N, K), scales(g, 0.02, 1, N)
    want, tol = expected(Xq[some], sx[some], Wq[0], sw[0], None, False, torch.float16)
    offsets = torch.tensor([0, S], dtype=torch.int32, device="cuda")
    Y = L.llmint8_grouped_matmul(Xq, sx, offsets, Wq, sw)
    check(Y[some], want, tol, "grouped")
    assert not Y[80:S - 80].any()
    Y = None
    check(L.llmint8_scaled_matmul(Xq, sx, Wq[0], sw[0])[some], want, tol, "dense")


def test_refusals(L):
    g = gen(0)
    Xq, Wq = codes(g, 8, 64), codes(g, 32, 64)
    sx, sw = scales(g, 1.0, 8), scales(g, 1.0, 32)
    off = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    f = L.llmint8_scaled_matmul
    for bad, error in [(dict(Xq=Xq.float()), TypeError), (dict(Xq=Xq.T), ValueError), (dict(sx=sx[:7]), ValueError),
                       (dict(sx=sx.half()), TypeError), (dict(Wq=Wq[:, :48].contiguous()), ValueError),
                       (dict(sw=sw[:31]), ValueError), (dict(sw=sw.cpu()), TypeError)]:
        a = {"Xq": Xq, "sx": sx, "Wq": Wq, "sw": sw, **bad}
        with pytest.raises(error):
            f(a["Xq"], a["sx"], a["Wq"], a["sw"])
    for bad, error in [(dict(bias=sw[:5]), ValueError), (dict(bias=sw.half()), TypeError),
                       (dict(dtype=torch.int8), TypeError), (dict(Y=torch.empty(8, 31, device="cuda")), ValueError),
                       (dict(Y=torch.empty(8, 32, device="cuda", dtype=torch.float64)), TypeError),
                       (dict(Y=torch.empty(32, 8, device="cuda").T), ValueError)]:
        with pytest.raises(error):
            f(Xq, sx, Wq, sw, **bad)
    with pytest.raises(ValueError, match="multiple of 16"):
        f(Xq, sx, Wq[:16].contiguous(), sw[:16].contiguous(), gated=True)
    with pytest.raises(L.LLMInt8Error):                  # K not a multiple of 16
        f(Xq[:, :40].contiguous(), sx, Wq[:, :40].contiguous(), sw)
    with pytest.raises(L.LLMInt8Error):                  # a base that is not 16-byte aligned
        f(torch.empty(8 * 64 + 4, dtype=torch.int8, device="cuda")[4:].view(8, 64), sx, Wq, sw)
    h = L.llmint8_grouped_matmul
    for o in (off.long(), off[:1], torch.zeros(3, dtype=torch.int32, device="cuda"), off.cpu()):
        with pytest.raises((TypeError, ValueError)):
            h(Xq, sx, o, Wq[None], sw[None])
    with pytest.raises(ValueError):
        h(Xq, sx, off, Wq, sw)
    X = torch.zeros(8, 64, device="cuda")
    pos = torch.zeros(8, 1, dtype=torch.int32, device="cuda")
    for call in (lambda: L.llmint8_quantize_rows(X.T), lambda: L.llmint8_quantize_rows(X, pos[:7]),
                 lambda: L.llmint8_quantize_rows(X, pos.long()), lambda: L.llmint8_quantize_rows(X, pos[:, :0]),
                 lambda: L.llmint8_quantize_rows(X, xscale=sx[:4].contiguous()),
                 lambda: L.llmint8_expert_positions(pos[:, 0], 4),
                 lambda: L.llmint8_expert_combine(X, pos, torch.ones(8, 2, device="cuda")),
                 lambda: L.llmint8_expert_combine(X, pos.long(), torch.ones(8, 1, device="cuda"))):
        with pytest.raises((TypeError, ValueError)):
            call()
    for experts in (0, L.MAX_EXPERTS + 1):
        with pytest.raises(ValueError):
            L.llmint8_expert_positions(pos, experts)
    torch.cuda.synchronize()


CALLS = {
    "decomposition": "L.llmint8_quantize_weight(torch.ones(8, 64, device='cuda').half())",
    "product": "L.llmint8_scaled_matmul(q, s, q, s)",
    "positions": "L.llmint8_expert_positions(torch.zeros(4, 2, dtype=torch.int32, device='cuda'), 4)",
    "quantize": "L.llmint8_quantize_rows(torch.ones(8, 64, device='cuda'))",
    "combine": "L.llmint8_expert_combine(torch.ones(8, 64, device='cuda'), torch.zeros(4, 2, dtype=torch.int32, "
               "device='cuda'), torch.ones(4, 2, device='cuda'))",
}


@pytest.mark.parametrize("order,parts", [(["decomposition"], 1), (["product"], 2), (["positions"], 4),
                                         (["quantize", "combine"], 0), (["decomposition", "product", "positions"], 7)])
@pytest.mark.parametrize("captured", [False, True])
def test_a_call_makes_its_own_kernels_ready(order, parts, captured):
    """In a process of its own: the kernels of other calls are neither loaded nor set up, and a first call may be one
    that is captured."""
    body = "".join(f"    keep.append({CALLS[c]})\n" for c in order)
    code = ("import torch, contextlib\nimport int8_mixed_precision_outlier_b200 as L\n"
            "q, s, keep = torch.ones(8, 64, dtype=torch.int8, device='cuda'), torch.ones(8, device='cuda'), []\n"
            "torch.cuda.synchronize()\n"
            "graph = torch.cuda.CUDAGraph()\n"
            f"with torch.cuda.graph(graph) if {captured} else contextlib.nullcontext():\n{body}"
            f"if {captured}:\n    graph.replay()\n"
            "assert L.llmint8_sync_status() == 0\n"
            f"assert L.load_library().llmint8_prepared_debug() == {parts}, L.load_library().llmint8_prepared_debug()\n"
            f"if 'product' in {order}:\n"
            f"    assert (keep[{order}.index('product')] == 64).all()\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr


def test_empty_calls(L):
    g = gen(0)
    Wq, sw = codes(g, 32, 64), scales(g, 1.0, 32)
    none = torch.empty(0, 64, dtype=torch.int8, device="cuda")
    assert L.llmint8_scaled_matmul(none, sw[:0].contiguous(), Wq, sw).shape == (0, 32)
    assert L.llmint8_scaled_matmul(Wq, sw, none, sw[:0].contiguous()).shape == (32, 0)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert L.llmint8_grouped_matmul(none, sw[:0].contiguous(), off, Wq.view(2, 16, 64), sw.view(2, 16)).shape == (0, 16)
    Y = torch.full((32, 16), 5.0, device="cuda")         # every group empty: nothing is written
    L.llmint8_grouped_matmul(Wq, sw, off, Wq.view(2, 16, 64), sw.view(2, 16), Y=Y)
    assert (Y == 5).all()
    q, s = L.llmint8_quantize_rows(torch.empty(0, 64, device="cuda"))
    assert q.shape == (0, 64) and s.shape == (0,)
    pos = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    assert L.llmint8_expert_combine(Y, pos, torch.empty(0, 2, device="cuda")).shape == (0, 16)
    pos = torch.full((4, 2), -1, dtype=torch.int32, device="cuda")
    assert not L.llmint8_expert_combine(Y[:0], pos, torch.ones(4, 2, device="cuda")).any()


# ------------------------------------------------------------------ the layer

@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("T,k,E,K,F,N", [(1, 2, 4, 128, 64, 128), (75, 3, 8, 256, 96, 200)])
def test_int8_experts(L, dtype, T, k, E, K, F, N):
    """The layer is the five calls, bit for bit, and near the layer in 64 bits: with codes within half a step of
    everything that is quantised (weights, x, hidden rows), each of the three quantised factors of an output is off by
    at most 1 / 254 of its row's maximum; the bound adds these up by absolute values."""
    g = gen(T + K + F)
    W1 = torch.randn(E, 2 * F, K, generator=g, device="cuda").to(dtype) / K ** 0.5
    W2 = torch.randn(E, N, F, generator=g, device="cuda").to(dtype) / F ** 0.5
    X = torch.randn(T, K, generator=g, device="cuda").to(dtype)
    ids = torch.rand(T, E, generator=g, device="cuda").topk(k, 1).indices
    w = torch.softmax(torch.randn(T, k, generator=g, device="cuda"), 1)
    if T > 1:
        ids[3] = E
    layer = L.Int8Experts(W1, W2)
    assert layer.resident_weight_bytes() == E * (2 * F * K + N * F + 4 * (2 * F + N))
    out = layer(X, ids, w)
    positions, offsets = L.llmint8_expert_positions(ids, E)
    Xq, sx = L.llmint8_quantize_rows(X, positions)
    H = L.llmint8_grouped_matmul(Xq, sx, offsets, layer.W1q, layer.W1scale, gated=True, dtype=torch.float32)
    Hq, sh = L.llmint8_quantize_rows(H)
    Y = L.llmint8_grouped_matmul(Hq, sh, offsets, layer.W2q, layer.W2scale, dtype=dtype)
    assert out.dtype == dtype and torch.equal(out, L.llmint8_expert_combine(Y, positions, w))

    x, step = X.double(), lambda a: a.abs().amax(-1, keepdim=True) / 254 * (1 + 1e-6)  # half a code
    want, tol = torch.zeros(T, N, device="cuda", dtype=torch.float64), torch.zeros(T, N, device="cuda", dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            if e >= E:
                continue
            w1, w2 = W1[e].double(), W2[e].double()
            z = w1 @ x[t]
            dz = step(w1)[:, 0] * (x[t].abs() + step(x[t])).sum() + w1.abs().sum(1) * step(x[t])
            gz, u, dg, du = z[:F], z[F:], dz[:F], dz[F:]
            h = gz * torch.sigmoid(gz) * u
            dh = 1.1 * dg * (u.abs() + du) + (gz * torch.sigmoid(gz)).abs() * du
            dh = dh + (h.abs() + dh).max() / 254 * (1 + 1e-6)
            y = w2 @ h
            dy = w2.abs() @ dh + step(w2)[:, 0] * (h.abs() + dh).sum()
            want[t] += w[t, j].double() * y
            tol[t] += w[t, j].double() * (dy + (y.abs() + dy) * torch.finfo(dtype).eps)
    check(out, want, tol * (1 + 1e-3) + torch.finfo(dtype).eps * (want.abs() + tol) + HALF_SUBNORMAL[dtype])


def test_int8_experts_refusals(L):
    W = torch.zeros(2, 64, 32, device="cuda")
    for W1, W2 in [(W, torch.zeros(2, 32, 64, device="cuda")), (W, torch.zeros(3, 32, 32, device="cuda")), (W[0], W),
                   (torch.zeros(2, 48, 32, device="cuda"), torch.zeros(2, 32, 24, device="cuda")),
                   (torch.zeros(2, 64, 24, device="cuda"), torch.zeros(2, 32, 32, device="cuda"))]:
        with pytest.raises(ValueError):
            L.Int8Experts(W1, W2)
    layer = L.Int8Experts(W, torch.zeros(2, 32, 32, device="cuda"))
    ids, w = torch.zeros(4, 1, dtype=torch.int64, device="cuda"), torch.ones(4, 1, device="cuda")
    with pytest.raises(ValueError):
        layer(torch.zeros(4, 48, device="cuda"), ids, w)
    with pytest.raises(ValueError):
        layer(torch.zeros(5, 32, device="cuda"), ids, w)
    with pytest.raises(TypeError):
        layer(torch.zeros(4, 32, device="cuda"), ids, w.double())


def test_int8_experts_on_a_stream_of_its_own(L):
    g = gen(21)
    layer = L.Int8Experts(torch.randn(4, 256, 512, generator=g, device="cuda"), torch.randn(4, 512, 128, generator=g, device="cuda"))
    X = torch.randn(200, 512, generator=g, device="cuda")
    ids = torch.randint(0, 4, (200, 2), generator=g, device="cuda")
    w = torch.rand(200, 2, generator=g, device="cuda")
    want = layer(X, ids, w)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [layer(X, ids, w, stream=s) for s in streams * 4]
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in got)
