"""Codes of 8-bit floating point with a scale for each block of 128, against
float64: every value must be the one nearest to F x / amax (16-bit inputs), so
codes are compared exactly; fp32 inputs may differ where F x / amax lies within
2^-22 of a tie.  Scales are one fp32 rounding (2^-24) off."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from f8_cases import BLOCK, FORMAT, IN_TYPE, LARGEST, blocks, nearest, row_blocks, table
from moe_cases import DTYPE, TORCH, group_offsets

pytestmark = pytest.mark.gpu
KIND = {"row": 0, "column": 1, "square": 2}


@pytest.fixture(scope="module")
def tcg():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from blackwell_tensor_core_swizzled_gb300 import build
    build.build()
    import blackwell_tensor_core_swizzled_gb300 as m
    return m


def data(R, C, dtype, seed, pad=0):
    """Rows of very unequal size, a block of zeros, in rows padded with NaN."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((R, C)) * np.exp(2 * rng.standard_normal((R, 1))) * np.exp(rng.standard_normal((1, C)))
    if R > 2 and C > 4:
        x[1, :] = 0
        x[:, C // 2] = 0
        x[2, :4] = [9, 3, -9, 4.5]   # quotients by 3 that are exact ties
    t = torch.from_numpy(x).float().to(TORCH[dtype])
    full = torch.full((R, C + pad), float("nan"), dtype=TORCH[dtype])
    full[:, :C] = t
    return full.cuda(), t.double().numpy()


def index_of(kind, R, C, offsets=None):
    """The scale's place of every element, [R][C] twice."""
    r, c = np.arange(R)[:, None], np.arange(C)[None, :]
    if kind == "row":
        return np.broadcast_to(c // BLOCK, (R, C)), np.broadcast_to(r, (R, C))
    if kind == "column":
        rb = r // BLOCK if offsets is None else row_blocks(offsets, R)[:, None]
        return np.broadcast_to(rb, (R, C)), np.broadcast_to(c, (R, C))
    return np.broadcast_to(r // BLOCK, (R, C)), np.broadcast_to(c // BLOCK, (R, C))


def run(tcg, X, R, C, dtype, kind, fmt, pow2, offsets=None, q_pad=0, s_pad=0):
    G = 1 if offsets is None else len(offsets) - 1
    shape = {"row": (blocks(C), R), "column": (blocks(R) if offsets is None else R // BLOCK + G, C),
             "square": (blocks(R), blocks(C))}[kind]
    Q = torch.full((R, C + q_pad), 0x55, dtype=torch.uint8, device="cuda")
    S = torch.full((shape[0], shape[1] + s_pad), -7.0, device="cuda")
    tcg.f8_quantize(IN_TYPE[fmt], KIND[kind], R, C, DTYPE[dtype], X, X.stride(0), Q, C + q_pad, S, shape[1] + s_pad,
                    pow2=pow2, groups=G, offsets=None if offsets is None else torch.from_numpy(offsets).cuda())
    assert tcg.check() == 0, tcg.last_error_string()
    assert bool((Q[:, C:] == 0x55).all()) and bool((S[:, shape[1]:] == -7.0).all()), "wrote past the rows"
    return Q[:, :C].cpu().numpy(), S[:, :shape[1]].double().cpu().numpy()


def reference(x, kind, fmt, pow2, shape, offsets=None):
    """Scales [blocks...] (-7 where no block is) and the quotients before rounding."""
    R, C = x.shape
    i, j = index_of(kind, R, C, offsets)
    kept = i >= 0
    amax = np.full(shape, -1.0)
    np.maximum.at(amax, (i[kept], j[kept]), np.abs(x[kept]))
    F = LARGEST[fmt]
    if pow2:
        man, e = np.frexp(np.maximum(amax, 0) / F)
        s = 2.0 ** np.where(man == 0.5, e - 1, e)
    else:
        s = amax / F
    s = np.where(amax > 0, s, np.where(amax == 0, 1.0, -7.0))
    top = np.where(amax > 0, amax, 1.0)
    unit = np.zeros(x.shape)
    unit[kept] = x[kept] / s[i[kept], j[kept]] if pow2 else x[kept] * F / top[i[kept], j[kept]]
    return s, unit, kept


def compare(Q, S, x, kind, fmt, pow2, dtype, offsets=None):
    s, unit, kept = reference(x, kind, fmt, pow2, S.shape, offsets)
    assert np.all(np.abs(S - s) <= 2.0 ** -24 * np.abs(s)), np.argwhere(np.abs(S - s) > 2.0 ** -24 * np.abs(s))[:4]
    got = table(fmt)[Q]
    want = nearest(unit, fmt)
    bad = (got != want) & kept
    if dtype == "f32" and not pow2:
        # next to a tie the fp32 quotient (two roundings of 2^-24, and one correction) may land on the other side
        near = np.abs(nearest(unit * (1 + 2.0 ** -22), fmt) - nearest(unit * (1 - 2.0 ** -22), fmt)) > 0
        bad &= ~near
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4], unit[bad][:4])
    assert np.all(Q[~kept] == 0x55), "codes of rows of no group were written"


SIZES = [(1, 1, 0), (1, 128, 0), (5, 4096, 0), (7, 130, 3), (129, 127, 1), (128, 256, 8), (300, 1000, 0), (33, 2056, 0),
         (260, 136, 4)]


@pytest.mark.parametrize("kind", ["row", "column", "square"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("R,C,pad", SIZES)
def test_quantize(tcg, kind, dtype, R, C, pad):
    for fmt in ("e4m3", "e5m2"):
        for pow2 in (False, True):
            X, x = data(R, C, dtype, 1, pad)
            Q, S = run(tcg, X, R, C, dtype, kind, fmt, pow2, q_pad=pad, s_pad=pad)
            compare(Q, S, x, kind, fmt, pow2, dtype)


@pytest.mark.parametrize("sizes,before,after", [([1], 0, 0), ([0, 0, 3], 2, 1), ([130, 0, 1, 127, 128, 129, 300], 5, 9),
                                                ([0, 0], 0, 4), ([7] * 300, 0, 0), ([1] * 1024, 3, 0)])
def test_grouped_columns(tcg, sizes, before, after):
    R, C = sum(sizes) + before + after, 72
    off = group_offsets(sizes, before)
    for dtype, fmt in (("bf16", "e4m3"), ("f32", "e5m2")):
        X, x = data(R, C, dtype, 2)
        Q, S = run(tcg, X, R, C, dtype, "column", fmt, False, offsets=off)
        compare(Q, S, x, "column", fmt, False, dtype, offsets=off)


@pytest.mark.parametrize("kind", ["row", "column", "square"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_extreme_values(tcg, kind, fmt):
    """Infinities, NaN, and magnitudes at both ends of fp32's range."""
    F = LARGEST[fmt]
    for top in (3.0e38, 2.0 ** 100, 2.0 ** -100, F * 2.0 ** -126, F * 2.0 ** -127, 2.0 ** -149):
        x = torch.zeros(8, 16)
        x[2, 3], x[4, 3], x[2, 9] = top, -top / 2, float("nan")
        Q, S = run(tcg, x.cuda(), 8, 16, "f32", kind, fmt, False)
        v = table(fmt)[Q]
        at = index_of(kind, 8, 16)
        s = S[at[0][2, 3], at[1][2, 3]]
        expect = max(top / F, 2.0 ** -126)
        assert abs(s - expect) <= 2.0 ** -24 * expect
        for r, c in ((2, 3), (4, 3)):
            block = S[at[0][r, c], at[1][r, c]]
            want = nearest(np.float64(x[r, c]) / np.float64(block), fmt)
            assert v[r, c] == np.clip(want, -F, F), (top, v[r, c], want)
        assert np.isnan(v[2, 9])
        assert not np.any(v[0])
    x = torch.ones(8, 16)
    x[2, 3], x[2, 4] = float("inf"), float("nan")
    Q, S = run(tcg, x.cuda(), 8, 16, "f32", kind, fmt, True)
    v, at = table(fmt)[Q], index_of(kind, 8, 16)
    same = (at[0] == at[0][2, 3]) & (at[1] == at[1][2, 3])
    assert np.isinf(S[at[0][2, 3], at[1][2, 3]])
    assert np.isnan(v[2, 3]) and np.isnan(v[2, 4])
    same[2, 3] = same[2, 4] = False
    assert not np.any(v[same])


def test_captured_on_a_side_stream(tcg):
    X, x = data(64, 512, "bf16", 3)
    Q = torch.zeros(64, 512, dtype=torch.uint8, device="cuda")
    S = torch.zeros(4, 64, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        tcg.f8_quantize(tcg.IN_E4M3, tcg.F8_ROW, 64, 512, tcg.BF16, X, 512, Q, 512, S, 64)
    X.copy_(X.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    compare(Q.cpu().numpy(), S.double().cpu().numpy(), x[::-1], "row", "e4m3", False, "bf16")


def next_to_ties(fmt, blocks_of, n, seed):
    """fp32 [blocks][n]: a block's largest value, then values up to two steps of
    fp32 beside those whose F x / amax lies half way between two codes."""
    rng = np.random.default_rng(seed)
    man, low, high = (3, -6, 8) if fmt == "e4m3" else (2, -14, 15)
    top = np.float32(1 + rng.random((blocks_of, 1))) * np.float32(2) ** rng.integers(-100, 100, (blocks_of, 1)).astype(np.float32)
    e = rng.integers(low - 1, high, (blocks_of, n))
    step = 2.0 ** (np.maximum(e, low) - man)
    first = np.where(e < low, 0, 1 << man)    # below the smallest normal code the steps are its own
    tie = (first + rng.integers(0, 1 << man, e.shape) + 0.5) * step
    x = (tie * top.astype(np.float64) / LARGEST[fmt]).astype(np.float32)
    x = (x.view(np.int32) + rng.integers(-2, 3, e.shape, dtype=np.int32)).view(np.float32)
    x *= rng.choice(np.float32([-1, 1]), e.shape)
    x[:, :1] = top
    assert np.all(np.abs(x) <= top)
    return x


def exact_code(x, top, fmt):
    """The value of the code nearest to F x / top (ties to even), in whole numbers."""
    man, low = (3, -6) if fmt == "e4m3" else (2, -14)
    q = Fraction(float(abs(x))) * int(LARGEST[fmt]) / Fraction(float(top))
    e = low
    while q >= Fraction(2) ** (e + 1):
        e += 1
    step = Fraction(2) ** (e - man)
    return float(round(q / step) * step) * np.sign(x)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("kind", ["row", "column", "square"])
@pytest.mark.parametrize("n", [128, 101])  # in words, and value by value
def test_fp32_is_rounded_once(tcg, fmt, kind, n):
    """Codes of fp32 values next to ties are the nearest, not the nearest to a rounded F x / amax."""
    if kind == "square":
        x = next_to_ties(fmt, 1, n * n, n).reshape(n, n)
    else:
        x = next_to_ties(fmt, n, 128, n)
        x = x.T.copy() if kind == "column" else x
    R, C = x.shape
    Q, S = run(tcg, torch.from_numpy(x).cuda(), R, C, "f32", kind, fmt, False)
    got = table(fmt)[Q]
    top = np.abs(x).max(axis={"row": 1, "column": 0, "square": (0, 1)}[kind], keepdims=True)
    assert np.all(np.abs(S.reshape(-1) - (top / LARGEST[fmt]).reshape(-1)) <= 2.0 ** -23 * S.reshape(-1))
    want = np.array([exact_code(v, t, fmt) for v, t in zip(x.ravel(), np.broadcast_to(top, x.shape).ravel())]).reshape(x.shape)
    wrong = got != want
    assert not wrong.any(), (int(wrong.sum()), x[wrong][:4], got[wrong][:4], want[wrong][:4])


@pytest.mark.parametrize("sizes,before,after", [([0, 0, 3], 2, 1), ([130, 0, 1, 127, 128, 129, 300], 5, 9), ([1] * 1024, 3, 0)])
@pytest.mark.parametrize("C", [72, 77])  # in words, and value by value
def test_grouped_columns_by_powers_of_two(tcg, sizes, before, after, C):
    R = sum(sizes) + before + after
    off = group_offsets(sizes, before)
    for dtype in ("bf16", "f16", "f32"):
        for fmt in ("e4m3", "e5m2"):
            X, x = data(R, C, dtype, 5)
            Q, S = run(tcg, X, R, C, dtype, "column", fmt, True, offsets=off)
            compare(Q, S, x, "column", fmt, True, dtype, offsets=off)


@pytest.mark.parametrize("kind", ["row", "column", "square"])
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("C", [256, 131])  # in words, and value by value
def test_fp32_full_of_ties(tcg, kind, pow2, C):
    """Small whole numbers, bf16 and f16 values in fp32: their ties go to even.  Their
    quotients are so far off other ties that float64 shows the side."""
    rng = np.random.default_rng(C)
    R = 200
    whole = rng.integers(-8, 9, (R, C)).astype(np.float32)
    some = torch.from_numpy(rng.standard_normal((R, C)) * np.exp2(rng.integers(-9, 2, (R, C))))
    for x in (whole, whole * np.float32(2.0 ** -120), some.bfloat16().float().numpy(), some.half().float().numpy()):
        for fmt in ("e4m3", "e5m2"):
            Q, S = run(tcg, torch.from_numpy(x).cuda(), R, C, "f32", kind, fmt, pow2)
            s, unit, _ = reference(x.astype(np.float64), kind, fmt, pow2, S.shape)
            i, j = index_of(kind, R, C)
            s = np.maximum(s, 2.0 ** -126)
            unit = np.where((s == 2.0 ** -126)[i, j], x.astype(np.float64) / s[i, j], unit)
            assert np.all(np.abs(S - s) <= 2.0 ** -24 * np.abs(s))
            got, want = table(fmt)[Q], nearest(unit, fmt)
            wrong = got != want
            assert not wrong.any(), (int(wrong.sum()), x[wrong][:4], got[wrong][:4], want[wrong][:4], unit[wrong][:4])
