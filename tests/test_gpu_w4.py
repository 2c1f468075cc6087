"""Few rows against 4-bit matrices against float64.

Tolerance: a term is activation x code value (exact in fp32) x scale; sums of K
terms, the scale, the groups' sums and alpha make at most K + 8 roundings of
2^-23 relative to the sum of magnitudes."""
import numpy as np
import pytest
import torch

from moe_cases import DTYPE, E2M1, IN_TYPE, TORCH, close, group_offsets, rows, to_host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tcg():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from blackwell_tensor_core_swizzled_gb300 import build
    build.build()
    import blackwell_tensor_core_swizzled_gb300 as m
    return m


def _ok(tcg):
    rc = tcg.check()
    assert rc == 0, tcg.last_error_string()


def ue4m3(b):
    e, m = b >> 3, b & 7
    return np.where(b >= 0x7F, np.nan, np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e.astype(int) - 7)))


def matrices(fmt, G, N, K, group, zeros, dtype, seed, pad_b=0, pad_s=0):
    """Device codes, scales, zero points (padded rows hold other codes) and the
    decoded float64 matrices."""
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 16, size=(G, N, K + pad_b))
    packed = (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)
    nb = K // group
    zero = None
    if fmt == "int4":
        st = torch.from_numpy(rng.uniform(0.01, 0.1, size=(G, N, nb + pad_s))).float().to(TORCH[dtype])
        s = st.double().numpy()
        z = rng.integers(0, 16, size=(G, N, nb + pad_s)).astype(np.uint8)
        zero = torch.from_numpy(z).cuda() if zeros else None
        zv = z[..., :nb].astype(np.float64) if zeros else np.full((G, N, nb), 8.0)
        val = codes[..., :K] - np.repeat(zv, group, axis=2)
    else:
        lo, hi = (120, 130) if fmt == "mxf4" else (0x01, 0x60)
        sb = rng.integers(lo, hi, size=(G, N, nb + pad_s)).astype(np.uint8)
        st = torch.from_numpy(sb)
        s = 2.0 ** (sb.astype(float) - 127) if fmt == "mxf4" else ue4m3(sb)
        val = E2M1[codes[..., :K]]
    w = val * np.repeat(s[..., :nb], group, axis=2)
    return torch.from_numpy(packed).cuda(), st.cuda(), zero, w


def run(tcg, fmt, dtype, out, a_dev, K, N, off, group, B, scale, zero, G, alpha=None, pad_b=0, pad_s=0, ldd=None):
    R = a_dev.shape[0]
    ldd = ldd or N
    D = torch.full((max(R, 1), ldd), 7.0, dtype=TORCH[out], device="cuda")
    tcg.gemv_w4({"int4": 0, "mxf4": 1, "nvf4": 2}[fmt], IN_TYPE[dtype], R, N, K, a_dev, a_dev.shape[1], B, scale, D,
                DTYPE[out], ldd, group=group, zero=zero, groups=G, offsets=off, alpha=alpha, ldb=K + pad_b,
                ld_scale=(K // group + pad_s))
    _ok(tcg)
    assert bool((D[:, N:] == 7.0).all()), "wrote past the row"
    return to_host(D)[:, :N]


FORMATS = [("int4", 32, False), ("int4", 64, True), ("int4", 128, True), ("int4", 128, False), ("mxf4", 32, False),
           ("nvf4", 16, False)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
@pytest.mark.parametrize("R,N,K,pad_b,pad_s", [
    (1, 1, 128, 0, 0), (1, 1000, 256, 0, 1), (2, 129, 384, 32, 0), (3, 1001, 1152, 0, 0), (5, 64, 4096, 64, 3),
    (8, 48, 8192, 0, 0), (9, 100, 640, 0, 0), (16, 257, 2048, 0, 0), (17, 33, 4224, 0, 0), (32, 80, 8192, 0, 0),
    (45, 30, 1024, 0, 0), (1, 20, 16640, 0, 0)])
def test_dense(tcg, dtype, fmt, group, zeros, R, N, K, pad_b, pad_s):
    A, a = rows((R, K), dtype, R + N, 8)
    B, scale, zero, w = matrices(fmt, 1, N, K, group, zeros, dtype, N + K, pad_b, pad_s)
    ref, S = a @ w[0].T, np.abs(a) @ np.abs(w[0].T)
    for out in (dtype, "f32"):
        got = run(tcg, fmt, dtype, out, A, K, N, None, group, B, scale, zero, 1, None, pad_b, pad_s, N + 3)
        close(got, ref, S, (K + 8) * 2.0 ** -23, out)


@pytest.mark.parametrize("fmt,group,zeros", [("mxf4", 32, False), ("int4", 32, True)])
def test_shortest_contraction(tcg, fmt, group, zeros):
    A, a = rows((4, 32), "f16", 1, 8)
    B, scale, zero, w = matrices(fmt, 1, 19, 32, group, zeros, "f16", 3)
    got = run(tcg, fmt, "f16", "f32", A, 32, 19, None, group, B, scale, zero, 1)
    close(got, a @ w[0].T, np.abs(a) @ np.abs(w[0].T), 40 * 2.0 ** -23, "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
@pytest.mark.parametrize("sizes,before,after,N,K", [
    ([1, 0, 2, 0, 0, 1, 3], 0, 0, 72, 256), ([8, 9, 17, 0, 33], 0, 0, 40, 1152), ([0, 0], 0, 3, 16, 128),
    ([2, 1, 1], 2, 1, 1000, 512), ([1] * 50, 0, 0, 100, 384), ([0, 4], 0, 0, 300, 4096)])
def test_groups(tcg, dtype, fmt, group, zeros, sizes, before, after, N, K):
    G, R = len(sizes), sum(sizes) + before + after
    off = group_offsets(sizes, before)
    A, a = rows((R, K), dtype, 5, 8)
    B, scale, zero, w = matrices(fmt, G, N, K, group, zeros, dtype, 6)
    alpha = np.random.default_rng(7).uniform(0.5, 2, G).astype(np.float32)
    ref, S = np.zeros((R, N)), np.zeros((R, N))
    for g in range(G):
        sl = slice(off[g], off[g + 1])
        ref[sl], S[sl] = alpha[g] * (a[sl] @ w[g].T), alpha[g] * (np.abs(a[sl]) @ np.abs(w[g].T))
    got = run(tcg, fmt, dtype, "f32", A, K, N, torch.from_numpy(off).cuda(), group, B, scale, zero, G,
              torch.from_numpy(alpha).cuda())
    close(got, ref, S, (K + 8) * 2.0 ** -23, "f32")


def test_every_code_and_scale(tcg):
    """One-hot activations read single weights back: every code under every
    scale byte (e8m0 255 and E4M3 0x7F and above are NaN)."""
    K = 32
    A = torch.eye(K, dtype=torch.bfloat16, device="cuda")[:16].contiguous()
    for fmt, group, bits in (("mxf4", 32, 256), ("nvf4", 16, 256)):
        codes = np.tile(np.arange(K) % 16, (bits, 1))
        B = torch.from_numpy((codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)).cuda()
        sb = np.repeat(np.arange(bits)[:, None], K // group, axis=1).astype(np.uint8)
        if fmt == "mxf4":
            s = np.where(sb == 255, np.nan, 2.0 ** (sb.astype(float) - 127))
        else:
            s = ue4m3(sb.astype(int))
        got = run(tcg, fmt, "bf16", "f32", A, K, bits, None, group, B, torch.from_numpy(sb).cuda(), None, 1)
        want = (E2M1[codes] * np.repeat(s, group, axis=1))[:, :16].T
        with np.errstate(over="ignore"):
            want = want.astype(np.float32).astype(np.float64)
        assert np.array_equal(np.isnan(got), np.isnan(want)), fmt
        fine = ~np.isnan(want) & (np.abs(want) >= 2.0 ** -126)
        assert np.array_equal(got[fine], want[fine]), fmt


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_wide_range_of_activations(tcg, dtype):
    """Activations over the type's whole range: each 128 of K spans up to 2^20,
    and the rows' magnitudes reach the type's ends."""
    K, N, R = 1024, 40, 6
    rng = np.random.default_rng(8)
    top = {"bf16": [2.0 ** 100, 2.0 ** -100, 1.0, 2.0 ** 60, 2.0 ** -60, 2.0 ** -30],
           "f16": [2.0 ** 15, 2.0 ** -8, 1.0, 2.0 ** 4, 2.0 ** -4, 2.0 ** 10]}[dtype]
    span = 20 if dtype == "bf16" else 6
    x = rng.standard_normal((R, K)) * np.array(top)[:, None] * 2.0 ** -rng.integers(0, span, (R, K))
    x = np.clip(x, -6e4, 6e4) if dtype == "f16" else x
    A = torch.from_numpy(x).float().to(TORCH[dtype])
    a = A.double().numpy()
    B, scale, zero, w = matrices("mxf4", 1, N, K, 32, False, dtype, 9)
    got = run(tcg, "mxf4", dtype, "f32", A.cuda(), K, N, None, 32, B, scale, zero, 1)
    close(got, a @ w[0].T, np.abs(a) @ np.abs(w[0].T), (K + 8) * 2.0 ** -23, "f32")


def test_infinite_and_nan_activations(tcg):
    """An infinity or NaN reaches its own row's outputs only."""
    K, N = 256, 24
    for dtype in ("bf16", "f16"):
        A, a = rows((3, K), dtype, 1)
        B, scale, zero, w = matrices("int4", 1, N, K, 32, False, dtype, 2)
        clean = run(tcg, "int4", dtype, "f32", A, K, N, None, 32, B, scale, zero, 1)
        A[1, 5], A[2, 200] = float("inf"), float("nan")
        got = run(tcg, "int4", dtype, "f32", A, K, N, None, 32, B, scale, zero, 1)
        assert np.array_equal(got[0], clean[0])
        assert np.isnan(got[2]).all()
        sign = np.sign(w[0][:, 5])
        assert np.array_equal(got[1][sign > 0], np.full((sign > 0).sum(), np.inf))
        assert np.array_equal(got[1][sign < 0], np.full((sign < 0).sum(), -np.inf))
        assert np.isnan(got[1][sign == 0]).all()


def test_matches_the_block_scaled_gemm_storage(tcg):
    """The same packed codes and scale bytes serve tcg_gemm's B: with
    activations that MXFP4 holds exactly both give the same sums."""
    R, N, K = 4, 64, 256
    rng = np.random.default_rng(10)
    ac = rng.integers(0, 16, size=(R, K))
    A4 = torch.from_numpy((ac[:, 0::2] | (ac[:, 1::2] << 4)).astype(np.uint8)).cuda()
    A16 = torch.from_numpy(E2M1[ac]).to(torch.bfloat16).cuda()
    B, scale, _, _ = matrices("mxf4", 1, N, K, 32, False, "bf16", 11)
    one = torch.full((R, K // 32), 127, dtype=torch.uint8, device="cuda")
    D = torch.empty(R, N, device="cuda")
    tcg.gemm_mxf4_blockscaled(R, N, K, A4, tcg.K_MAJOR, K, B, tcg.K_MAJOR, K, one, scale, D, tcg.F32, N)
    got = run(tcg, "mxf4", "bf16", "f32", A16, K, N, None, 32, B, scale, None, 1)
    S = np.abs(to_host(D)) + 2.0 ** 10
    assert np.all(np.abs(got - to_host(D)) <= 2 * K * 2.0 ** -23 * S)


def test_long_matrix_past_32_bits(tcg):
    """Codes beyond 2^32 bytes and 2^32 elements in the last group."""
    N, K, G = 65536, 8192, 18
    assert G * N * K // 2 > 2 ** 32
    B = torch.randint(0, 256, (G, N, K // 2), dtype=torch.uint8, device="cuda")
    scale = torch.full((G, N, K // 32), 120, dtype=torch.uint8, device="cuda")
    A, a = rows((1, K), "bf16", 1)
    off = torch.zeros(G + 1, dtype=torch.int32, device="cuda")
    off[G] = 1
    D = torch.empty(1, N, device="cuda")
    tcg.gemv_w4(tcg.W4_MXF4, tcg.IN_BF16, 1, N, K, A, K, B, scale, D, tcg.F32, N, groups=G, offsets=off)
    _ok(tcg)
    pick = [0, 1, N // 2, N - 1]
    b = B[G - 1][pick].cpu().numpy()
    codes = np.stack([b & 15, b >> 4], -1).reshape(4, K)
    w = E2M1[codes] * 2.0 ** -7
    close(to_host(D)[:, pick], a @ w.T, np.abs(a) @ np.abs(w.T), (K + 8) * 2.0 ** -23, "f32")


def test_no_contraction_and_graph(tcg):
    D = torch.full((3, 20), 7.0, device="cuda")
    tcg.gemv_w4(tcg.W4_MXF4, tcg.IN_BF16, 3, 20, 0, None, 0, None, None, D, tcg.F32, 20)
    _ok(tcg)
    assert bool((D == 0).all())
    A, _ = rows((2, 512), "bf16", 1)
    B, scale, _, _ = matrices("nvf4", 1, 300, 512, 16, False, "bf16", 2)
    s = torch.cuda.Stream()
    D = torch.empty(2, 300, device="cuda")

    def call():
        tcg.gemv_w4(tcg.W4_NVF4, tcg.IN_BF16, 2, 300, 512, A, 512, B, scale, D, tcg.F32, 300, stream=s)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        call()
        s.synchronize()
        want = D.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call()
    D.zero_()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(D, want)


@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
@pytest.mark.parametrize("K", [384, 2048, 4224])
def test_scales_off_a_boundary(tcg, fmt, group, zeros, K):
    """Scales and zero points may start on any 4-byte boundary; the answers are
    those of the same bytes elsewhere, to the bit."""
    G, N, R = 2, 70, 5
    A, _ = rows((R, K), "bf16", 3, 8)
    off = torch.from_numpy(group_offsets([2, 3])).cuda()
    B, scale, zero, _ = matrices(fmt, G, N, K, group, zeros, "bf16", K)
    want = run(tcg, fmt, "bf16", "f32", A, K, N, off, group, B, scale, zero, G)

    def moved(t, by):
        if t is None:
            return None
        flat = t.contiguous().view(torch.uint8).flatten()
        room = torch.full((flat.numel() + 64,), 0xFF, dtype=torch.uint8, device="cuda")
        room[by:by + flat.numel()] = flat
        return room[by:by + flat.numel()].view(t.dtype)

    for by in (4, 8, 12, 16):
        got = run(tcg, fmt, "bf16", "f32", A, K, N, off, group, B, moved(scale, by), moved(zero, by), G)
        assert np.array_equal(got, want), by


def zero_weights(fmt, shape, zero):
    """Codes whose weight is 0: E2M1 0 or -0, INT4 the zero point (None: 8)."""
    if fmt != "int4":
        return np.random.default_rng(0).choice([0, 8], size=shape)
    return np.full(shape, 8) if zero is None else zero


@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
@pytest.mark.parametrize("R", [1, 4, 7, 13])
def test_small_activations_beside_large_ones(tcg, fmt, group, zeros, R):
    """Column k's activations are of the size 2^(40 (k % 6) - 100), and matrix
    row n has weights in the columns of one such size alone: whatever else the
    row of activations holds is multiplied by zero and must not count."""
    K, N = 640, 36
    rng = np.random.default_rng(R)
    x = rng.standard_normal((R, K)) * 2.0 ** (40.0 * (np.arange(K) % 6) - 100)
    A = torch.from_numpy(x).float().bfloat16()
    a = A.double().numpy()
    nb = K // group
    codes = rng.integers(0, 16, size=(N, K))
    zero, zv = None, None
    if zeros:
        zero = rng.integers(0, 16, size=(1, N, nb)).astype(np.uint8)
        zv = np.repeat(zero[0].astype(int), group, axis=1)
    mine = np.arange(K)[None] % 6 == np.arange(N)[:, None] % 6
    codes = np.where(mine, codes, zero_weights(fmt, (N, K), zv))
    if fmt == "int4":
        st = torch.from_numpy(rng.uniform(0.01, 0.1, size=(1, N, nb))).float().bfloat16()
        s, val = st.double().numpy()[0], codes - (8 if zv is None else zv)
    else:
        sb = rng.integers(*((120, 130) if fmt == "mxf4" else (0x10, 0x60)), size=(1, N, nb)).astype(np.uint8)
        st, val = torch.from_numpy(sb), E2M1[codes]
        s = 2.0 ** (sb[0].astype(float) - 127) if fmt == "mxf4" else ue4m3(sb[0])
    w = val * np.repeat(s, group, axis=1)
    packed = torch.from_numpy((codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)).cuda()
    got = run(tcg, fmt, "bf16", "f32", A.cuda(), K, N, None, group, packed, st.cuda(),
              None if zero is None else torch.from_numpy(zero).cuda(), 1)
    close(got, a @ w.T, np.abs(a) @ np.abs(w.T), (K + 8) * 2.0 ** -23, "f32")


@pytest.mark.parametrize("R", [1, 4, 7, 13])
def test_scales_against_activations(tcg, R):
    """Groups of one slab whose scales undo their activations' sizes, over the
    whole range of both: every group counts alike."""
    K, N, group = 512, 24, 32
    rng = np.random.default_rng(R + 20)
    size = rng.integers(-100, 120, size=K // group)
    x = rng.standard_normal((R, K)) * 2.0 ** np.repeat(size, group)
    A = torch.from_numpy(x).float().bfloat16()
    a = A.double().numpy()
    codes = rng.integers(0, 16, size=(N, K))
    B = torch.from_numpy((codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)).cuda()
    for fmt in ("mxf4", "int4"):
        if fmt == "mxf4":
            st = torch.from_numpy(np.broadcast_to(127 - size, (N, K // group)).astype(np.uint8).copy())
        else:
            st = torch.from_numpy(np.broadcast_to(2.0 ** -size, (N, K // group)).copy()).float().bfloat16()
        val = E2M1[codes] if fmt == "mxf4" else codes - 8
        w = val * np.repeat(2.0 ** -size.astype(float), group)
        got = run(tcg, fmt, "bf16", "f32", A.cuda(), K, N, None, group, B, st.cuda(), None, 1)
        close(got, a @ w.T, np.abs(a) @ np.abs(w.T), (K + 8) * 2.0 ** -23, "f32", fmt)


def test_smallest_activations(tcg):
    """bf16's subnormal activations under a scale that brings them back, beside
    ones of ordinary size that meet zero weights."""
    K, N, R = 256, 16, 3
    rng = np.random.default_rng(31)
    A = torch.from_numpy(rng.integers(-127, 128, size=(R, K)) * 2.0 ** -133).float().bfloat16()
    A[1:, ::7] = 1.0
    a = A.double().numpy()
    codes = rng.integers(0, 16, size=(N, K))
    codes[:, ::7] = 0
    B = torch.from_numpy((codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)).cuda()
    sb = np.full((N, K // 32), 127 + 100, np.uint8)
    got = run(tcg, "mxf4", "bf16", "f32", A.cuda(), K, N, None, 32, B, torch.from_numpy(sb).cuda(), None, 1)
    w = E2M1[codes] * 2.0 ** 100
    close(got, a @ w.T, np.abs(a) @ np.abs(w.T), (K + 8) * 2.0 ** -23, "f32")


@pytest.mark.parametrize("R", [1, 7, 13])
def test_finite_results_of_the_largest_activations(tcg, R):
    """Activations near the end of bf16's range whose scales keep the result
    far from fp32's."""
    K, N, group = 256, 16, 32
    A = torch.full((R, K), 2.0 ** 126, dtype=torch.bfloat16)
    a = A.double().numpy()
    B = torch.full((N, K // 2), 0x77, dtype=torch.uint8, device="cuda")  # 6, INT4 7 - 8
    for fmt, st, w in (("mxf4", torch.full((N, K // group), 127 - 20, dtype=torch.uint8), 6 * 2.0 ** -20),
                       ("int4", torch.full((N, K // group), 2.0 ** -20, dtype=torch.bfloat16), -2.0 ** -20)):
        got = run(tcg, fmt, "bf16", "f32", A.cuda(), K, N, None, group, B, st.cuda(), None, 1)
        ref = a @ np.full((K, N), w)
        close(got, ref, np.abs(ref), (K + 8) * 2.0 ** -23, "f32", fmt)


def device_matrices(fmt, G, N, K, group, zeros, dtype, seed, pad_s):
    """As matrices(), made on the GPU: device codes, scales, zero points, and
    weights(g) -> float64 matrix g."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    nb = K // group
    B = torch.randint(0, 256, (G, N, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
    zero = None
    if fmt == "int4":
        scale = (0.01 + 0.09 * torch.rand((G, N, nb + pad_s), device="cuda", generator=gen)).to(TORCH[dtype])
        if zeros:
            zero = torch.randint(0, 16, (G, N, nb + pad_s), dtype=torch.uint8, device="cuda", generator=gen)
    else:
        lo, hi = (120, 130) if fmt == "mxf4" else (0x01, 0x60)
        scale = torch.randint(lo, hi, (G, N, nb + pad_s), dtype=torch.uint8, device="cuda", generator=gen)
    table = torch.from_numpy(E2M1).cuda()

    def weights(g):
        code = torch.stack([B[g] & 15, B[g] >> 4], -1).view(N, nb, group)
        sc = scale[g, :, :nb]
        if fmt == "int4":
            val = code.double() - (8 if zero is None else zero[g, :, :nb, None].double())
            s = sc.double()
        else:
            val = table[code.int()]
            s = torch.exp2(sc.double() - 127) if fmt == "mxf4" else sc.view(torch.float8_e4m3fn).double()
        return (val * s[..., None]).view(N, K)
    return B, scale, zero, weights


@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
@pytest.mark.parametrize("sizes,N,K", [([3], 20001, 1024), ([8], 12000, 4608), ([16], 9001, 2560),
                                       ([3, 0, 9, 2], 4001, 4608)])
def test_many_tiles_of_a_wide_range(tcg, fmt, group, zeros, sizes, N, K):
    """Activations of the sizes 2^90, 1 and 2^-90 column by column, in every
    other 256 of K; a matrix row has weights under all of them, under the two
    smaller or under the smallest alone.  Every output is compared."""
    G, R = len(sizes), sum(sizes)
    off = group_offsets(sizes)
    rng = np.random.default_rng(K)
    column = np.arange(K) % 3 * (np.arange(K) // 256 % 2) + np.arange(K) // 256 % 2 - 1  # -1: usual, 0..3
    x = rng.standard_normal((R, K)) * np.choose(column + 1, [1.0, 2.0 ** 90, 1.0, 2.0 ** -90, 1.0])
    A = torch.from_numpy(x).float().bfloat16().cuda()
    x = A.double()
    none = torch.from_numpy(np.where(column[None] < 0, np.arange(3)[:, None] > 0,
                                     column[None] < np.arange(3)[:, None])).cuda()[torch.arange(N).cuda() % 3]
    for pad_s in (0, 1):
        B, scale, zero, weights = device_matrices(fmt, G, N, K, group, zeros, "bf16", N + K, pad_s)
        for g in range(G):
            null = torch.zeros((), dtype=torch.uint8, device="cuda")
            if fmt == "int4":
                null = null + 8 if zero is None else zero[g, :, :K // group].repeat_interleave(group, 1)
            code = torch.where(none, null, torch.stack([B[g] & 15, B[g] >> 4], -1).view(N, K))
            B[g] = code[:, 0::2] | code[:, 1::2] << 4
        got = run(tcg, fmt, "bf16", "f32", A, K, N, torch.from_numpy(off).cuda(), group, B, scale, zero, G, None, 0,
                  pad_s)
        for g in range(G):
            sl, w = slice(off[g], off[g + 1]), weights(g)
            close(got[sl], to_host(x[sl] @ w.T), to_host(x[sl].abs() @ w.abs().T), (K + 8) * 2.0 ** -23, "f32", (g, pad_s))


@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
@pytest.mark.parametrize("stride", [1, 8, 3000001])
def test_one_group_takes_any_scale_stride(tcg, fmt, group, zeros, stride):
    """With one group nothing lies a stride further on."""
    R, N, K = 2, 40, 4096
    A, a = rows((R, K), "bf16", 1)
    B, scale, zero, w = matrices(fmt, 1, N, K, group, zeros, "bf16", 2)
    D = torch.empty(R, N, device="cuda")
    tcg.gemv_w4({"int4": 0, "mxf4": 1, "nvf4": 2}[fmt], tcg.IN_BF16, R, N, K, A, K, B, scale, D, tcg.F32, N,
                group=group, zero=zero, stride_scale=stride)
    _ok(tcg)
    close(to_host(D), a @ w[0].T, np.abs(a) @ np.abs(w[0].T), (K + 8) * 2.0 ** -23, "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
@pytest.mark.parametrize("R,N,K", [(1, 45001, 256), (8, 30001, 512), (16, 20003, 512), (3, 45001, 4608),
                                   (7, 40003, 4352), (13, 45000, 2304), (2, 20000, 1152)])
def test_many_tiles(tcg, dtype, fmt, group, zeros, R, N, K):
    """Many tiles a CTA, one below the other: short contractions, whose tiles
    hold up to 512 rows, and ones of several passes over more tiles than their
    sums have room for.  Every output is compared, scales on 16-byte
    boundaries and off them."""
    A, a = rows((R, K), dtype, 1, 8)
    for pad_s in (0, 1):
        B, scale, zero, weights = device_matrices(fmt, 1, N, K, group, zeros, dtype, N + K, pad_s)
        got = run(tcg, fmt, dtype, "f32", A, K, N, None, group, B, scale, zero, 1, None, 0, pad_s, N + 3)
        w, x = weights(0), torch.from_numpy(a).cuda()
        close(got, to_host(x @ w.T), to_host(x.abs() @ w.abs().T), (K + 8) * 2.0 ** -23, "f32", pad_s)


@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
@pytest.mark.parametrize("sizes,N,K", [([3, 0, 1, 5, 2, 4], 9001, 512), ([9, 0, 20, 1], 7000, 2304)])
def test_many_tiles_of_groups(tcg, fmt, group, zeros, sizes, N, K):
    G, R = len(sizes), sum(sizes)
    off = group_offsets(sizes)
    A, a = rows((R, K), "bf16", 1, 8)
    x = torch.from_numpy(a).cuda()
    for pad_s in (0, 1):
        B, scale, zero, weights = device_matrices(fmt, G, N, K, group, zeros, "bf16", N + K, pad_s)
        got = run(tcg, fmt, "bf16", "f32", A, K, N, torch.from_numpy(off).cuda(), group, B, scale, zero, G, None, 0,
                  pad_s)
        for g in range(G):
            sl, w = slice(off[g], off[g + 1]), weights(g)
            close(got[sl], to_host(x[sl] @ w.T), to_host(x[sl].abs() @ w.abs().T), (K + 8) * 2.0 ** -23, "f32", (g, pad_s))


def test_long_matrix_every_output(tcg):
    """All outputs of a matrix of 65536 rows of 8192, the second of two groups."""
    N, K, G = 65536, 8192, 2
    A, a = rows((2, K), "bf16", 1)
    B, scale, _, weights = device_matrices("mxf4", G, N, K, 32, False, "bf16", 3, 0)
    off = torch.tensor([0, 0, 2], dtype=torch.int32, device="cuda")
    got = run(tcg, "mxf4", "bf16", "f32", A, K, N, off, 32, B, scale, None, G)
    w, x = weights(1), torch.from_numpy(a).cuda()
    close(got, to_host(x @ w.T), to_host(x.abs() @ w.abs().T), (K + 8) * 2.0 ** -23, "f32")
