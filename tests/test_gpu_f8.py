"""Products of 8-bit codes with a scale for each block of 128, dense and grouped,
against float64.

Tolerance, of sum |products|: a product of two codes is exact in fp32 and a
block's sum makes at most 128 roundings of 2^-23 (the tensor core may
truncate); forming the factor, scaling and adding the block are four roundings
of 2^-24, and adding ceil(K/128) blocks at most as many of 2^-24.  Then the
rounding to the stored type."""
import numpy as np
import pytest
import torch

from f8_cases import BLOCK, IN_TYPE, along, blocks, codes, row_blocks, scales, spread
from moe_cases import DTYPE, TORCH, close, group_offsets, to_host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tcg():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from blackwell_tensor_core_swizzled_gb300 import build
    build.build()
    import blackwell_tensor_core_swizzled_gb300 as m
    return m


def ok(tcg):
    rc = tcg.check()
    assert rc == 0, tcg.last_error_string()


def tau(K):
    return min(K, BLOCK) * 2.0 ** -23 + (4 + blocks(K)) * 2.0 ** -24


def dense(tcg, M, N, K, fmt, a_major, b_major, square, out, pad=0):
    A, a = codes((M, K) if a_major == "k" else (K, M), fmt, 1, pad)
    B, b = codes((N, K) if b_major == "k" else (K, N), fmt, 2, pad)
    SA, sa = scales((blocks(K), M), fmt, 3, 1.0, pad)
    shape = (blocks(K), N) if not square else (blocks(N), blocks(K)) if b_major == "k" else (blocks(K), blocks(N))
    SB, sb = scales(shape, fmt, 4, K ** -0.5, pad)
    D = torch.full((M, N + pad), 7.0, dtype=TORCH[out], device="cuda")
    tcg.gemm_f8(IN_TYPE[fmt], M, N, K, A, tcg.K_MAJOR if a_major == "k" else tcg.MN_MAJOR, A.shape[1], SA,
                SA.shape[1], B, tcg.K_MAJOR if b_major == "k" else tcg.MN_MAJOR, B.shape[1], SB, SB.shape[1], square, D,
                DTYPE[out], N + pad)
    ok(tcg)
    assert bool((D[:, N:] == 7.0).all()), "wrote past the row"
    am = (a if a_major == "k" else a.T) * along(sa, K).T
    if square:
        bm = b * spread(sb, *b.shape)
        bm = bm if b_major == "k" else bm.T
    else:
        bm = (b if b_major == "k" else b.T) * along(sb, K).T
    close(to_host(D)[:, :N], am @ bm.T, np.abs(am) @ np.abs(bm).T, tau(K), out, (M, N, K, a_major, b_major, square))


SIZES = [(1, 1, 1), (1, 128, 128), (3, 257, 129), (5, 40, 1023), (8, 1000, 3000), (16, 136, 1000), (17, 384, 512), (64, 129, 260), (65, 264, 384),
         (129, 130, 640), (256, 512, 2048), (300, 1000, 1100), (513, 200, 100)]


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_forward(tcg, fmt, M, N, K):
    for out in ("f32", "bf16", "f16"):
        dense(tcg, M, N, K, fmt, "k", "k", True, out)


@pytest.mark.parametrize("M,N,K", SIZES)
def test_rows_gradient(tcg, M, N, K):
    dense(tcg, M, N, K, "e5m2", "k", "mn", True, "f32", 1)
    dense(tcg, M, N, K, "e4m3", "k", "mn", True, "bf16", 2)


@pytest.mark.parametrize("M,N,K", SIZES)
def test_matrix_gradient(tcg, M, N, K):
    dense(tcg, M, N, K, "e4m3", "mn", "mn", False, "f32", 1)
    dense(tcg, M, N, K, "e5m2", "mn", "mn", False, "f16")


@pytest.mark.parametrize("M,N,K", [(1, 130, 200), (65, 264, 384), (300, 200, 1000)])
def test_other_majors(tcg, M, N, K):
    for a_major in ("k", "mn"):
        for b_major in ("k", "mn"):
            for square in (False, True):
                dense(tcg, M, N, K, "e4m3", a_major, b_major, square, "f32", 1)


@pytest.mark.parametrize("M,N,K", [(1300, 1000, 300), (700, 2057, 72), (2049, 1032, 1), (577, 2600, 8200)])
def test_large_tiles(tcg, M, N, K):
    """More tiles of 128 x 64 than SMs: those of 256 x 256, ragged on every side."""
    for out in ("f32", "bf16"):
        dense(tcg, M, N, K, "e4m3", "k", "k", True, out)
        assert "tile 256x256" in tcg.last_plan_string()
    dense(tcg, M, N, K, "e5m2", "k", "mn", True, "f16", 1)


def test_many_tiles(tcg):
    dense(tcg, 3000, 2600, 400, "e4m3", "k", "k", True, "bf16")
    dense(tcg, 40, 20000, 300, "e4m3", "k", "k", True, "f32")


def test_empty_contraction_and_empty_outputs(tcg):
    D = torch.full((5, 40), 7.0, device="cuda")
    tcg.gemm_f8(tcg.IN_E4M3, 5, 40, 0, None, 0, 0, None, 0, None, 0, 0, None, 0, True, D, tcg.F32, 40)
    ok(tcg)
    assert not to_host(D).any()
    D.fill_(7.0)
    tcg.gemm_f8(tcg.IN_E4M3, 0, 40, 128, None, 0, 0, None, 0, None, 0, 0, None, 0, True, D, tcg.F32, 40)
    ok(tcg)
    assert tcg.last_launch_count() == 0 and bool((D == 7.0).all())


def test_grouped_without_rows_or_contraction(tcg):
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    W = torch.full((3, 40, 48), 7.0, device="cuda")
    tcg.gemm_f8_grouped_wgrad(tcg.IN_E4M3, 0, 40, 48, 3, None, 0, None, 0, None, 0, None, 0, off, W, tcg.F32, 48, 0)
    ok(tcg)
    assert not to_host(W).any()
    D = torch.full((5, 40), 7.0, device="cuda")
    tcg.gemm_f8_grouped(tcg.IN_E4M3, 0, 40, 48, 3, None, 0, None, 0, off, None, tcg.K_MAJOR, 0, 0, None, 0, 0, D, tcg.F32,
                        40)
    assert tcg.last_launch_count() == 0 and bool((D == 7.0).all())
    off.fill_(5)
    off[0] = 0
    tcg.gemm_f8_grouped(tcg.IN_E4M3, 5, 40, 0, 3, None, 0, None, 0, off, None, tcg.K_MAJOR, 0, 0, None, 0, 0, D, tcg.F32,
                        40)
    ok(tcg)
    assert not to_host(D).any()


CASES = [
    # sizes of the groups, loose rows before and after, N, K, rows padded by
    ([1], 0, 0, 16, 16, 0),
    ([5], 0, 0, 1, 1, 0),
    ([0, 3, 0, 0, 130, 1, 0], 0, 0, 264, 72, 1),
    ([128, 128, 256], 0, 0, 256, 128, 0),
    ([17, 33, 64, 65, 127, 129], 0, 5, 200, 136, 0),
    ([700, 0, 300], 3, 4, 130, 520, 1),
    ([0, 0, 0], 0, 9, 72, 64, 0),
    ([257, 255, 513], 0, 0, 513, 1000, 0),
    ([3] * 40, 1, 1, 384, 192, 0),
    ([1, 2, 4, 8, 16, 31, 32, 48], 0, 0, 1030, 2056, 0),
    ([20, 0, 1, 0, 0, 9, 0, 0, 2], 2, 3, 40, 1100, 1),
    ([1] * 1024, 0, 0, 24, 130, 0),
    # tiles of 256 rows
    ([700, 0, 300], 3, 4, 2610, 520, 1),
    ([130, 65, 33, 127, 129, 200], 0, 5, 1304, 136, 0),
    ([257, 255, 513], 0, 0, 2104, 1000, 0),
    ([128, 128, 256], 0, 0, 2560, 128, 0),
    ([400, 1, 0, 31, 600], 1, 0, 1301, 264, 0),
]


@pytest.mark.parametrize("major", ["k", "mn"])
@pytest.mark.parametrize("sizes,before,after,N,K,pad", CASES)
def test_grouped(tcg, major, sizes, before, after, N, K, pad):
    G, R = len(sizes), sum(sizes) + before + after
    off = group_offsets(sizes, before)
    fmt = "e4m3" if major == "k" else "e5m2"
    A, a = codes((R, K), fmt, 1, pad)
    SA, sa = scales((blocks(K), R), fmt, 2, 1.0, pad)
    rows, cols = (N, K) if major == "k" else (K, N)
    B, b = codes((G, rows, cols), fmt, 3, pad)
    SB, sb = scales((G, blocks(rows), blocks(cols)), fmt, 4, K ** -0.5, pad)
    a = a * along(sa, K).T
    b = b * spread(sb, rows, cols)
    ref, S = np.zeros((R, N)), np.zeros((R, N))
    for g in range(G):
        sl, m = slice(off[g], off[g + 1]), b[g].T if major == "k" else b[g]
        ref[sl], S[sl] = a[sl] @ m, np.abs(a[sl]) @ np.abs(m)
    for out, more in (("f32", 3), ("bf16", 3), ("f32", 8), ("bf16", 8), ("f16", 8)):  # rows that end on 16 bytes or not
        D = torch.full((R, N + more), 7.0, dtype=TORCH[out], device="cuda")
        tcg.gemm_f8_grouped(IN_TYPE[fmt], R, N, K, G, A, A.shape[1], SA, SA.shape[1], torch.from_numpy(off).cuda(), B,
                            tcg.K_MAJOR if major == "k" else tcg.MN_MAJOR, B.shape[2], 0, SB, SB.shape[2], 0, D,
                            DTYPE[out], N + more)
        ok(tcg)
        close(to_host(D)[:, :N], ref, S, tau(K), out, (major, out))
        assert bool((D[:, N:] == 7.0).all()), "wrote past the row"


@pytest.mark.parametrize("sizes,before,after,N,K,pad", CASES)
def test_grouped_wgrad(tcg, sizes, before, after, N, K, pad):
    G, R = len(sizes), sum(sizes) + before + after
    off = group_offsets(sizes, before)
    DY, dy = codes((R, N), "e4m3", 5, pad)
    A, a = codes((R, K), "e4m3", 6, pad)
    SDY, sdy = scales((R // BLOCK + G, N), "e4m3", 7, 0.1, pad)
    SA, sa = scales((R // BLOCK + G, K), "e4m3", 8, 1.0, pad)
    at = row_blocks(off, R)
    dy, a = dy * sdy[at], a * sa[at]
    for out, more in (("f32", 5), ("bf16", 5), ("f32", 8), ("bf16", 8), ("f16", 8)):
        DW = torch.full((G, N, K + more), 7.0, dtype=TORCH[out], device="cuda")
        tcg.gemm_f8_grouped_wgrad(tcg.IN_E4M3, R, N, K, G, DY, DY.shape[1], SDY, SDY.shape[1], A, A.shape[1], SA,
                                  SA.shape[1], torch.from_numpy(off).cuda(), DW, DTYPE[out], K + more, 0)
        ok(tcg)
        ref, S = np.zeros((G, N, K)), np.zeros((G, N, K))
        for g in range(G):
            sl = slice(off[g], off[g + 1])
            ref[g], S[g] = dy[sl].T @ a[sl], np.abs(dy[sl]).T @ np.abs(a[sl])
        close(to_host(DW)[:, :, :K], ref, S, tau(max(sizes)), out, out)
        assert bool((DW[:, :, K:] == 7.0).all())


def test_plans(tcg):
    """Which kernel a size takes, so that the cases above reach them all."""
    for M, N, K, square, plan in ((8, 1000, 300, True, "8-bit, blocks of 8"), (9, 1000, 300, True, "tile 128x64"),
                                  (16, 1000, 2000, True, "cta_group 2, tile 256x64"),
                                  (16, 1000, 4000, True, "cta_group 4, tile 512x64"),
                                  (256, 1000, 300, True, "tile 128x64"), (1300, 1000, 300, True, "tile 256x256"), (1, 300, 300, False, "tile 256x256")):
        dense(tcg, M, N, K, "e4m3", "k", "k", square, "f32")
        assert plan in tcg.last_plan_string(), (M, N, K, tcg.last_plan_string())


@pytest.mark.parametrize("bad", [0x7f, 0xff])
def test_other_groups_values_stay_out(tcg, bad):
    """NaN codes in one group's rows or matrix reach no other group, nor do they
    come back through loose rows."""
    for sizes, N in (([5, 9, 70, 3], 136), ([2, 1, 3, 1], 136), ([300, 40, 200, 120], 2568)):
        K = 200
        G, R = len(sizes), sum(sizes) + 4
        off = group_offsets(sizes, 2)
        t_off = torch.from_numpy(off).cuda()
        A, _ = codes((R, K), "e4m3", 1)
        B, _ = codes((G, N, K), "e4m3", 2)
        DY, _ = codes((R, N), "e4m3", 3)
        SA, _ = scales((blocks(K), R), "e4m3", 4)
        SB, _ = scales((G, blocks(N), blocks(K)), "e4m3", 5)
        SX, _ = scales((R // BLOCK + G, K), "e4m3", 6)
        SY, _ = scales((R // BLOCK + G, N), "e4m3", 7)
        outs = []
        for poison in (False, True):
            if poison:
                A[off[2]:off[3]] = bad
                A[:2] = A[R - 2:] = bad
                DY[off[2]:off[3]] = bad
                DY[:2] = DY[R - 2:] = bad
                B[2] = bad
            D = torch.zeros(R, N, device="cuda")
            tcg.gemm_f8_grouped(tcg.IN_E4M3, R, N, K, G, A, A.shape[1], SA, R, t_off, B, tcg.K_MAJOR, B.shape[2], 0, SB, 0,
                                0, D, tcg.F32, N)
            W = torch.zeros(G, N, K, device="cuda")
            tcg.gemm_f8_grouped_wgrad(tcg.IN_E4M3, R, N, K, G, DY, DY.shape[1], SY, N, A, A.shape[1], SX, K, t_off, W,
                                      tcg.F32, K, 0)
            ok(tcg)
            outs.append((to_host(D), to_host(W)))
        kept = np.r_[0:off[2], off[3]:R]
        assert np.array_equal(outs[0][0][kept], outs[1][0][kept])
        assert np.isnan(outs[1][0][off[2]:off[3]]).all()
        groups = [0, 1, 3]
        assert np.array_equal(outs[0][1][groups], outs[1][1][groups])
        assert np.isnan(outs[1][1][2]).all()


def test_gradients_against_differences(tcg):
    """Codes that are small integers under scales of one: every sum is exact, so
    the gradients equal differences of L = <DY, grouped(A, B)> exactly."""
    sizes, N, K = [3, 0, 140, 6], 48, 144
    G, R = len(sizes), sum(sizes)
    off = torch.from_numpy(group_offsets(sizes)).cuda()
    rng = np.random.default_rng(9)

    def ints(*s):
        return torch.from_numpy(rng.integers(-3, 4, size=s)).float().to(torch.float8_e4m3fn).view(torch.uint8).cuda()
    A, B, DY = ints(R, K), ints(G, N, K), ints(R, N)
    one = lambda *s: torch.ones(*s, device="cuda")  # noqa: E731
    dy = DY.view(torch.float8_e4m3fn).double()

    def loss(a, b):
        D = torch.empty(R, N, device="cuda")
        tcg.gemm_f8_grouped(tcg.IN_E4M3, R, N, K, G, a, K, one(blocks(K), R), R, off, b, tcg.K_MAJOR, K, 0,
                            one(G, blocks(N), blocks(K)), 0, 0, D, tcg.F32, N)
        return float((D.double() * dy).sum())
    DA = torch.empty(R, K, device="cuda")
    tcg.gemm_f8_grouped(tcg.IN_E4M3, R, K, N, G, DY, N, one(blocks(N), R), R, off, B, tcg.MN_MAJOR, K, N * K,
                        one(G, blocks(N), blocks(K)), 0, 0, DA, tcg.F32, K)
    DW = torch.empty(G, N, K, device="cuda")
    tcg.gemm_f8_grouped_wgrad(tcg.IN_E4M3, R, N, K, G, DY, N, one(R // BLOCK + G, N), N, A, K, one(R // BLOCK + G, K), K,
                              off, DW, tcg.F32, K, N * K)
    ok(tcg)
    base = loss(A, B)

    def up(t, *i):
        c = t.clone()
        v = c.view(torch.float8_e4m3fn)[i].float() + 1
        c[i] = v.to(torch.float8_e4m3fn).view(torch.uint8)
        return c
    for i in range(0, R, 7):
        k = 7 * i % K
        assert loss(up(A, i, k), B) - base == float(DA[i, k])
    for g in range(G):
        for n in (0, 17, N - 1):
            k = (n + 5 * g) % K
            assert loss(A, up(B, g, n, k)) - base == float(DW[g, n, k])


def test_captured_on_two_streams(tcg):
    """Two graphs on two streams, replayed together: nothing is shared."""
    graphs = []
    for M, N, K, seed in ((4, 2048, 2048, 1), (300, 512, 1024, 2), (16, 512, 4096, 3), (1300, 1024, 256, 4)):
        A, a = codes((M, K), "e4m3", seed)
        B, b = codes((N, K), "e4m3", seed + 10)
        SA, sa = scales((blocks(K), M), "e4m3", seed + 20)
        SB, sb = scales((blocks(N), blocks(K)), "e4m3", seed + 30, K ** -0.5)
        D = torch.zeros(M, N, device="cuda")
        side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=side):
            tcg.gemm_f8(tcg.IN_E4M3, M, N, K, A, tcg.K_MAJOR, K, SA, M, B, tcg.K_MAJOR, K, SB, blocks(K), True, D, tcg.F32,
                        N)
        am, bm = a * along(sa, K).T, b * spread(sb, N, K)
        graphs.append((graph, side, D, am @ bm.T, np.abs(am) @ np.abs(bm).T, K, (A, B, SA, SB)))
    for _ in range(5):
        for graph, side, *_ in graphs:
            with torch.cuda.stream(side):
                graph.replay()
    torch.cuda.synchronize()
    ok(tcg)
    for _, _, D, ref, S, K, _ in graphs:
        close(to_host(D), ref, S, tau(K), "f32")


def test_plan_names_the_tile_and_who_shares_it(tcg):
    """The plan says the tile of the kernel that ran, the CTAs that share a
    contraction, and whether there are groups."""
    for M, N, K, square, tile, shared in (
            (9, 1000, 300, True, "tile 128x64 by cta_group 1", 1), (16, 1000, 2000, True, "tile 128x64 by cta_group 1", 2),
            (16, 1000, 4000, True, "tile 128x64 by cta_group 1", 4), (1300, 1000, 300, True, "tile 256x256 by cta_group 2", 1),
            (1, 300, 300, False, "tile 256x256 by cta_group 2", 1)):
        dense(tcg, M, N, K, "e4m3", "k", "k", square, "f32")
        plan = tcg.last_plan_string()
        assert plan.startswith("8-bit, " + tile) and "grouped" not in plan, plan
        assert (f"contraction over {shared} CTAs" in plan) == (shared > 1), plan
    off = torch.tensor([0, 20, 40], dtype=torch.int32, device="cuda")
    for call in ("rows", "weight"):
        A, SA, D = torch.zeros(40, 256, dtype=torch.uint8, device="cuda"), torch.ones(2, 256, device="cuda"), torch.empty(
            2, 256, 256, device="cuda")
        if call == "rows":
            tcg.gemm_f8_grouped(tcg.IN_E4M3, 40, 256, 256, 2, A, 256, SA, 256, off, torch.zeros(
                2, 256, 256, dtype=torch.uint8, device="cuda"), tcg.MN_MAJOR, 256, 0, torch.ones(2, 2, 2, device="cuda"), 0, 0,
                D, tcg.F32, 256)
        else:
            tcg.gemm_f8_grouped_wgrad(tcg.IN_E4M3, 40, 256, 256, 2, A, 256, SA, 256, A, 256, SA, 256, off, D, tcg.F32, 256, 0)
        ok(tcg)
        assert tcg.last_plan_string().startswith("8-bit, grouped, tile "), tcg.last_plan_string()


def apart(t, more, fill):
    """t [G][...] in a buffer whose matrices lie `more` elements further apart, and their stride."""
    n = t[0].numel()
    big = torch.full((t.shape[0], n + more), fill, dtype=t.dtype, device="cuda")
    big[:, :n] = t.reshape(t.shape[0], n)
    return big, n + more


@pytest.mark.parametrize("major", ["k", "mn"])
@pytest.mark.parametrize("sizes,N,K", [([1, 2, 0, 1], 136, 200), ([5, 0, 70, 30], 264, 300), ([300, 40, 0, 520], 2568, 200)])
def test_matrices_and_scales_apart(tcg, major, sizes, N, K):
    """Matrices, scales and gradients inside larger buffers, with NaN between them:
    bit for bit the packed results, and nothing written between."""
    G, R = len(sizes), sum(sizes)
    off = torch.from_numpy(group_offsets(sizes)).cuda()
    rows, cols = (N, K) if major == "k" else (K, N)
    A, _ = codes((R, K), "e4m3", 1)
    SA, _ = scales((blocks(K), R), "e4m3", 2)
    B, _ = codes((G, rows, cols), "e4m3", 3)
    SB, _ = scales((G, blocks(rows), blocks(cols)), "e4m3", 4)
    DY, _ = codes((R, N), "e4m3", 5)
    SY, _ = scales((R // BLOCK + G, N), "e4m3", 6)
    SX, _ = scales((R // BLOCK + G, K), "e4m3", 7)
    B2, stride_b = apart(B, 48, 0x7f)
    SB2, stride_sb = apart(SB, 5, float("nan"))
    outs, grads = [], []
    for b, sb, s, ss in ((B, 0, SB, 0), (B2, stride_b, SB2, stride_sb)):
        D = torch.zeros(R, N, device="cuda")
        tcg.gemm_f8_grouped(tcg.IN_E4M3, R, N, K, G, A, A.shape[1], SA, R, off, b,
                            tcg.K_MAJOR if major == "k" else tcg.MN_MAJOR, B.shape[2], sb, s, SB.shape[2], ss, D, tcg.F32, N)
        ok(tcg)
        outs.append(D)
    assert torch.equal(*outs)
    for more in (0, 12, 7):  # 16-byte strides, and none
        W = torch.full((G, N * K + more), 7.0, device="cuda")
        tcg.gemm_f8_grouped_wgrad(tcg.IN_E4M3, R, N, K, G, DY, DY.shape[1], SY, N, A, A.shape[1], SX, K, off, W, tcg.F32, K,
                                  N * K + more if more else 0)
        ok(tcg)
        assert bool((W[:, N * K:] == 7.0).all()), "wrote between the matrices"
        grads.append(W[:, :N * K])
    assert torch.equal(grads[0], grads[1]) and torch.equal(grads[0], grads[2])


@pytest.mark.parametrize("sizes,before,after,N,K,pad", [CASES[2], CASES[5], CASES[9], CASES[12]])
def test_grouped_wgrad_of_e5m2(tcg, sizes, before, after, N, K, pad):
    G, R = len(sizes), sum(sizes) + before + after
    off = group_offsets(sizes, before)
    DY, dy = codes((R, N), "e5m2", 5, pad)
    A, a = codes((R, K), "e5m2", 6, pad)
    SDY, sdy = scales((R // BLOCK + G, N), "e5m2", 7, 0.1, pad)
    SA, sa = scales((R // BLOCK + G, K), "e5m2", 8, 1.0, pad)
    at = row_blocks(off, R)
    dy, a = dy * sdy[at], a * sa[at]
    ref, S = np.zeros((G, N, K)), np.zeros((G, N, K))
    for g in range(G):
        sl = slice(off[g], off[g + 1])
        ref[g], S[g] = dy[sl].T @ a[sl], np.abs(dy[sl]).T @ np.abs(a[sl])
    for out in ("f32", "bf16"):
        DW = torch.full((G, N, K), 7.0, dtype=TORCH[out], device="cuda")
        tcg.gemm_f8_grouped_wgrad(tcg.IN_E5M2, R, N, K, G, DY, DY.shape[1], SDY, SDY.shape[1], A, A.shape[1], SA, SA.shape[1],
                                  torch.from_numpy(off).cuda(), DW, DTYPE[out], K, 0)
        ok(tcg)
        close(to_host(DW), ref, S, tau(max(sizes)), out, out)


@pytest.mark.parametrize("sizes,N,K,plan", [
    ([2] * 16, 256, 272, "8-bit, blocks of 8"), ([1] * 48, 2048, 4096, "8-bit, blocks of 8"),
    ([2] * 512, 128, 272, "tile 128x64"), ([0] * 300 + [600] + [0] * 299, 40, 272, "tile 128x64"),
    ([8] * 8, 256, 272, "8-bit, blocks of 8"), ([0, 30, 2, 0, 0], 256, 272, "8-bit, blocks of 8"), ([8] * 300, 128, 272, "tile 128x64")])
def test_many_matrices_are_not_streamed(tcg, sizes, N, K, plan):
    """Few rows a group: streamed where the matrices' tiles are few, tiles where
    they are many (one popular group among them), with the same results."""
    G, R = len(sizes), sum(sizes)
    off = group_offsets(sizes)
    A, a = codes((R, K), "e4m3", 1)
    SA, sa = scales((blocks(K), R), "e4m3", 2)
    few = min(G, 40)            # as many matrices, the rest the first again
    B, b = codes((few, N, K), "e4m3", 3)
    SB, sb = scales((few, blocks(N), blocks(K)), "e4m3", 4, K ** -0.5)
    pick = np.arange(G) % few
    b = b * spread(sb, N, K)
    ld = B.shape[2]
    B, SB = B[torch.from_numpy(pick).cuda()].contiguous(), SB[torch.from_numpy(pick).cuda()].contiguous()
    D = torch.full((R, N), 7.0, device="cuda")
    tcg.gemm_f8_grouped(tcg.IN_E4M3, R, N, K, G, A, A.shape[1], SA, R, torch.from_numpy(off).cuda(), B, tcg.K_MAJOR, ld, 0,
                        SB, 0, 0, D, tcg.F32, N)
    ok(tcg)
    assert plan in tcg.last_plan_string(), tcg.last_plan_string()
    a = a * along(sa, K).T
    ref, S = np.zeros((R, N)), np.zeros((R, N))
    for g in range(G):
        sl = slice(off[g], off[g + 1])
        ref[sl], S[sl] = a[sl] @ b[pick[g]].T, np.abs(a[sl]) @ np.abs(b[pick[g]]).T
    close(to_host(D), ref, S, tau(K), "f32", (sizes[:8], N, K))


@pytest.mark.parametrize("M,square", [(3, True), (70, True), (1300, True), (70, False)])
def test_factors_below_the_normal_range(tcg, M, square):
    """Scales whose product is no normal fp32 number: it is off by 2^-150 at most,
    so that many times a block's sum is added to the tolerance."""
    N, K = 1000, 300
    A, a = codes((M, K), "e4m3", 1)
    B, b = codes((N, K), "e4m3", 2)
    SA, sa = scales((blocks(K), M), "e4m3", 3, 2.0 ** -82)
    SB, sb = scales((blocks(N), blocks(K)) if square else (blocks(K), N), "e4m3", 4, 2.0 ** -42)
    D = torch.full((M, N), 7.0, device="cuda")
    tcg.gemm_f8(tcg.IN_E4M3, M, N, K, A, tcg.K_MAJOR, A.shape[1], SA, M, B, tcg.K_MAJOR, B.shape[1], SB, SB.shape[1], square,
                D, tcg.F32, N)
    ok(tcg)
    x, y = a * along(sa, K).T, b * (spread(sb, N, K) if square else along(sb, K).T)
    S = tau(K) * (np.abs(x) @ np.abs(y).T) + 2.0 ** -150 * (1 + tau(K)) * (np.abs(a) @ np.abs(b).T)
    close(to_host(D), x @ y.T, S, 1.0, "f32")
