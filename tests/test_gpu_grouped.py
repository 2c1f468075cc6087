"""Products of sorted rows with their group's matrix and the matrices' gradient
against float64, at sizes that cut tiles, with empty groups and loose rows.

Tolerance: products of 16-bit values are exact in fp32, and a sum of K of them
makes at most K roundings of 2^-23 relative to the sum of magnitudes (the
tensor core may truncate), so |error| <= K 2^-23 sum |a b| before the rounding
to the stored type."""
import numpy as np
import pytest
import torch

from moe_cases import DTYPE, IN_TYPE, TORCH, close, group_offsets, rows, to_host

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


def pad_to(n, extra=0):
    """Padding that makes a row of n elements a multiple of 8, plus `extra` octets."""
    return -n % 8 + 8 * extra


CASES = [
    # sizes of the groups, loose rows before and after, N, K, B rows padded by
    ([1], 0, 0, 8, 8, 0),
    ([5], 0, 0, 1, 1, 0),
    ([0, 3, 0, 0, 130, 1, 0], 0, 0, 264, 72, 1),
    ([128, 128, 256], 0, 0, 256, 128, 0),
    ([17, 33, 64, 65, 127, 129], 0, 5, 200, 136, 0),
    ([700, 0, 300], 3, 4, 130, 520, 1),
    ([0, 0, 0], 0, 9, 72, 64, 0),
    ([257, 255, 513], 0, 0, 513, 1000, 0),
    ([3] * 40, 1, 1, 384, 192, 0),
    ([1, 2, 4, 8, 16, 31, 32, 48], 0, 0, 1030, 2056, 0),
    ([2100], 0, 0, 300, 64, 0),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("major", ["k", "mn"])
@pytest.mark.parametrize("sizes,before,after,N,K,extra", CASES)
def test_grouped(tcg, dtype, major, sizes, before, after, N, K, extra):
    G, R = len(sizes), sum(sizes) + before + after
    off = group_offsets(sizes, before)
    A, a = rows((R, K), dtype, 1, pad_to(K, 1))
    shape = (G, N, K) if major == "k" else (G, K, N)
    B, b = rows(shape, dtype, 2, pad_to(shape[2], extra))
    if major == "mn":
        b = b.transpose(0, 2, 1)
    for out in (dtype, "f32") if sizes != [2100] else ("bf16",):
        D = torch.full((R, N + 3), 7.0, dtype=TORCH[out], device="cuda")
        tcg.gemm_grouped(IN_TYPE[dtype], R, N, K, G, A, A.shape[1], torch.from_numpy(off).cuda(), B,
                         tcg.K_MAJOR if major == "k" else tcg.MN_MAJOR, B.shape[2], 0, D, DTYPE[out], N + 3)
        _ok(tcg)
        ref, S = np.zeros((R, N)), np.zeros((R, N))
        for g in range(G):
            sl = slice(off[g], off[g + 1])
            ref[sl], S[sl] = a[sl] @ b[g].T, np.abs(a[sl]) @ np.abs(b[g].T)
        close(to_host(D)[:, :N], ref, S, K * 2.0 ** -23, out, (major, out))
        assert bool((D[:, N:] == 7.0).all()), "wrote past the row"


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("sizes,before,after,N,K,extra", CASES)
def test_wgrad(tcg, dtype, sizes, before, after, N, K, extra):
    G, R = len(sizes), sum(sizes) + before + after
    off = group_offsets(sizes, before)
    DY, dy = rows((R, N), dtype, 3, pad_to(N, extra))
    A, a = rows((R, K), dtype, 4, pad_to(K, 1))
    for out in (dtype, "f32"):
        DW = torch.full((G, N, K + 5), 7.0, dtype=TORCH[out], device="cuda")
        tcg.gemm_grouped_wgrad(IN_TYPE[dtype], R, N, K, G, DY, DY.shape[1], A, A.shape[1],
                               torch.from_numpy(off).cuda(), DW, DTYPE[out], K + 5, 0)
        _ok(tcg)
        ref, S = np.zeros((G, N, K)), np.zeros((G, N, K))
        for g in range(G):
            sl = slice(off[g], off[g + 1])
            ref[g], S[g] = dy[sl].T @ a[sl], np.abs(dy[sl]).T @ np.abs(a[sl])
        close(to_host(DW)[:, :, :K], ref, S, max(sizes) * 2.0 ** -23, out, out)
        assert bool((DW[:, :, K:] == 7.0).all())


def test_gradients_against_differences(tcg):
    """Small integers: every sum is exact, so the gradients equal differences
    of L = <DY, grouped(A, B)> exactly (it is bilinear)."""
    sizes, N, K = [3, 0, 20, 6], 40, 24
    G, R = len(sizes), sum(sizes)
    off = torch.from_numpy(group_offsets(sizes)).cuda()
    rng = np.random.default_rng(9)

    def ints(*s):
        return torch.from_numpy(rng.integers(-3, 4, size=s)).to(torch.bfloat16).cuda()
    A, B, DY = ints(R, K), ints(G, N, K), ints(R, N)

    def loss(a, b):
        D = torch.empty(R, N, device="cuda")
        tcg.gemm_grouped(tcg.IN_BF16, R, N, K, G, a, K, off, b, tcg.K_MAJOR, K, 0, D, tcg.F32, N)
        return float((D * DY.float()).double().sum())
    DA = torch.empty(R, K, device="cuda")
    tcg.gemm_grouped(tcg.IN_BF16, R, K, N, G, DY, N, off, B, tcg.MN_MAJOR, K, N * K, DA, tcg.F32, K)
    DW = torch.empty(G, N, K, device="cuda")
    tcg.gemm_grouped_wgrad(tcg.IN_BF16, R, N, K, G, DY, N, A, K, off, DW, tcg.F32, K, N * K)
    base = loss(A, B)
    for i in range(R):
        a2 = A.clone()
        a2[i, (7 * i) % K] += 1
        assert loss(a2, B) - base == float(DA[i, (7 * i) % K])
    for g in range(G):
        for n in (0, 17, N - 1):
            b2 = B.clone()
            b2[g, n, (n + g) % K] += 1
            assert loss(A, b2) - base == float(DW[g, n, (n + g) % K])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_other_groups_values_stay_out(tcg, bad):
    """NaN and infinities in one group's rows or matrix reach no other group,
    nor do they come back through loose rows."""
    sizes, N, K = [5, 9, 70, 3], 136, 72
    G, R = len(sizes), sum(sizes) + 4
    off = group_offsets(sizes, 2)
    t_off = torch.from_numpy(off).cuda()
    A, _ = rows((R, K), "bf16", 1)
    B, _ = rows((G, N, K), "bf16", 2)
    DY, _ = rows((R, N), "bf16", 3)
    outs = []
    for poison in (False, True):
        if poison:
            A[off[1]:off[2]] = bad
            A[:2], A[-2:], DY[:2], DY[-2:] = bad, bad, bad, bad
            B[2] = bad
            DY[off[1]:off[2]] = bad
        D = torch.empty(R, N, device="cuda")
        tcg.gemm_grouped(tcg.IN_BF16, R, N, K, G, A, K, t_off, B, tcg.K_MAJOR, K, 0, D, tcg.F32, N)
        DW = torch.empty(G, N, K, device="cuda")
        tcg.gemm_grouped_wgrad(tcg.IN_BF16, R, N, K, G, DY, N, A, K, t_off, DW, tcg.F32, K, 0)
        _ok(tcg)
        outs.append((D, DW))
    (d0, w0), (d1, w1) = outs
    for g in (0, 3):
        assert torch.equal(d0[off[g]:off[g + 1]], d1[off[g]:off[g + 1]])
    for g in (0, 2, 3):
        assert torch.equal(w0[g], w1[g])
    assert not bool(d1[off[1]:off[2]].isfinite().any()) and not bool(w1[1].isfinite().any())
    assert bool((d1[:2] == 0).all()) and bool((d1[-2:] == 0).all())


def test_wild_offsets_stay_in_range(tcg):
    """Offsets that decrease, are negative or pass R are clamped to [previous, R]."""
    R, N, K = 40, 16, 16
    A, a = rows((R, K), "bf16", 1)
    B, b = rows((4, N, K), "bf16", 2)
    off = torch.tensor([-5, 10, 4, 1000000, 7], dtype=torch.int32, device="cuda")   # 0, 10, 10, 40, 40
    D = torch.empty(R, N, device="cuda")
    tcg.gemm_grouped(tcg.IN_BF16, R, N, K, 4, A, K, off, B, tcg.K_MAJOR, K, 0, D, tcg.F32, N)
    DW = torch.empty(4, N, K, device="cuda")
    tcg.gemm_grouped_wgrad(tcg.IN_BF16, R, N, K, 4, A, K, A, K, off, DW, tcg.F32, K, 0)
    _ok(tcg)
    ref = np.concatenate([a[:10] @ b[0].T, a[10:] @ b[2].T])
    S = np.concatenate([np.abs(a[:10]) @ np.abs(b[0].T), np.abs(a[10:]) @ np.abs(b[2].T)])
    close(to_host(D), ref, S, K * 2.0 ** -23, "f32")
    wref = np.stack([a[:10].T @ a[:10], np.zeros((N, K)), a[10:].T @ a[10:], np.zeros((N, K))])
    wS = np.stack([np.abs(a[:10]).T @ np.abs(a[:10]), np.zeros((N, K)), np.abs(a[10:]).T @ np.abs(a[10:]),
                   np.zeros((N, K))])
    close(to_host(DW), wref, wS, R * 2.0 ** -23, "f32")


def test_empty_contractions(tcg):
    off = torch.tensor([0, 3, 5], dtype=torch.int32, device="cuda")
    D = torch.full((5, 24), 7.0, device="cuda")
    tcg.gemm_grouped(tcg.IN_BF16, 5, 24, 0, 2, None, 0, off, None, tcg.K_MAJOR, 0, 0, D, tcg.F32, 24)
    DW = torch.full((2, 24, 8), 7.0, device="cuda")
    zero = torch.zeros(3, dtype=torch.int32, device="cuda")
    tcg.gemm_grouped_wgrad(tcg.IN_BF16, 0, 24, 8, 2, None, 0, None, 0, zero, DW, tcg.F32, 8, 0)
    _ok(tcg)
    assert bool((D == 0).all()) and bool((DW == 0).all())


def test_separate_matrices_and_many_groups(tcg):
    """A stride between the groups' matrices beyond N * ldb, and 1000 groups."""
    rng = np.random.default_rng(4)
    sizes = rng.integers(0, 4, size=1000)
    G, R, N, K = 1000, int(sizes.sum()), 24, 40
    off = group_offsets(sizes)
    A, a = rows((R, K), "f16", 1)
    Bfull, b = rows((G, N + 2, K), "f16", 2)
    D = torch.empty(R, N, device="cuda", dtype=torch.float16)
    tcg.gemm_grouped(tcg.IN_F16, R, N, K, G, A, K, torch.from_numpy(off).cuda(), Bfull, tcg.K_MAJOR, K,
                     (N + 2) * K, D, tcg.F16, N)
    DWfull = torch.full((G, N + 2, K), 7.0, device="cuda")
    tcg.gemm_grouped_wgrad(tcg.IN_F16, R, K, K, G, A, K, A, K, torch.from_numpy(off).cuda(),
                           torch.empty(G, K, K, device="cuda"), tcg.F32, K, 0)
    DY, dy = rows((R, N), "f16", 5)
    tcg.gemm_grouped_wgrad(tcg.IN_F16, R, N, K, G, DY, N, A, K, torch.from_numpy(off).cuda(), DWfull, tcg.F32, K,
                           (N + 2) * K)
    _ok(tcg)
    group = np.repeat(np.arange(G), sizes)
    ref = np.einsum("rk,rnk->rn", a, b[group][:, :N])
    S = np.einsum("rk,rnk->rn", np.abs(a), np.abs(b[group][:, :N]))
    close(to_host(D), ref, S, K * 2.0 ** -23, "f16")
    wref, wS = np.zeros((G, N, K)), np.zeros((G, N, K))
    np.add.at(wref, group, dy[:, :, None] * a[:, None])
    np.add.at(wS, group, np.abs(dy[:, :, None] * a[:, None]))
    close(to_host(DWfull)[:, :N], wref, wS, 4 * 2.0 ** -23, "f32")
    assert bool((DWfull[:, N:] == 7.0).all())


def test_rerun_is_identical_and_other_streams(tcg):
    sizes = [100, 0, 345, 60]
    R, N, K = sum(sizes), 520, 384
    off = torch.from_numpy(group_offsets(sizes)).cuda()
    A, _ = rows((R, K), "bf16", 1)
    B, _ = rows((4, N, K), "bf16", 2)
    DY, _ = rows((R, N), "bf16", 3)
    torch.cuda.synchronize()
    outs = []
    for st in (torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.current_stream()):
        D = torch.empty(R, N, device="cuda", dtype=torch.bfloat16)
        DW = torch.empty(4, N, K, device="cuda")
        tcg.gemm_grouped(tcg.IN_BF16, R, N, K, 4, A, K, off, B, tcg.K_MAJOR, K, 0, D, tcg.BF16, N, stream=st)
        tcg.gemm_grouped_wgrad(tcg.IN_BF16, R, N, K, 4, DY, N, A, K, off, DW, tcg.F32, K, 0, stream=st)
        outs.append((D, DW))
    torch.cuda.synchronize()
    for D, DW in outs[1:]:
        assert torch.equal(D, outs[0][0]) and torch.equal(DW, outs[0][1])


#: both kernel forms (up to 64 rows a group on average, and more), groups that
#: end inside a block of 32 columns, a last tile that is not full
ALIGNED = [
    ([40, 64, 33, 0, 100, 5], 0, 0, 264, 72),
    ([32, 48, 64, 1], 3, 2, 128, 200),
    ([257, 255, 513], 0, 0, 520, 200),
    ([700, 0, 300], 1, 6, 1032, 136),
    ([96, 160, 290], 0, 0, 264, 1032),
    ([1100], 0, 0, 40, 64),
]


def guarded_output(shape, ld, gap, dtype, guard=64):
    """A tensor of `shape` with rows of `ld` elements and `gap` elements between
    matrices, inside a buffer of sevens (16-byte aligned), and that buffer."""
    n = 1
    for d in shape[:-2]:
        n *= d
    stride = shape[-2] * ld + gap
    buf = torch.full((2 * guard + n * stride,), 7.0, dtype=TORCH[dtype], device="cuda")
    strides = (stride, ld, 1)[3 - len(shape):]
    return buf.as_strided(shape, strides, guard), buf


def untouched(view, buf):
    """Whether all of the buffer but the view still holds sevens."""
    view.fill_(7.0)
    return bool((buf == 7.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("major", ["k", "mn"])
@pytest.mark.parametrize("sizes,before,after,N,K", ALIGNED)
def test_grouped_aligned_outputs(tcg, dtype, major, sizes, before, after, N, K):
    """Output rows on 16-byte boundaries (packed and padded) and off them."""
    G, R = len(sizes), sum(sizes) + before + after
    off = group_offsets(sizes, before)
    A, a = rows((R, K), dtype, 1)
    B, b = rows((G, N, K) if major == "k" else (G, K, N), dtype, 2)
    if major == "mn":
        b = b.transpose(0, 2, 1)
    ref, S = np.zeros((R, N)), np.zeros((R, N))
    for g in range(G):
        sl = slice(off[g], off[g + 1])
        ref[sl], S[sl] = a[sl] @ b[g].T, np.abs(a[sl]) @ np.abs(b[g].T)
    for out in (dtype, "f32"):
        for pad in (0, 8, 3):
            D, buf = guarded_output((R, N), N + pad, 0, out)
            tcg.gemm_grouped(IN_TYPE[dtype], R, N, K, G, A, K, torch.from_numpy(off).cuda(), B,
                             tcg.K_MAJOR if major == "k" else tcg.MN_MAJOR, 0, 0, D, DTYPE[out], N + pad)
            _ok(tcg)
            close(to_host(D), ref, S, K * 2.0 ** -23, out, (out, pad))
            assert untouched(D, buf), (out, pad)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("sizes,before,after,N,K", ALIGNED)
def test_wgrad_aligned_outputs(tcg, dtype, sizes, before, after, N, K):
    G, R = len(sizes), sum(sizes) + before + after
    off = group_offsets(sizes, before)
    DY, dy = rows((R, N), dtype, 3)
    A, a = rows((R, K), dtype, 4)
    ref, S = np.zeros((G, N, K)), np.zeros((G, N, K))
    for g in range(G):
        sl = slice(off[g], off[g + 1])
        ref[g], S[g] = dy[sl].T @ a[sl], np.abs(dy[sl]).T @ np.abs(a[sl])
    for out in (dtype, "f32"):
        for pad, gap in ((0, 0), (8, 16), (0, 40), (3, 5)):
            DW, buf = guarded_output((G, N, K), K + pad, gap, out)
            tcg.gemm_grouped_wgrad(IN_TYPE[dtype], R, N, K, G, DY, N, A, K, torch.from_numpy(off).cuda(), DW,
                                   DTYPE[out], K + pad, DW.stride(0))
            _ok(tcg)
            close(to_host(DW), ref, S, max(sizes) * 2.0 ** -23, out, (out, pad, gap))
            assert untouched(DW, buf), (out, pad, gap)


def test_long_fp32_sums(tcg):
    """fp32 outputs of contractions of 4096 are closer than one running sum of
    the tensor core gets.  It drops what lies below its last bit at each step of
    16 terms, half a bit of 2^-23 on average and always towards zero; a sum that
    grows as a walk does loses 2/3 n 2^-24 of itself over n steps.  One sum of
    4096 (n = 256) may lose 1.0e-5; sums of at most 512 (n = 32), added in
    rounded fp32, 1.3e-6."""
    bound = 2 / 3 * 32 * 2.0 ** -24
    K, N, R = 4096, 256, 512
    A, a = rows((R, K), "bf16", 1)
    B, b = rows((2, N, K), "bf16", 2)
    off = torch.tensor([0, 200, 512], dtype=torch.int32, device="cuda")
    D = torch.empty(R, N, device="cuda")
    tcg.gemm_grouped(tcg.IN_BF16, R, N, K, 2, A, K, off, B, tcg.K_MAJOR, K, 0, D, tcg.F32, N)
    ref = np.concatenate([a[:200] @ b[0].T, a[200:] @ b[1].T])
    assert np.linalg.norm(to_host(D) - ref) <= bound * np.linalg.norm(ref)
    R = 4096 + 64
    DY, dy = rows((R, N), "bf16", 3)
    A, a = rows((R, N), "bf16", 4)
    off = torch.tensor([0, 64, R], dtype=torch.int32, device="cuda")
    DW = torch.empty(2, N, N, device="cuda")
    tcg.gemm_grouped_wgrad(tcg.IN_BF16, R, N, N, 2, DY, N, A, N, off, DW, tcg.F32, N, 0)
    _ok(tcg)
    ref = dy[64:].T @ a[64:]
    assert np.linalg.norm(to_host(DW[1]) - ref) <= bound * np.linalg.norm(ref)


def test_large_16_bit_outputs_repeat(tcg):
    """Long contractions of unequal groups, many tiles a CTA: the same inputs
    give the same bits each time, and every value is within its bound."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    sizes = [1, 2500, 700, 0, 1311, 4096, 513, 2047]
    G, R, N, K = len(sizes), sum(sizes), 2048, 4096
    off = torch.from_numpy(group_offsets(sizes)).cuda()
    A = torch.randn(R, K, generator=gen, device="cuda").bfloat16()
    B = (torch.randn(G, N, K, generator=gen, device="cuda") * K ** -0.5).bfloat16()
    outs = []
    for _ in range(6):
        D = torch.full((R, N), 7.0, device="cuda", dtype=torch.bfloat16)
        tcg.gemm_grouped(tcg.IN_BF16, R, N, K, G, A, K, off, B, tcg.K_MAJOR, K, 0, D, tcg.BF16, N)
        outs.append(D)
    _ok(tcg)
    assert all(torch.equal(D, outs[0]) for D in outs[1:])
    lo = 0
    for g, n in enumerate(sizes):
        x, w = A[lo:lo + n].double(), B[g].double()
        close(to_host(outs[0][lo:lo + n]), to_host(x @ w.T), to_host(x.abs() @ w.abs().T), K * 2.0 ** -23, "bf16", g)
        lo += n


def test_plan_is_the_last_products(tcg):
    """The plan string describes the product that was called last, dense,
    grouped or 4-bit, and is empty after one that queued nothing or failed."""
    N = K = 64
    A, B = torch.zeros(4, K, device="cuda").bfloat16(), torch.zeros(2, N, K, device="cuda").bfloat16()
    D, DW = torch.empty(4, N, device="cuda"), torch.empty(2, N, K, device="cuda")
    off = torch.tensor([0, 1, 4], dtype=torch.int32, device="cuda")
    codes, scale = torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda"), torch.zeros(
        N, K // 32, dtype=torch.uint8, device="cuda")

    def dense():
        tcg.gemm_bf16(4, N, K, A, tcg.K_MAJOR, K, B, tcg.K_MAJOR, K, D, tcg.F32, N, tcg.F32)
        assert "pass" in tcg.last_plan_string()

    def grouped(rows=4, major=tcg.K_MAJOR):
        tcg.gemm_grouped(tcg.IN_BF16, rows, N, K, 2, A, K, off, B, major, K, 0, D, tcg.F32, N)

    def wgrad():
        tcg.gemm_grouped_wgrad(tcg.IN_BF16, 4, K, K, 2, A, K, A, K, off, DW, tcg.F32, K, 0)

    def w4(k=K):
        tcg.gemv_w4(tcg.W4_MXF4, tcg.IN_BF16, 4, N, k, A, K, codes, scale, D, tcg.F32, N)
    for call, text in ((grouped, "grouped, cta_group 1"), (wgrad, "grouped, cta_group 2"), (w4, "4-bit, blocks of 4"),
                       (lambda: grouped(0), ""), (lambda: w4(0), "K = 0")):
        dense()
        call()
        plan = tcg.last_plan_string()
        assert plan.startswith(text) and bool(plan) == bool(text), plan
    dense()
    with pytest.raises(tcg.TcgError):
        grouped(major=7)
    assert tcg.last_plan_string() == ""
    _ok(tcg)
