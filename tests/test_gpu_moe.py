"""Routing of tokens to experts and back against plain 64-bit forms: the sorted
order, the copies, the weighted sum and its gradient."""
import numpy as np
import pytest
import torch

from moe_cases import DTYPE, TORCH, close, order, rows, to_host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tcg():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from blackwell_tensor_core_swizzled_gb300 import build
    build.build()
    import blackwell_tensor_core_swizzled_gb300 as m
    return m


def _ok(tcg, stream=None):
    rc = tcg.check(stream)
    assert rc == 0, tcg.last_error_string()


def choices(T, topk, E, kind, seed=0):
    rng = np.random.default_rng(seed)
    if kind == "one":            # every token chooses the same expert
        return np.full((T, topk), E - 1, np.int32)
    if kind == "masked":         # nothing kept
        return rng.choice(np.array([-1, -7, E, E + 5, 2 ** 31 - 1, -2 ** 31]), size=(T, topk)).astype(np.int32)
    e = rng.integers(0, E, size=(T, topk))
    if kind == "mixed":          # some choices outside [0, E)
        e = np.where(rng.random((T, topk)) < 0.2, rng.choice(np.array([-1, E, 2 ** 31 - 1]), size=(T, topk)), e)
    if kind == "few":            # popular experts, many without a token
        e = (e * rng.random((T, topk)) ** 6).astype(np.int64)
    return e.astype(np.int32)


def run_sort(tcg, expert, E, stream=None):
    T, topk = expert.shape
    off = torch.full((E + 1,), -99, dtype=torch.int32, device="cuda")
    pos = torch.full((T, topk), 2 ** 30, dtype=torch.int32, device="cuda")
    src = torch.full((T * topk,), -99, dtype=torch.int32, device="cuda")
    tcg.moe_sort(T, topk, E, torch.from_numpy(expert).cuda(), off, pos, src, stream=stream)
    return off, pos, src


@pytest.mark.parametrize("T,topk,E,kind", [
    (1, 1, 1, "any"), (1, 8, 128, "any"), (3, 5, 7, "mixed"), (31, 1, 1024, "any"), (1024, 1, 1024, "mixed"),
    (2048, 8, 64, "few"), (2049, 8, 64, "mixed"), (4097, 8, 1024, "any"), (1000, 6, 3, "one"), (700, 4, 9, "masked"),
    (8192, 2, 16, "any"), (16385, 1, 5, "few"), (40000, 8, 256, "mixed"), (40001, 7, 1, "mixed"),
    (30000, 8, 300, "one"), (20000, 4, 1000, "masked"), (131072, 8, 128, "few")])
def test_sort(tcg, T, topk, E, kind):
    expert = choices(T, topk, E, kind, seed=T + topk + E)
    got = run_sort(tcg, expert, E)
    _ok(tcg)
    for g, r, what in zip(got, order(expert, E), ("offsets", "position", "source")):
        assert np.array_equal(g.cpu().numpy(), r), what


def test_sort_without_tokens_writes_offsets(tcg):
    off = torch.full((6,), -3, dtype=torch.int32, device="cuda")
    tcg.moe_sort(0, 4, 5, None, off, None, None)
    _ok(tcg)
    assert off.tolist() == [0] * 6


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,topk,E,H,pad,kind", [
    (1, 1, 2, 1, 0, "any"), (5, 3, 4, 8, 8, "mixed"), (64, 8, 16, 1024, 0, "any"), (33, 6, 8, 1001, 3, "mixed"),
    (40, 2, 4, 4096, 16, "masked"), (17, 64, 8, 260, 4, "few"), (300, 4, 32, 520, 0, "mixed"),
    (2, 8, 8, 16392, 0, "any")])
def test_dispatch_and_back(tcg, dtype, T, topk, E, H, pad, kind):
    """Copies are exact; the weighted sum and its gradient follow the formulas
    (sums of topk, of H terms in fp32: one rounding of 2^-24 a term and one for
    each product)."""
    expert = choices(T, topk, E, kind, seed=H)
    _, position, _ = order(expert, E)
    pos = torch.from_numpy(position).cuda()
    kept = position >= 0
    prow = np.where(kept, position, -1 - position)
    d, td = DTYPE[dtype], TORCH[dtype]
    n = T * topk
    # dispatch
    X, x = rows((T, H), dtype, 1, pad)
    Xs = torch.full((n, H + pad), 7.0, dtype=td, device="cuda")
    tcg.moe_dispatch(d, T, topk, H, X, H + pad, pos, Xs, H + pad)
    _ok(tcg)
    ref = np.zeros((n, H))
    ref[prow[kept]] = np.broadcast_to(x[:, None], (T, topk, H))[kept]
    assert np.array_equal(to_host(Xs)[:, :H], ref)
    assert bool((Xs[:, H:] == 7.0).all()), "wrote past the row"
    # combine: the rows of dropped entries hold NaN and are not read
    Ys, ys = rows((n, H), dtype, 2, pad)
    Ys[torch.from_numpy(prow[~kept].astype(np.int64)).cuda()] = float("nan")
    w = np.random.default_rng(3).standard_normal((T, topk)).astype(np.float32)
    wt = torch.from_numpy(w).cuda()
    for weight in (wt, None):
        wv = np.where(kept, w if weight is not None else 1.0, 0.0).astype(np.float64)
        Y = torch.full((T, H + pad), 7.0, dtype=td, device="cuda")
        tcg.moe_combine(d, T, topk, H, Ys, H + pad, pos, weight, Y, H + pad)
        _ok(tcg)
        terms = wv[..., None] * np.where(kept[..., None], ys[prow], 0.0)
        close(to_host(Y)[:, :H], terms.sum(1), np.abs(terms).sum(1), (topk + 1) * 2.0 ** -24, dtype, "combine")
        assert bool((Y[:, H:] == 7.0).all())
        # gradient
        dY, dy = rows((T, H), dtype, 4, pad)
        dYs = torch.full((n, H + pad), 7.0, dtype=td, device="cuda")
        dw = torch.full((T, topk), 7.0, dtype=torch.float32, device="cuda")
        tcg.moe_combine_grad(d, T, topk, H, dY, H + pad, Ys, H + pad, pos, weight, dYs, H + pad, dw)
        _ok(tcg)
        ref = np.zeros((n, H))
        ref[prow[kept]] = (wv[..., None] * dy[:, None])[kept]
        close(to_host(dYs)[:, :H], ref, np.abs(ref), 2.0 ** -24, dtype, "dYs")
        assert bool((dYs[:, H:] == 7.0).all())
        prod = np.where(kept[..., None], dy[:, None] * ys[prow], 0.0)
        close(to_host(dw), prod.sum(2), np.abs(prod).sum(2), (H + 1) * 2.0 ** -24, "f32", "dweight")
        # without the weights' gradient
        dYs2 = torch.full_like(dYs, 7.0)
        tcg.moe_combine_grad(d, T, topk, H, dY, H + pad, None, 0, pos, weight, dYs2, H + pad, None)
        _ok(tcg)
        assert torch.equal(dYs2, dYs)


def test_gradient_against_differences(tcg):
    """Small integers keep every step exact, so the gradient equals the
    differences of L = <dY, combine(Ys, w)> exactly (it is bilinear)."""
    T, topk, E, H = 6, 3, 5, 24
    expert = choices(T, topk, E, "mixed", seed=5)
    _, position, _ = order(expert, E)
    pos = torch.from_numpy(position).cuda()
    rng = np.random.default_rng(6)
    n = T * topk

    def ints(*s):
        return torch.from_numpy(rng.integers(-3, 4, size=s)).float().cuda()
    Ys, w, dY = ints(n, H), ints(T, topk), ints(T, H)

    def loss(ys, wt):
        Y = torch.empty(T, H, device="cuda")
        tcg.moe_combine(tcg.F32, T, topk, H, ys, H, pos, wt, Y, H)
        return float((Y * dY).double().sum())
    dYs, dw = torch.empty(n, H, device="cuda"), torch.empty(T, topk, device="cuda")
    tcg.moe_combine_grad(tcg.F32, T, topk, H, dY, H, Ys, H, pos, w, dYs, H, dw)
    base = loss(Ys, w)
    for i in range(n):
        w2 = w.clone()
        w2.view(-1)[i] += 2
        assert loss(Ys, w2) - base == 2 * float(dw.view(-1)[i])
        y2 = Ys.clone()
        y2[i, (5 * i) % H] += 2
        assert loss(y2, w) - base == 2 * float(dYs[i, (5 * i) % H])
    # dispatch: <dXs, dispatch(X)> moves with X by combine(dXs, no weights)
    X, dXs = ints(T, H), ints(n, H)

    def loss_x(x):
        Xs = torch.empty(n, H, device="cuda")
        tcg.moe_dispatch(tcg.F32, T, topk, H, x, H, pos, Xs, H)
        return float((Xs * dXs).double().sum())
    dX = torch.empty(T, H, device="cuda")
    tcg.moe_combine(tcg.F32, T, topk, H, dXs, H, pos, None, dX, H)
    for t in range(T):
        x2 = X.clone()
        x2[t, t] += 2
        assert loss_x(x2) - loss_x(X) == 2 * float(dX[t, t])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_unaligned_bases(tcg, dtype):
    """Bases one element past a 16-byte boundary, rows of even and odd length."""
    T, topk, E = 9, 2, 4
    expert = choices(T, topk, E, "mixed", seed=8)
    _, position, _ = order(expert, E)
    pos = torch.from_numpy(position).cuda()
    kept, prow = position >= 0, np.where(position >= 0, position, -1 - position)
    for H in (64, 65):
        buf = torch.randn(T * H + 1, device="cuda").to(TORCH[dtype])
        X = buf[1:].view(T, H)
        out = torch.full((T * topk * H + 1,), 7.0, dtype=TORCH[dtype], device="cuda")
        Xs = out[1:].view(T * topk, H)
        tcg.moe_dispatch(DTYPE[dtype], T, topk, H, X, H, pos, Xs, H)
        ref = np.zeros((T * topk, H))
        ref[prow[kept]] = np.broadcast_to(to_host(X)[:, None], (T, topk, H))[kept]
        assert np.array_equal(to_host(Xs), ref) and float(out[0]) == 7.0
        back = torch.empty(T * H + 1, dtype=TORCH[dtype], device="cuda")[1:].view(T, H)
        tcg.moe_combine(DTYPE[dtype], T, topk, H, Xs, H, pos, None, back, H)
        want = to_host(X) * kept.sum(1)[:, None]      # at most twice the value: exact
        assert np.array_equal(to_host(back), want)


def test_offsets_past_32_bits(tcg):
    """Sorted rows beyond 2^32 bytes and 2^31 elements."""
    T, topk, E, H = 34000, 8, 16, 8192
    assert T * topk * H > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(1)
    expert = torch.randint(0, E, (T, topk), generator=g, device="cuda", dtype=torch.int32)
    off, pos, src = run_sort(tcg, expert.cpu().numpy(), E)
    X = torch.randn(T, H, generator=g, device="cuda", dtype=torch.bfloat16)
    Xs = torch.empty(T * topk, H, device="cuda", dtype=torch.bfloat16)
    tcg.moe_dispatch(tcg.BF16, T, topk, H, X, H, pos, Xs, H)
    _ok(tcg)
    for p in (0, 1, T * topk // 2, T * topk - 2, T * topk - 1):
        assert torch.equal(Xs[p], X[int(src[p]) // topk])
    w = torch.full((T, topk), 0.125, device="cuda")
    Y = torch.empty_like(X)
    tcg.moe_combine(tcg.BF16, T, topk, H, Xs, H, pos, w, Y, H)
    _ok(tcg)
    assert torch.equal(Y, X)                          # eight exact eighths
    dw = torch.empty_like(w)
    dYs = torch.empty_like(Xs)
    tcg.moe_combine_grad(tcg.BF16, T, topk, H, X, H, Xs, H, pos, w, dYs, H, dw)
    _ok(tcg)
    for p in (0, T * topk - 1):
        assert torch.equal(dYs[p].float(), X[int(src[p]) // topk].float() * 0.125)
    norm = (X.float() ** 2).sum(1)
    assert float(((dw - norm[:, None]).abs() / norm[:, None]).max()) < 2 * (H + 1) * 2.0 ** -24


def test_special_values_travel(tcg):
    """Infinities and NaN of kept rows arrive; a zero weight on a NaN row is
    NaN, as the sum says; dropped entries stay out."""
    pos = torch.tensor([[0, -3], [1, -4]], dtype=torch.int32, device="cuda")
    Ys = torch.zeros(4, 16, device="cuda")
    Ys[0, 0], Ys[0, 1], Ys[2], Ys[3] = float("inf"), float("nan"), float("nan"), float("inf")
    Ys[1] = float("nan")
    w = torch.tensor([[2.0, float("nan")], [0.0, 1.0]], device="cuda")
    Y = torch.empty(2, 16, device="cuda")
    tcg.moe_combine(tcg.F32, 2, 2, 16, Ys, 16, pos, w, Y, 16)
    assert float(Y[0, 0]) == float("inf") and bool(Y[0, 1].isnan()) and bool((Y[0, 2:] == 0).all())
    assert bool(Y[1].isnan().all())


def test_streams_and_graphs(tcg):
    T, topk, E, H = 3000, 8, 64, 256
    expert = choices(T, topk, E, "mixed", seed=11)
    ref = order(expert, E)
    X = torch.randn(T, H, device="cuda").bfloat16()
    ex = torch.from_numpy(expert).cuda()
    off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    pos = torch.empty(T, topk, dtype=torch.int32, device="cuda")
    src = torch.empty(T * topk, dtype=torch.int32, device="cuda")
    Xs, Y = torch.empty(T * topk, H, device="cuda").bfloat16(), torch.empty_like(X)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()

    def step():
        tcg.moe_sort(T, topk, E, ex, off, pos, src, stream=s)
        tcg.moe_dispatch(tcg.BF16, T, topk, H, X, H, pos, Xs, H, stream=s)
        tcg.moe_combine(tcg.BF16, T, topk, H, Xs, H, pos, None, Y, H, stream=s)
    with torch.cuda.stream(s):
        step()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step()
    want = Y.clone()
    for t in (off, pos, src):
        t.fill_(-5)
    Y.zero_()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    for g, r in zip((off, pos, src), ref):
        assert np.array_equal(g.cpu().numpy(), r)
    assert torch.equal(Y, want)
