"""A mixture-of-experts layer for a few tokens, in two kernels, against float64.

Tolerance (first order; u = 2^-24): products of weights and x are exact in fp32;
a sum of H of them makes at most H roundings of 2u of the sum of magnitudes (the
tensor core may truncate) and a few more for scales and partial sums.  The
activation passes that on (|silu'| <= 1.1) and adds some 8 roundings of its own;
h = hi + lo leaves 2^-16 (bf16) or 2^-22 (f16) of it, and f16 below its smallest
values 2^-25.  The second sum adds its own roundings, then Y is rounded once."""
import numpy as np
import pytest
import torch

from f8_cases import blocks, codes, scales, spread
from moe_cases import DTYPE, IN_TYPE, TORCH, close, rows, to_host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tcg():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from blackwell_tensor_core_swizzled_gb300 import build
    build.build()
    import blackwell_tensor_core_swizzled_gb300 as m
    return m


def silu(g):
    return g / (1.0 + np.exp(-g))


def layer(x, expert, weight, w1, w3, w2, dtype):
    """Y, and a bound of what fp32 may lose of it."""
    T, H = x.shape
    E, I, _ = w1.shape
    u = 2.0 ** -24
    kept, tiny = (2.0 ** -16, 0.0) if dtype == "bf16" else (2.0 ** -22, 2.0 ** -25)
    y, off = np.zeros((T, w2.shape[1])), np.zeros((T, w2.shape[1]))
    for t in range(T):
        for e in sorted(set(int(v) for v in expert[t] if 0 <= v < E)):
            w = weight[t][expert[t] == e].sum()
            g, dg = w1[e] @ x[t], 2 * u * (H + 24) * (np.abs(w1[e]) @ np.abs(x[t]))
            h, dh = silu(g), 1.1 * dg
            if w3 is not None:
                v, dv = w3[e] @ x[t], 2 * u * (H + 24) * (np.abs(w3[e]) @ np.abs(x[t]))
                h, dh = h * v, dh * np.abs(v) + np.abs(h) * dv + dh * dv
            h, dh = w * h, np.abs(w) * dh
            dh = dh + (16 * u + kept) * np.abs(h) + tiny
            y[t] += w2[e] @ h
            off[t] += np.abs(w2[e]) @ dh + 2 * u * (2 * I + 24 + 2 * expert.size) * (np.abs(w2[e]) @ np.abs(h))
    return y, off


class Case:
    def __init__(self, T, topk, E, H, I, dtype, weights, gated, seed=0, pad=0, scale=1.0):
        self.T, self.topk, self.E, self.H, self.I = T, topk, E, H, I
        self.dtype, self.weights = dtype, weights
        rng = np.random.default_rng(seed)
        self.X, self.x = rows((T, H), dtype, seed + 1, 8 * pad, scale)
        self.expert = rng.integers(0, E, (T, topk)).astype(np.int32)   # the same expert twice, now and then
        self.weight = rng.random((T, topk)).astype(np.float32)
        self.s, self.w, self.W, self.S = {}, {}, {}, {}
        for i, (name, n, k) in enumerate((("1", I, H), ("3", I, H), ("2", H, I))):
            if name == "3" and not gated:
                self.W[name] = self.S[name] = self.w[name] = None
                continue
            if weights == "e4m3":
                self.W[name], c = codes((E, n, k), "e4m3", seed + 2 + i, pad)
                self.S[name], sc = scales((E, blocks(n), blocks(k)), "e4m3", seed + 5 + i, k ** -0.5, pad)
                self.w[name] = c * spread(sc, n, k)
            else:
                self.W[name], self.w[name] = rows((E, n, k), weights, seed + 2 + i, -k % 8 + 8 * pad, k ** -0.5)
                self.S[name] = None

    def run(self, tcg, out="f32", Y=None, ldy=None, expert=None, stream=None, work=None, weight=True, W=None):
        E, T = self.E, self.T
        ldy = ldy or self.H
        if Y is None:
            Y = torch.full((T, ldy), 7.0, dtype=TORCH[out], device="cuda")
        if expert is None:
            expert = torch.from_numpy(self.expert).cuda()
        if work is None:
            work = torch.full((tcg.moe_few_work_bytes(T, self.topk, self.I),), 0xFF, dtype=torch.uint8, device="cuda")
        self.alive = expert, torch.from_numpy(self.weight).cuda() if W is None else W, work
        s = lambda n: dict(ld=0 if self.S[n] is None else self.S[n].shape[2])["ld"]  # noqa: E731
        tcg.moe_few(IN_TYPE[self.dtype], 3 if self.weights == "e4m3" else IN_TYPE[self.dtype], T, self.H, self.I,
                    self.topk, E, self.X, self.X.shape[1], expert, self.alive[1] if weight else None, self.W["1"],
                    self.W["3"], self.W["2"], work, Y, DTYPE[out], ldy, s1=self.S["1"], s3=self.S["3"], s2=self.S["2"],
                    ld1=self.W["1"].shape[2], ld2=self.W["2"].shape[2], ld_s1=s("1"), ld_s2=s("2"), stream=stream)
        return Y

    def reference(self, weight=True):
        w = self.weight.astype(np.float64) if weight else np.ones_like(self.weight, dtype=np.float64)
        return layer(self.x, self.expert, w, self.w["1"], self.w["3"], self.w["2"], self.dtype)

    def check(self, tcg, out="f32", **kw):
        Y = self.run(tcg, out, **kw)
        rc = tcg.check()
        assert rc == 0, tcg.last_error_string()
        y, off = self.reference(kw.get("weight", True))
        close(to_host(Y)[:, :self.H], y, off, 1.0, out, (self.T, self.topk, self.E, self.H, self.I))
        assert bool((Y[:, self.H:] == 7.0).all()), "wrote past the row"


SIZES = [
    # tokens, topk, experts, H, I
    (1, 1, 1, 16, 16),
    (1, 8, 128, 256, 128),
    (3, 2, 4, 48, 80),
    (8, 4, 16, 1040, 144),
    (9, 3, 5, 128, 1024),
    (16, 2, 1000, 144, 48),
    (17, 2, 3, 2064, 272),
    (33, 6, 8, 272, 1040),
    (64, 8, 16, 512, 96),
    (64, 1, 1, 64, 32),
]


@pytest.mark.parametrize("dtype,weights", [("bf16", "e4m3"), ("f16", "e4m3"), ("bf16", "bf16"), ("f16", "f16")])
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("T,topk,E,H,I", SIZES)
def test_layer(tcg, dtype, weights, gated, T, topk, E, H, I):
    c = Case(T, topk, E, H, I, dtype, weights, gated, seed=T + H, pad=T % 3)
    if T > 2:
        c.expert[1] = -1                  # a padding token
        c.expert[2, 0] = E                # an expert that is held elsewhere
        c.expert[T - 1] = c.expert[T - 1, 0]  # one expert many times
    c.check(tcg, "f32", ldy=H + 3)
    c.check(tcg, dtype)


@pytest.mark.parametrize("weights", ["e4m3", "bf16"])
def test_all_tokens_choose_one_expert(tcg, weights):
    c = Case(64, 2, 7, 256, 256, "bf16", weights, True, seed=4)
    c.expert[:] = 5
    c.check(tcg)


def test_no_choice_kept(tcg):
    c = Case(5, 2, 4, 64, 64, "bf16", "e4m3", True)
    c.expert[:] = -1
    Y = c.run(tcg)
    assert tcg.check() == 0
    assert not to_host(Y).any()


def test_without_weights_and_without_inner(tcg):
    c = Case(4, 2, 6, 64, 48, "f16", "f16", True, seed=2)
    c.check(tcg, weight=False)
    Y = torch.full((4, 64), 7.0, device="cuda")
    tcg.moe_few(tcg.IN_F16, tcg.IN_F16, 4, 64, 0, 2, 6, None, 0, torch.from_numpy(c.expert).cuda(), None, None, None,
                None, None, Y, tcg.F32, 64)
    assert tcg.check() == 0
    assert not to_host(Y).any()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_every_code_is_decoded(tcg, dtype):
    """W2 holds all codes in turn, h is one for the first inner row alone."""
    H, I = 256, 16
    c = Case(1, 1, 1, H, I, dtype, "e4m3", False, seed=1)
    c.X.zero_()
    c.X[0, 0] = c.x[0, 0] = 1.0
    c.x[0, 1:] = 0
    w1 = torch.zeros(1, I, H)
    w1[0, 0, 0] = 448.0
    c.W["1"], c.w["1"] = w1.to(torch.float8_e4m3fn).view(torch.uint8).cuda(), w1.double().numpy()
    c.S["1"] = torch.ones(1, 1, 2, device="cuda")
    c.S["2"] = torch.ones(1, 2, 1, device="cuda")
    w2 = torch.zeros(1, H, I, dtype=torch.uint8)
    w2[0, :, 0] = torch.arange(256).to(torch.uint8)
    c.W["2"] = w2.cuda()
    c.weight[:] = 1
    c.expert[:] = 0
    Y = to_host(c.run(tcg))[0]
    assert tcg.check() == 0
    v = w2[0, :, 0].view(torch.float8_e4m3fn).double().numpy()
    nan = np.isnan(v)
    assert np.array_equal(np.isnan(Y), nan)
    assert np.array_equal(Y[~nan], (448.0 * v)[~nan])


def test_values_of_other_experts_stay_out(tcg):
    """NaN in an expert's weights or in a token reach only the tokens that use them."""
    for weights in ("e4m3", "bf16"):
        c = Case(6, 2, 5, 128, 64, "bf16", weights, True, seed=8)
        c.expert[:] = [[0, 1], [1, 2], [0, 2], [4, 0], [2, 2], [1, 4]]
        clean = to_host(c.run(tcg))
        for n in ("1", "2"):
            c.W[n][4] = 0x7f if weights == "e4m3" else float("nan")
            c.W[n][3] = 0x7f if weights == "e4m3" else float("nan")
        c.X[4] = float("inf")
        got = to_host(c.run(tcg))
        assert tcg.check() == 0
        for t in (0, 1, 2):
            assert np.array_equal(got[t], clean[t])
        assert np.isnan(got[3]).all() and np.isnan(got[5]).all()


def test_activations_of_any_range(tcg):
    """bf16 activations far apart keep their bits against 8-bit weights."""
    c = Case(2, 1, 2, 256, 64, "bf16", "e4m3", False, seed=3)
    mag = np.exp2(np.random.default_rng(5).integers(-60, 3, c.x.shape).astype(np.float64))
    x = torch.from_numpy(c.x * mag).to(torch.bfloat16)
    c.X, c.x = x.cuda(), x.double().numpy()
    c.check(tcg)


def test_f16_beyond_its_range_is_infinite(tcg):
    c = Case(1, 1, 1, 64, 16, "f16", "f16", True, seed=6, scale=400.0)
    c.W["1"].mul_(50)
    c.W["3"].mul_(50)
    Y = to_host(c.run(tcg))
    assert tcg.check() == 0
    assert not np.isfinite(Y).all()


def test_same_result_every_time_on_two_streams(tcg):
    a = Case(20, 4, 16, 512, 256, "bf16", "e4m3", True, seed=1)
    b = Case(7, 2, 16, 256, 512, "f16", "f16", False, seed=2)
    ya, yb = a.run(tcg, "bf16").clone(), b.run(tcg, "f16").clone()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(20):
        with torch.cuda.stream(s1):
            outs.append((a.run(tcg, "bf16"), ya, a.alive))
        with torch.cuda.stream(s2):
            outs.append((b.run(tcg, "f16"), yb, b.alive))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y, _ in outs)


def test_captured_with_new_choices(tcg):
    c = Case(12, 2, 8, 256, 192, "bf16", "e4m3", True, seed=9)
    expert = torch.from_numpy(c.expert).cuda()
    work = torch.empty(tcg.moe_few_work_bytes(12, 2, 192), dtype=torch.uint8, device="cuda")
    Y, W = torch.zeros(12, 256, device="cuda"), torch.from_numpy(c.weight).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        # the choices of the graph's first kernel are the layer's
        expert.remainder_(8)
        c.run(tcg, Y=Y, expert=expert, work=work, W=W)
    for seed in range(3):
        c.expert = np.random.default_rng(seed).integers(0, 8, (12, 2)).astype(np.int32)
        expert.copy_(torch.from_numpy(c.expert + 8 * seed))
        graph.replay()
        torch.cuda.synchronize()
        assert tcg.check() == 0
        y, off = c.reference()
        close(to_host(Y), y, off, 1.0, "f32")


@pytest.mark.parametrize("weights", ["e4m3", "f16"])
@pytest.mark.parametrize("T,size", [(3, 2.0 ** -7), (3, 2.0 ** -11), (21, 2.0 ** -9)])
def test_small_f16_activations_keep_their_bits(tcg, weights, T, size):
    """Weights of the choices so small that w h lies below f16's normal range.  hi
    leaves at most 2^-11 of it or 2^-25, lo = 2^11 times that 2^-11 of the rest or
    2^-25: 2^-22 of w h or 2^-36."""
    c = Case(T, 2, 4, 256, 192, "f16", weights, True, seed=T, scale=0.1)
    c.weight *= np.float32(size)
    if weights == "e4m3":
        c.S["2"] *= 4096            # scales that bring y back
        c.w["2"] = c.w["2"] * 4096
    Y = c.run(tcg, "f32")
    assert tcg.check() == 0, tcg.last_error_string()
    y, off = c.reference()
    for t in range(T):              # the bound above instead of the layer's 2^-25
        for e in set(c.expert[t].tolist()):
            off[t] -= (2.0 ** -25 - 2.0 ** -36) * np.abs(c.w["2"][e]).sum(axis=1)
    close(to_host(Y), y, off, 1.0, "f32", (weights, T))


@pytest.mark.parametrize("dtype,weights", [("bf16", "e4m3"), ("f16", "f16")])
@pytest.mark.parametrize("T", [2, 24])
def test_experts_and_their_scales_apart(tcg, dtype, weights, T):
    """Experts inside larger buffers: strides between matrices and between scales
    beyond the packed ones, NaN between them."""
    c = Case(T, 2, 5, 272, 144, dtype, weights, True, seed=11)
    want = to_host(c.run(tcg, "f32"))
    stride = {}

    def apart(t, more, fill):
        if t is None:
            return None, 0
        E, n, k = t.shape
        big = torch.full((E, n * k + more), fill, dtype=t.dtype, device="cuda")
        big[:, :n * k] = t.reshape(E, n * k)
        return big, n * k + more
    for name, W in c.W.items():
        ld = W.shape[2]
        more = 16 * (3 if name == "2" else 5)
        big, stride[name] = apart(W, more, 0x7f if weights == "e4m3" else float("nan"))
        S, stride["s" + name] = apart(c.S[name], 7 if name == "2" else 3, float("nan"))
        c.W[name], c.S[name] = (big, ld), (S, 0 if c.S[name] is None else c.S[name].shape[2])
    expert, weight = torch.from_numpy(c.expert).cuda(), torch.from_numpy(c.weight).cuda()
    work = torch.full((tcg.moe_few_work_bytes(T, 2, c.I),), 0xFF, dtype=torch.uint8, device="cuda")
    Y = torch.full((T, c.H), 7.0, device="cuda")
    tcg.moe_few(IN_TYPE[dtype], 3 if weights == "e4m3" else IN_TYPE[dtype], T, c.H, c.I, 2, 5, c.X, c.X.shape[1], expert,
                weight, c.W["1"][0], c.W["3"][0], c.W["2"][0], work, Y, tcg.F32, c.H, s1=c.S["1"][0], s3=c.S["3"][0],
                s2=c.S["2"][0], ld1=c.W["1"][1], stride1=stride["1"], ld2=c.W["2"][1], stride2=stride["2"],
                ld_s1=c.S["1"][1], stride_s1=stride["s1"], ld_s2=c.S["2"][1], stride_s2=stride["s2"])
    assert tcg.check() == 0, tcg.last_error_string()
    assert np.array_equal(to_host(Y), want)
