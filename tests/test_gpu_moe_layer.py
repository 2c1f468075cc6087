"""The mixture-of-experts layer of examples/moe_layer.py, whose operators run
together: forward and every gradient against a 64-bit layer, gradients against
differences, and decoding with 4-bit experts."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from moe_cases import E2M1

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def moe():
    spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def silu(h):
    return h / (1.0 + np.exp(-h))


def plain(x, expert, weight, w1, w2):
    """y of the layer, float64; experts outside [0, E) are dropped."""
    y = np.zeros((x.shape[0], w2.shape[1]))
    for t in range(x.shape[0]):
        for j, e in enumerate(expert[t]):
            if 0 <= e < w1.shape[0]:
                y[t] += weight[t, j] * (w2[e] @ silu(w1[e] @ x[t]))
    return y


def inputs(moe, T, H, I, E, topk, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed)
    draw = lambda *s: (torch.randn(s, generator=gen) * s[-1] ** -0.5).to(dtype).cuda()  # noqa: E731
    layer = moe.MoeLayer(draw(E, H), draw(E, I, H), draw(E, H, I), topk)
    x = torch.randn(T, H, generator=gen).to(dtype).cuda()
    expert, weight = layer.choose(x)
    return layer, x, expert, weight


def host(t):
    return t.double().cpu().numpy()


def near(got, ref, u):
    """Every stored intermediate rounds once (u of its size), five at most one
    after the other; what they feed is bounded by its norm."""
    err = np.linalg.norm(got - ref) / np.linalg.norm(ref)
    assert err <= 5 * u, err


@pytest.mark.parametrize("T,H,I,E,topk,dtype", [
    (1, 64, 32, 4, 2, torch.bfloat16), (37, 128, 96, 8, 3, torch.float16), (300, 256, 128, 16, 4, torch.bfloat16)])
def test_training_step(moe, T, H, I, E, topk, dtype):
    layer, x, expert, weight = inputs(moe, T, H, I, E, topk, dtype)
    if T > 1:
        expert[T // 2] = -1       # a padding token
        expert[0, 0] = E          # an expert that is held elsewhere
    y, kept = layer.forward(x, expert, weight)
    dy = torch.randn(T, H, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    dx, dweight, dw1, dw2 = layer.backward(dy, kept)
    u = 2.0 ** -8 if dtype is torch.bfloat16 else 2.0 ** -11
    x64, w1, w2, p, e, g = (host(v) for v in (x, layer.w1, layer.w2, weight, expert, dy))
    e = e.astype(int)
    near(host(y), plain(x64, e, p, w1, w2), u)
    # the formulas' gradients
    rx, rp, r1, r2 = np.zeros_like(x64), np.zeros_like(p), np.zeros_like(w1), np.zeros_like(w2)
    for t in range(T):
        for j, k in enumerate(e[t]):
            if not 0 <= k < E:
                continue
            h = w1[k] @ x64[t]
            s = 1.0 / (1.0 + np.exp(-h))
            rp[t, j] = g[t] @ (w2[k] @ (h * s))
            dys = p[t, j] * g[t]
            r2[k] += np.outer(dys, h * s)
            dh = (w2[k].T @ dys) * s * (1 + h * (1 - s))
            r1[k] += np.outer(dh, x64[t])
            rx[t] += w1[k].T @ dh
    for got, ref in ((dx, rx), (dweight, rp), (dw1, r1), (dw2, r2)):
        near(host(got), ref, u)
    if T > 1:
        assert not host(y)[T // 2].any() and not host(dx)[T // 2].any() and not host(dweight)[T // 2].any()
    # and differences of the 64-bit layer along a random direction of all inputs
    rng = np.random.default_rng(2)
    d = [rng.standard_normal(v.shape) for v in (x64, p, w1, w2)]
    eps = 1e-5
    up = plain(x64 + eps * d[0], e, p + eps * d[1], w1 + eps * d[2], w2 + eps * d[3])
    down = plain(x64 - eps * d[0], e, p - eps * d[1], w1 - eps * d[2], w2 - eps * d[3])
    slope = ((up - down) * g).sum() / (2 * eps)
    parts = [(host(got), v) for got, v in zip((dx, dweight, dw1, dw2), d)]
    size = np.sqrt(sum((a ** 2).sum() for a, _ in parts))
    assert abs(sum((a * v).sum() for a, v in parts) - slope) <= 5 * u * size * 4  # 4 deviations of a unit direction


def test_decoding_with_4_bit_experts(moe):
    T, H, I, E, topk = 5, 256, 512, 8, 2
    layer, x, expert, weight = inputs(moe, T, H, I, E, topk, torch.bfloat16)
    decoder = moe.MoeDecoder(layer)

    def decoded(w):
        codes, scale, alpha = w
        c = codes.cpu().numpy()
        v = np.stack([E2M1[c & 15], E2M1[c >> 4]], axis=-1).reshape(c.shape[0], c.shape[1], -1)
        s = scale.view(torch.float8_e4m3fn).float().double().cpu().numpy()
        return v * np.repeat(s, 16, axis=2) * host(alpha)[:, None, None]

    w1, w2 = decoded(decoder.w1), decoded(decoder.w2)
    # a code is within half the widest step of E2M1, and the scale within 2^-4 of its own value
    for w, q in ((layer.w1, w1), (layer.w2, w2)):
        blocks = host(w).reshape(E, -1, 16)
        off = np.abs(host(w) - q).reshape(E, -1, 16).max(axis=2)
        assert np.all(off <= np.abs(blocks).max(axis=2) * (1 / 6 + 2.0 ** -3) + 1e-3 * np.abs(blocks).max())
    y = decoder.forward(x, expert, weight)
    near(host(y), plain(host(x), expert.cpu().numpy(), host(weight), w1, w2), 2.0 ** -8)
