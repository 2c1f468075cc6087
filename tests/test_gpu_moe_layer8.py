"""The 8-bit mixture-of-experts layer of examples/moe_layer.py, whose operators run
together (sort, dispatch, quantiser, grouped products, combine): forward and
every gradient against a 64-bit layer with the decoded experts, gradients against
differences, and decoding by the few-token kernels."""
import numpy as np
import pytest
import torch

from f8_cases import spread, values
from test_gpu_moe_layer import host, inputs, moe, near, plain  # noqa: F401

pytestmark = pytest.mark.gpu


def decoded(codes):
    return values(codes.q, "e4m3") * spread(host(codes.scale), *codes.q.shape[1:])


@pytest.mark.parametrize("T,H,I,E,topk,dtype", [
    (1, 128, 256, 4, 2, torch.bfloat16), (40, 256, 128, 8, 3, torch.float16), (700, 384, 256, 6, 4, torch.bfloat16)])
def test_training_step(moe, T, H, I, E, topk, dtype):  # noqa: F811
    layer, x, expert, weight = inputs(moe, T, H, I, E, topk, dtype)
    if T > 1:
        expert[T // 2] = -1       # a padding token
        expert[0, 0] = E          # an expert that is held elsewhere
    layer8 = moe.MoeLayer8(layer)
    w1, w2 = decoded(layer8.w1), decoded(layer8.w2)
    for w, q in ((layer.w1, w1), (layer.w2, w2)):
        # a code is within half a step, 2^-4 of its value, or half the smallest step, 2^-10, of its scale
        # (which is the largest value of 128 x 128 over 448)
        blocks = np.abs(host(w)).reshape(E, w.shape[1] // 128, 128, w.shape[2])
        top = np.stack([blocks[..., i:i + 128].max(axis=(2, 3)) for i in range(0, w.shape[2], 128)], axis=2)
        assert np.all(np.abs(host(w) - q) <= 2.0 ** -4 * np.abs(host(w)) * (1 + 2.0 ** -20)
                      + spread(top, *w.shape[1:]) / 448 * 2.0 ** -10 * (1 + 2.0 ** -20))
    y, kept = layer8.forward(x, expert, weight)
    dy = torch.randn(T, H, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    dx, dweight, dw1, dw2 = layer8.backward(dy, kept)
    x64, p, e, g = (host(v) for v in (x, weight, expert, dy))
    e = e.astype(int)
    # rows in 8 bits round once each, 2^-4 of their size; five such roundings at most one after the other
    u = 2.0 ** -4
    near(host(y), plain(x64, e, p, w1, w2), u)
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
    # and differences of the 64-bit layer along the gradients themselves
    d = [host(v) for v in (dx, dweight, dw1, dw2)]
    size = np.sqrt(sum((v ** 2).sum() for v in d))
    eps = 1e-4 / max(np.abs(v).max() for v in d)
    up = plain(x64 + eps * d[0], e, p + eps * d[1], w1 + eps * d[2], w2 + eps * d[3])
    down = plain(x64 - eps * d[0], e, p - eps * d[1], w1 - eps * d[2], w2 - eps * d[3])
    slope = ((up - down) * g).sum() / (2 * eps)
    assert abs(slope - size ** 2) <= 5 * u * size ** 2


@pytest.mark.parametrize("T", [1, 8, 37, 64])
def test_decoding(moe, T):  # noqa: F811
    layer, x, expert, weight = inputs(moe, T, 256, 384, 8, 2, torch.bfloat16)
    layer8 = moe.MoeLayer8(layer)
    y = layer8.decode(x, expert, weight)
    # x as it is, sums in fp32, one rounding
    near(host(y), plain(host(x), expert.cpu().numpy(), host(weight), decoded(layer8.w1), decoded(layer8.w2)), 2.0 ** -8)


def test_captured_step_equals_the_eager_one(moe):  # noqa: F811
    """Every operator of the 8-bit layer in one graph, forward, back and decoding,
    each reading what the one before wrote: bit for bit the eager results, on new
    inputs too."""
    T, H, I, E, topk = 200, 256, 384, 6, 2
    layer, x, expert, weight = inputs(moe, T, H, I, E, topk, torch.bfloat16)
    layer8 = moe.MoeLayer8(layer)
    dy = torch.randn(T, H, generator=torch.Generator().manual_seed(2)).to(x.dtype).cuda()

    def step():
        y, kept = layer8.forward(x, expert, weight)
        return (y, *layer8.backward(dy, kept), layer8.decode(x[:16], expert[:16], weight[:16]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for seed in range(4):
        g = torch.Generator().manual_seed(10 + seed)
        x.copy_(torch.randn(T, H, generator=g))
        dy.copy_(torch.randn(T, H, generator=g))
        expert.copy_(torch.randint(-1, E + 1, (T, topk), generator=g))
        weight.copy_(torch.rand(T, topk, generator=g))
        want = [t.clone() for t in step()]
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
