"""A mixture-of-experts layer: a training step forward and back, and decoding
with 4-bit experts.

    y[t] = sum_j p[t, j] W2[e] silu(W1[e] x[t]),   e = expert[t, j]

with p, expert the softmax of the topk router logits.  Routing, products and
gradients are the library's; torch holds the tensors and does the router's
softmax and the activation.

    python examples/moe_layer.py [--tokens 4096 --hidden 2048 --inner 1024 --experts 32 --topk 4]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import blackwell_tensor_core_swizzled_gb300 as tcg  # noqa: E402

IN = {torch.float16: tcg.IN_F16, torch.bfloat16: tcg.IN_BF16}
OUT = {torch.float32: tcg.F32, torch.float16: tcg.F16, torch.bfloat16: tcg.BF16}


class Route:
    """The order of the tokens' choices by expert."""

    def __init__(self, expert: torch.Tensor, experts: int):
        self.T, self.topk = expert.shape
        self.experts, self.rows = experts, expert.numel()
        new = lambda *shape: torch.empty(shape, dtype=torch.int32, device=expert.device)  # noqa: E731
        self.offsets, self.position, self.source = new(experts + 1), new(self.T, self.topk), new(self.rows)
        tcg.moe_sort(self.T, self.topk, experts, expert, self.offsets, self.position, self.source)

    def dispatch(self, x: torch.Tensor) -> torch.Tensor:
        """Token rows [T, H] to sorted rows [T * topk, H]."""
        H = x.shape[1]
        out = x.new_empty(self.rows, H)
        tcg.moe_dispatch(OUT[x.dtype], self.T, self.topk, H, x, x.stride(0), self.position, out, H)
        return out

    def combine(self, rows: torch.Tensor, weight: torch.Tensor | None) -> torch.Tensor:
        """Weighted sum of each token's sorted rows; without weights the gradient of dispatch."""
        H = rows.shape[1]
        out = rows.new_empty(self.T, H)
        tcg.moe_combine(OUT[rows.dtype], self.T, self.topk, H, rows, H, self.position, weight, out, H)
        return out

    def combine_grad(self, dy: torch.Tensor, rows: torch.Tensor, weight: torch.Tensor):
        """Gradients of combine: of the sorted rows and of the weights."""
        H = dy.shape[1]
        drows, dweight = torch.empty_like(rows), torch.empty_like(weight)
        tcg.moe_combine_grad(OUT[dy.dtype], self.T, self.topk, H, dy, dy.stride(0), rows, H, self.position, weight,
                             drows, H, dweight)
        return drows, dweight

    def product(self, rows: torch.Tensor, w: torch.Tensor, transposed: bool = False) -> torch.Tensor:
        """rows [R, K] by w [E, N, K] to [R, N]; transposed: rows [R, N] to [R, K]."""
        E, n, k = w.shape
        if transposed:
            n, k = k, n
        out = rows.new_empty(rows.shape[0], n)
        tcg.gemm_grouped(IN[rows.dtype], rows.shape[0], n, k, E, rows, k, self.offsets, w,
                         tcg.MN_MAJOR if transposed else tcg.K_MAJOR, w.stride(1), w.stride(0), out, OUT[out.dtype], n)
        return out

    def matrix_grad(self, dout: torch.Tensor, rows: torch.Tensor) -> torch.Tensor:
        """Gradient of product's matrices in fp32: [E, N, K]."""
        n, k = dout.shape[1], rows.shape[1]
        dw = torch.empty(self.experts, n, k, dtype=torch.float32, device=rows.device)
        tcg.gemm_grouped_wgrad(IN[rows.dtype], rows.shape[0], n, k, self.experts, dout, n, rows, k, self.offsets, dw,
                               tcg.F32, k, n * k)
        return dw


class MoeLayer:
    """router [E, H], w1 [E, I, H], w2 [E, H, I], all of one 16-bit type."""

    def __init__(self, router: torch.Tensor, w1: torch.Tensor, w2: torch.Tensor, topk: int):
        self.router, self.w1, self.w2, self.topk = router, w1, w2, topk

    def choose(self, x: torch.Tensor):
        logits, expert = (x @ self.router.T).float().topk(self.topk, dim=1)
        return expert.int(), logits.softmax(dim=1)

    def forward(self, x: torch.Tensor, expert: torch.Tensor, weight: torch.Tensor):
        """y [T, H], and what backward needs."""
        route = Route(expert, self.w1.shape[0])
        xs = route.dispatch(x)
        h = route.product(xs, self.w1)
        a = torch.nn.functional.silu(h)
        ys = route.product(a, self.w2)
        return route.combine(ys, weight), (route, xs, h, a, ys, weight)

    def backward(self, dy: torch.Tensor, kept):
        """Gradients of x, of the routing weights, w1 and w2."""
        route, xs, h, a, ys, weight = kept
        dys, dweight = route.combine_grad(dy, ys, weight)
        dw2 = route.matrix_grad(dys, a)
        da = route.product(dys, self.w2, transposed=True)
        dh = torch.ops.aten.silu_backward(da, h)
        dw1 = route.matrix_grad(dh, xs)
        dx = route.combine(route.product(dh, self.w1, transposed=True), None)
        return dx, dweight, dw1, dw2


def to_nvf4(w: torch.Tensor):
    """[E, N, K] as 4-bit codes [E, N, K / 2], scales [E, N, K / 16] and a factor an expert."""
    E, N, K = w.shape
    blocks = w.float().view(E, N, K // 16, 16)
    top = blocks.abs().amax(dim=3) / 6.0
    alpha = (top.amax(dim=(1, 2)) / 448.0).clamp(min=1e-30)
    scale = (top / alpha[:, None, None]).to(torch.float8_e4m3fn)
    unit = blocks / (scale.float() * alpha[:, None, None]).clamp(min=1e-30)[..., None]
    steps = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device)  # between E2M1's magnitudes
    code = torch.bucketize(unit.abs(), steps).to(torch.uint8) | (unit < 0).to(torch.uint8) << 3
    code = code.view(E, N, K)
    return code[..., 0::2] | code[..., 1::2] << 4, scale.view(torch.uint8), alpha


class MoeDecoder:
    """The same layer with its experts in 4 bits, for a few tokens at a time."""

    def __init__(self, layer: MoeLayer):
        self.layer, self.w1, self.w2 = layer, to_nvf4(layer.w1), to_nvf4(layer.w2)

    def product(self, route: Route, rows: torch.Tensor, w) -> torch.Tensor:
        codes, scale, alpha = w
        E, n, k = codes.shape[0], codes.shape[1], 2 * codes.shape[2]
        out = rows.new_empty(rows.shape[0], n)
        tcg.gemv_w4(tcg.W4_NVF4, IN[rows.dtype], rows.shape[0], n, k, rows, k, codes, scale, out, OUT[out.dtype], n,
                    groups=E, offsets=route.offsets, alpha=alpha)
        return out

    def forward(self, x: torch.Tensor, expert: torch.Tensor, weight: torch.Tensor) -> torch.Tensor:
        route = Route(expert, self.w1[0].shape[0])
        h = self.product(route, route.dispatch(x), self.w1)
        return route.combine(self.product(route, torch.nn.functional.silu(h), self.w2), weight)


def microseconds(f, n: int) -> float:
    for _ in range(3):
        f()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    start.record()
    for _ in range(n):
        f()
    end.record()
    torch.cuda.synchronize()
    return start.elapsed_time(end) * 1e3 / n


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 4096), ("hidden", 2048), ("inner", 1024), ("experts", 32), ("topk", 4), ("batch", 8),
                        ("repeat", 20)):
        ap.add_argument("--" + name, type=int, default=value)
    o = ap.parse_args()
    torch.manual_seed(0)
    draw = lambda *shape: torch.randn(shape, device="cuda").mul_(shape[-1] ** -0.5).bfloat16()  # noqa: E731
    layer = MoeLayer(draw(o.experts, o.hidden), draw(o.experts, o.inner, o.hidden), draw(o.experts, o.hidden, o.inner),
                     o.topk)
    x, dy = draw(o.tokens, o.hidden) * o.hidden ** 0.5, draw(o.tokens, o.hidden)
    expert, weight = layer.choose(x)
    kept = layer.forward(x, expert, weight)[1]
    print(f"forward  {o.tokens} tokens: {microseconds(lambda: layer.forward(x, expert, weight), o.repeat):.0f} us")
    print(f"backward {o.tokens} tokens: {microseconds(lambda: layer.backward(dy, kept), o.repeat):.0f} us")
    decoder, few = MoeDecoder(layer), slice(0, o.batch)
    y16, _ = layer.forward(x[few], expert[few], weight[few])
    y4 = decoder.forward(x[few], expert[few], weight[few])
    off = ((y4 - y16).float().norm() / y16.float().norm()).item()
    print(f"decoding {o.batch} tokens with 4-bit experts: "
          f"{microseconds(lambda: decoder.forward(x[few], expert[few], weight[few]), o.repeat):.0f} us, "
          f"{100 * off:.1f} % from the 16-bit layer")
    rc = tcg.check()
    if rc:
        raise SystemExit(tcg.last_error_string())


if __name__ == "__main__":
    main()
