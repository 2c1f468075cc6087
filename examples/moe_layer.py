"""A mixture-of-experts layer: a training step forward and back, in 16 bits and in
8 bits with a scale for each block of 128, and decoding with 4-bit and with 8-bit
experts.

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


class Codes:
    """A matrix (or one for each expert) in 8 bits and its scales for each block of 128."""

    def __init__(self, x: torch.Tensor, blocks: int, route: Route | None = None):
        R, C = x.shape
        groups = 1 if route is None else route.experts
        shape = {tcg.F8_ROW: (-(-C // 128), R), tcg.F8_COLUMN: (R // 128 + groups if route else -(-R // 128), C),
                 tcg.F8_SQUARE: (-(-R // 128), -(-C // 128))}[blocks]
        self.q = torch.empty(R, C, dtype=torch.float8_e4m3fn, device=x.device)
        self.scale = torch.empty(shape, device=x.device)
        tcg.f8_quantize(tcg.IN_E4M3, blocks, R, C, OUT[x.dtype], x, x.stride(0), self.q, C, self.scale, shape[1],
                        groups=groups, offsets=None if route is None else route.offsets)

    @classmethod
    def of_experts(cls, w: torch.Tensor) -> "Codes":
        """w [E, N, K] with square blocks (N a multiple of 128: blocks end with the experts)."""
        E, N, K = w.shape
        c = cls(w.view(E * N, K), tcg.F8_SQUARE)
        c.q, c.scale = c.q.view(E, N, K), c.scale.view(E, N // 128, -1)
        return c


class MoeLayer8:
    """The layer with its products in 8 bits: of the experts, quantised once, and of
    the rows and their gradients, as they come."""

    def __init__(self, layer: MoeLayer):
        self.layer, self.w1, self.w2 = layer, Codes.of_experts(layer.w1), Codes.of_experts(layer.w2)

    def product(self, route: Route, rows: torch.Tensor, w: Codes, transposed: bool = False) -> torch.Tensor:
        a = Codes(rows, tcg.F8_ROW)
        E, n, k = w.q.shape
        if transposed:
            n, k = k, n
        out = rows.new_empty(rows.shape[0], n)
        tcg.gemm_f8_grouped(tcg.IN_E4M3, rows.shape[0], n, k, E, a.q, k, a.scale, rows.shape[0], route.offsets, w.q,
                            tcg.MN_MAJOR if transposed else tcg.K_MAJOR, w.q.stride(1), w.q.stride(0), w.scale,
                            w.scale.stride(1), w.scale.stride(0), out, OUT[out.dtype], n)
        return out

    def matrix_grad(self, route: Route, dout: torch.Tensor, rows: torch.Tensor) -> torch.Tensor:
        d, a = Codes(dout, tcg.F8_COLUMN, route), Codes(rows, tcg.F8_COLUMN, route)
        n, k = dout.shape[1], rows.shape[1]
        dw = torch.empty(route.experts, n, k, dtype=torch.float32, device=rows.device)
        tcg.gemm_f8_grouped_wgrad(tcg.IN_E4M3, rows.shape[0], n, k, route.experts, d.q, n, d.scale, n, a.q, k, a.scale, k,
                                  route.offsets, dw, tcg.F32, k, n * k)
        return dw

    def forward(self, x: torch.Tensor, expert: torch.Tensor, weight: torch.Tensor):
        route = Route(expert, self.layer.w1.shape[0])
        xs = route.dispatch(x)
        h = self.product(route, xs, self.w1)
        a = torch.nn.functional.silu(h)
        ys = self.product(route, a, self.w2)
        return route.combine(ys, weight), (route, xs, h, a, ys, weight)

    def backward(self, dy: torch.Tensor, kept):
        route, xs, h, a, ys, weight = kept
        dys, dweight = route.combine_grad(dy, ys, weight)
        dw2 = self.matrix_grad(route, dys, a)
        dh = torch.ops.aten.silu_backward(self.product(route, dys, self.w2, transposed=True), h)
        dw1 = self.matrix_grad(route, dh, xs)
        dx = route.combine(self.product(route, dh, self.w1, transposed=True), None)
        return dx, dweight, dw1, dw2

    def decode(self, x: torch.Tensor, expert: torch.Tensor, weight: torch.Tensor) -> torch.Tensor:
        """y of up to 64 tokens in one call, with x as it is against the 8-bit experts."""
        T, H = x.shape
        E, inner, _ = self.w1.q.shape
        y = torch.empty_like(x)
        work = torch.empty(tcg.moe_few_work_bytes(T, expert.shape[1], inner), dtype=torch.uint8, device=x.device)
        tcg.moe_few(IN[x.dtype], tcg.IN_E4M3, T, H, inner, expert.shape[1], E, x, x.stride(0), expert, weight, self.w1.q,
                    None, self.w2.q, work, y, OUT[y.dtype], H, s1=self.w1.scale, s2=self.w2.scale)
        return y


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
    layer8 = MoeLayer8(layer)
    y8, kept = layer8.forward(x, expert, weight)
    y = layer.forward(x, expert, weight)[0]
    off = ((y8 - y).float().norm() / y.float().norm()).item()
    print(f"in 8 bits: forward {microseconds(lambda: layer8.forward(x, expert, weight), o.repeat):.0f} us, backward "
          f"{microseconds(lambda: layer8.backward(dy, kept), o.repeat):.0f} us, {100 * off:.1f} % from the 16-bit layer")
    y8 = layer8.decode(x[few], expert[few], weight[few])
    off = ((y8 - y16).float().norm() / y16.float().norm()).item()
    print(f"decoding {o.batch} tokens with 8-bit experts: "
          f"{microseconds(lambda: layer8.decode(x[few], expert[few], weight[few]), o.repeat):.0f} us, "
          f"{100 * off:.1f} % from the 16-bit layer")
    rc = tcg.check()
    if rc:
        raise SystemExit(tcg.last_error_string())


if __name__ == "__main__":
    main()
