"""Performance cases of the 8-bit operators with a scale for each block of 128,
and of the mixture-of-experts layer for a few tokens.

Each case runs either the plain form (``own`` false: elementary torch
operations in 32 bits, rounded once at the end) or the library's operators
(``own`` true).  ``prepare`` makes what a program has in hand before the call,
``run`` is one pass, ``exact`` the same outputs from the definition in 64 bits.

Operators
    quantize  X [R][C] to 8-bit codes with an fp32 scale for each block: a row
              of 128 (`row`), a column of 128 (`column`) or 128 x 128
              (`square`).  With a = max |x| of a block and F the format's
              largest value (e4m3 448, e5m2 57344): scale = a / F and code =
              F x / a rounded to the format; `pow2`: scale = the smallest
              power of two that is not below a / F, code = x / scale rounded.
              A block of zeros has scale 1.  Scales of rows and columns are
              stored [block][row or column].  Column blocks of grouped rows
              begin again with every group: block j of group g is the scale
              row offsets[g] // 128 + g + j.
    product   D[m, n] = sum_b SA[b, m] SB[b, n] sum_{k in block b} A[m, k] B[n, k].
              forward: A [M][K], B [N][K] with square scales; input (the
              gradient of the rows): B stored [K][N]; weight (the gradient of
              the matrix): A stored [K][M] and B [K][N], both with column
              scales.
    grouped   the same for rows [offsets[g], offsets[g+1]) and matrix g;
              weight: DW[g][n, k] = sum over the group's rows of DY[r, n]
              A[r, k], the group's blocks of 128 rows scaled.
    layer     y[t] = sum_j w[t, j] W2[e] h(x[t]), e = expert[t, j] in [0, E),
              h(x) = silu(W1[e] x) * (W3[e] x) (gated) or silu(W1[e] x).
              Weights of x's type, or e4m3 with square scales.
"""
import math

import torch

own = False

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn,
         "e5m2": torch.float8_e5m2}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
BLOCK = 128


def listed():
    return [
        # a few decoded tokens' rows before a product: pure latency
        {"name": "quantize_few", "op": "quantize", "blocks": "row", "rows": 5, "columns": 4096, "groups": 0,
         "dtype": "f16", "format": "e4m3", "pow2": False, "skew": 0.0},
        # the activations of a training or prompt batch
        {"name": "quantize_batch", "op": "quantize", "blocks": "row", "rows": 16384, "columns": 8192, "groups": 0,
         "dtype": "bf16", "format": "e4m3", "pow2": False, "skew": 0.0},
        # experts' rows, once more for the matrices' gradient: blocks along the rows, ragged
        {"name": "quantize_columns", "op": "quantize", "blocks": "column", "rows": 16385, "columns": 4096,
         "groups": 32, "dtype": "bf16", "format": "e4m3", "pow2": True, "skew": 0.5},
        # one decoded token through a large matrix: bound by reading it
        {"name": "product_token", "op": "product", "direction": "forward", "m": 1, "n": 8192, "k": 8192,
         "format": "e4m3", "out": "bf16"},
        # a training or prompt batch: bound by the tensor cores
        {"name": "product_forward", "op": "product", "direction": "forward", "m": 8192, "n": 8192, "k": 8192,
         "format": "e4m3", "out": "bf16"},
        # a matrix' gradient over an odd number of tokens, kept in 32 bits
        {"name": "product_weight_gradient", "op": "product", "direction": "weight", "m": 4096, "n": 4096, "k": 8191,
         "format": "e4m3", "out": "f32"},
        # a decoding batch: a few rows for each expert, bound by reading the matrices
        {"name": "grouped_few", "op": "grouped", "direction": "forward", "rows": 37, "groups": 16, "n": 1032,
         "k": 2048, "format": "e4m3", "out": "bf16", "skew": 1.0},
        # a large batch over few experts
        {"name": "grouped_forward", "op": "grouped", "direction": "forward", "rows": 32768, "groups": 16, "n": 4096,
         "k": 4096, "format": "e4m3", "out": "bf16", "skew": 0.5},
        # the rows' gradient of a training step over many experts, ragged, in the wider format
        {"name": "grouped_input_gradient", "op": "grouped", "direction": "input", "rows": 12289, "groups": 64,
         "n": 4096, "k": 2048, "format": "e5m2", "out": "f16", "skew": 1.0},
        # the matrices' gradient of a training step
        {"name": "grouped_weight_gradient", "op": "grouped", "direction": "weight", "rows": 16385, "groups": 32,
         "n": 2048, "k": 4096, "format": "e4m3", "out": "f32", "skew": 0.5},
        # one decoded token through eight of many 8-bit experts
        {"name": "layer_token", "op": "layer", "tokens": 1, "topk": 8, "experts": 128, "hidden": 4096, "inner": 1024,
         "gated": True, "weights": "e4m3", "dtype": "bf16", "masked": 0.0},
        # a decoding batch through 16-bit experts, nearly all of them chosen by some token
        {"name": "layer_batch", "op": "layer", "tokens": 32, "topk": 4, "experts": 32, "hidden": 4096, "inner": 2048,
         "gated": True, "weights": "f16", "dtype": "f16", "masked": 0.1},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("quantize", "product", "grouped", "layer"))
    fmt = rng.choice(("e4m3", "e4m3", "e5m2"))
    if op == "quantize":
        c = {"op": op, "blocks": rng.choice(("row", "column", "square")), "rows": log(1, 16384),
             "columns": log(64, 8192), "groups": 0, "dtype": rng.choice(("bf16", "f16", "f32")), "format": fmt,
             "pow2": rng.random() < 0.3, "skew": rng.choice((0.5, 1.0))}
        if rng.random() < 0.7:
            c["columns"] = max(8, c["columns"] // 8 * 8)
        if c["blocks"] == "column" and rng.random() < 0.5:
            c["groups"] = log(1, 128)
        return c
    if op == "product":
        return {"op": op, "direction": rng.choice(("forward", "forward", "input", "weight")), "m": log(1, 8192),
                "n": log(64, 8192), "k": log(64, 8192), "format": fmt, "out": rng.choice(("bf16", "f16", "f32"))}
    if op == "grouped":
        while True:
            c = {"op": op, "direction": rng.choice(("forward", "input", "weight")), "rows": log(1, 32768),
                 "groups": log(1, 128), "n": log(64, 4096), "k": log(64, 4096), "format": fmt,
                 "out": rng.choice(("bf16", "f16", "f32")), "skew": rng.choice((0.0, 0.5, 1.0))}
            if c["groups"] * c["n"] * c["k"] <= 256 * 1024 * 1024:
                return c
    while True:
        c = {"op": op, "tokens": log(1, 64), "topk": rng.randint(1, 8), "experts": log(8, 128),
             "hidden": 16 * log(32, 256), "inner": 16 * log(8, 128), "gated": rng.random() < 0.7,
             "weights": "e4m3", "dtype": rng.choice(("bf16", "f16")), "masked": rng.choice((0.0, 0.0, 0.1))}
        if rng.random() < 0.5:
            c["weights"] = c["dtype"]
        if c["experts"] * c["hidden"] * c["inner"] <= 256 * 1024 * 1024 and c["topk"] <= c["experts"]:
            return c


# --------------------------------------------------------------------- inputs

def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _uniform(gen, *shape):
    return torch.rand(*shape, generator=gen, device="cuda")


def _normal(gen, dtype, scale, *shape):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


def _codes(gen, fmt, *shape):
    """Codes as a quantiser leaves them: normal values whose blocks reach the
    format's end, in rows padded to 16 bytes."""
    top = LARGEST[fmt]
    padded = shape[:-1] + ((shape[-1] + 15) // 16 * 16,)
    full = torch.randn(padded, generator=gen, device="cuda").mul_(top / 3).clamp_(-top, top).to(TORCH[fmt])
    return full[..., :shape[-1]]


def _scales(gen, fmt, size, *shape):
    """Positive scales under which codes of `fmt` have a deviation of `size`."""
    return (0.5 + _uniform(gen, *shape)) * (size * 3 / LARGEST[fmt])


def _offsets(gen, rows, groups, skew):
    """Groups are not equally popular: log-normal weights, in no order."""
    share = torch.softmax(torch.randn(groups, generator=gen, device="cuda") * skew, 0).double()
    group = torch.bucketize(_uniform(gen, rows).double(), share.cumsum(0)[:-1].contiguous(), right=True)
    counts = torch.bincount(group, minlength=groups)
    return torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = {"case": case}

    def buffer(dtype, *shape):  # a program keeps the buffers of its outputs
        return torch.empty(*shape, dtype=dtype, device="cuda")

    if op == "quantize":
        r, c, g = case["rows"], case["columns"], case["groups"]
        # rows and columns of unequal size, as activations have them
        x = torch.randn(r, c, generator=gen, device="cuda")
        x *= torch.exp(torch.randn(r, 1, generator=gen, device="cuda"))
        x *= torch.exp(torch.randn(1, c, generator=gen, device="cuda") * 0.5)
        s["x"] = x.to(TORCH[case["dtype"]])
        if g:
            s["offsets"] = _offsets(gen, r, g, case["skew"])
        s["q"] = buffer(TORCH[case["format"]], r, c)
        shape = {"row": (_blocks(c), r), "column": (r // BLOCK + g if g else _blocks(r), c),
                 "square": (_blocks(r), _blocks(c))}[case["blocks"]]
        # scale rows that no group uses keep their value
        s["scale"] = torch.zeros(shape, device="cuda")
        return s
    fmt = case.get("format", "e4m3")
    if op == "product":
        m, n, k, way = case["m"], case["n"], case["k"], case["direction"]
        s["a"] = _codes(gen, fmt, k, m) if way == "weight" else _codes(gen, fmt, m, k)
        s["sa"] = _scales(gen, fmt, 1.0, _blocks(k), m)
        s["b"] = _codes(gen, fmt, n, k) if way == "forward" else _codes(gen, fmt, k, n)
        shape = {"forward": (_blocks(n), _blocks(k)), "input": (_blocks(k), _blocks(n)), "weight": (_blocks(k), n)}[way]
        s["sb"] = _scales(gen, fmt, k ** -0.5, *shape)
        s["d"] = buffer(TORCH[case["out"]], m, n)
    elif op == "grouped":
        r, g, n, k, way = case["rows"], case["groups"], case["n"], case["k"], case["direction"]
        s["offsets"] = _offsets(gen, r, g, case["skew"])
        s["a"] = _codes(gen, fmt, r, k)
        if way == "weight":
            s["sa"] = _scales(gen, fmt, 1.0, r // BLOCK + g, k)
            s["dy"] = _codes(gen, fmt, r, n)
            s["sdy"] = _scales(gen, fmt, 0.1, r // BLOCK + g, n)
            s["d"] = buffer(TORCH[case["out"]], g, n, k)
        else:
            s["sa"] = _scales(gen, fmt, 1.0, _blocks(k), r)
            shape = (n, k) if way == "forward" else (k, n)
            s["b"] = _codes(gen, fmt, g, *shape)
            s["sb"] = _scales(gen, fmt, k ** -0.5, g, _blocks(shape[0]), _blocks(shape[1]))
            s["d"] = buffer(TORCH[case["out"]], r, n)
    else:
        t, e, topk, h, i = case["tokens"], case["experts"], case["topk"], case["hidden"], case["inner"]
        dt = TORCH[case["dtype"]]
        noise = -torch.log(-torch.log(_uniform(gen, t, e).clamp(1e-6, 1 - 1e-6)))
        score, expert = torch.topk(noise + torch.randn(e, generator=gen, device="cuda") * 0.5, topk, dim=1)
        masked = _uniform(gen, t, 1) < case["masked"]
        s["expert"] = torch.where(masked, -1, expert).to(torch.int32).contiguous()
        s["weight"] = torch.softmax(score, dim=1).contiguous()
        s["x"] = _normal(gen, dt, 1.0, t, h)
        for name, n, k in (("w1", i, h), ("w3", i, h), ("w2", h, i)):
            if name == "w3" and not case["gated"]:
                continue
            if case["weights"] == "e4m3":
                s[name] = _codes(gen, "e4m3", e, n, k)
                s["s" + name[1]] = _scales(gen, "e4m3", k ** -0.5, e, _blocks(n), _blocks(k))
            else:
                s[name] = torch.empty(e, n, k, dtype=dt, device="cuda")
                for j in range(e):
                    s[name][j] = _normal(gen, dt, k ** -0.5, n, k)
        s["work"] = buffer(torch.uint8, 4 * t * topk * i)
        s["y"] = buffer(dt, t, h)
    return s


# ----------------------------------------------------------------------- runs

def _run_own(s):
    import blackwell_tensor_core_swizzled_gb300 as tcg

    case, op = s["case"], s["case"]["op"]
    dtype = {"f32": tcg.F32, "f16": tcg.F16, "bf16": tcg.BF16}
    intype = {"f16": tcg.IN_F16, "bf16": tcg.IN_BF16, "e4m3": tcg.IN_E4M3, "e5m2": tcg.IN_E5M2}
    if op == "quantize":
        r, c, g = case["rows"], case["columns"], case["groups"]
        blocks = {"row": tcg.F8_ROW, "column": tcg.F8_COLUMN, "square": tcg.F8_SQUARE}[case["blocks"]]
        tcg.f8_quantize(intype[case["format"]], blocks, r, c, dtype[case["dtype"]], s["x"], c, s["q"], c, s["scale"],
                        s["scale"].shape[1], pow2=case["pow2"], groups=max(1, g), offsets=s.get("offsets"))
        return [s["q"], s["scale"]]
    if op == "product":
        m, n, k, way = case["m"], case["n"], case["k"], case["direction"]
        tcg.gemm_f8(intype[case["format"]], m, n, k, s["a"], tcg.MN_MAJOR if way == "weight" else tcg.K_MAJOR,
                    s["a"].stride(0), s["sa"], m, s["b"], tcg.K_MAJOR if way == "forward" else tcg.MN_MAJOR,
                    s["b"].stride(0), s["sb"], s["sb"].shape[1], way != "weight", s["d"], dtype[case["out"]], n)
        return s["d"]
    if op == "grouped":
        r, g, n, k, way = case["rows"], case["groups"], case["n"], case["k"], case["direction"]
        if way == "weight":
            tcg.gemm_f8_grouped_wgrad(intype[case["format"]], r, n, k, g, s["dy"], s["dy"].stride(0), s["sdy"], n,
                                      s["a"], s["a"].stride(0), s["sa"], k, s["offsets"], s["d"], dtype[case["out"]],
                                      k, n * k)
        else:
            tcg.gemm_f8_grouped(intype[case["format"]], r, n, k, g, s["a"], s["a"].stride(0), s["sa"], r, s["offsets"],
                                s["b"], tcg.K_MAJOR if way == "forward" else tcg.MN_MAJOR, s["b"].stride(1),
                                s["b"].stride(0), s["sb"], s["sb"].shape[2], s["sb"].stride(0), s["d"],
                                dtype[case["out"]], n)
        return s["d"]
    t, e, topk, h, i = case["tokens"], case["experts"], case["topk"], case["hidden"], case["inner"]
    tcg.moe_few(intype[case["dtype"]], intype[case["weights"]], t, h, i, topk, e, s["x"], h, s["expert"], s["weight"],
                s["w1"], s.get("w3"), s["w2"], s["work"], s["y"], dtype[case["dtype"]], h, s1=s.get("s1"),
                s3=s.get("s3"), s2=s.get("s2"))
    return s["y"]


def _spread(scale, rows, columns):
    """Square scales [..., blocks, blocks] to one for each element."""
    return scale.repeat_interleave(BLOCK, -2)[..., :rows, :].repeat_interleave(BLOCK, -1)[..., :columns]


def _along(scale, n):
    """Scales [blocks][m] of blocks along the first dimension to [n][m]."""
    return scale.repeat_interleave(BLOCK, 0)[:n]


def _group_rows(offsets, rows):
    """Each group's rows in a row of [groups][most rows], and which of them exist."""
    start, end = offsets[:-1].long(), offsets[1:].long()
    most = max(1, int((end - start).max()))
    index = start[:, None] + torch.arange(most, device="cuda")
    return index.clamp(max=rows - 1), index < end[:, None]


def _row_blocks(offsets, rows):
    """The scale row of each of the grouped rows."""
    row = torch.arange(rows, device="cuda")
    group = torch.bucketize(row, offsets[1:].long(), right=True)
    start = offsets[group].long()
    return start // BLOCK + group + (row - start) // BLOCK


def _quantized(x, top, scale, amax, fmt):
    """Codes of x in blocks of largest value `amax`; `scale` given: x / scale."""
    unit = x.double() / scale.double() if scale is not None else x.double() * top / amax.double().clamp(min=1e-300)
    return unit.float().to(TORCH[fmt])


def _run_plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "quantize":
        r, c, fmt = case["rows"], case["columns"], case["format"]
        top, x = LARGEST[fmt], s["x"].float()
        if case["blocks"] == "row":
            pad = torch.nn.functional.pad(x, (0, -c % BLOCK))
            amax = pad.view(r, -1, BLOCK).abs().amax(2).t()
            each = lambda v: v.t().repeat_interleave(BLOCK, 1)[:, :c]  # noqa: E731
        elif case["blocks"] == "column":
            if case["groups"]:
                index = _row_blocks(s["offsets"], r)
            else:
                index = torch.arange(r, device="cuda") // BLOCK
            amax = torch.full(s["scale"].shape, -1.0, device="cuda")
            amax.scatter_reduce_(0, index[:, None].expand(r, c), x.abs(), "amax")
            each = lambda v: v[index]  # noqa: E731
        else:
            pad = torch.nn.functional.pad(x, (0, -c % BLOCK, 0, -r % BLOCK))
            amax = pad.view(_blocks(r), BLOCK, _blocks(c), BLOCK).abs().amax((1, 3))
            each = lambda v: _spread(v, r, c)  # noqa: E731
        scale = amax / top
        if case["pow2"]:
            unit = amax.double() / top
            scale = torch.exp2(torch.round(torch.log2(unit)))  # within one step: log2 may be off where unit is a power
            scale = torch.where(scale < unit, 2 * scale, torch.where(scale / 2 >= unit, scale / 2, scale)).float()
        scale = torch.where(amax > 0, scale.clamp(min=2.0 ** -126), 1.0)
        q = _quantized(x, top, each(scale) if case["pow2"] else None, each(amax), fmt)
        return [q, torch.where(amax >= 0, scale, s["scale"])]
    if op == "product":
        m, n, k, way = case["m"], case["n"], case["k"], case["direction"]
        a = s["a"].float() * _along(s["sa"], k) if way == "weight" else s["a"].float() * _along(s["sa"], k).t()
        if way == "weight":
            return (a.t() @ (s["b"].float() * _along(s["sb"], k))).to(s["d"].dtype)
        b = s["b"].float() * _spread(s["sb"], *s["b"].shape)
        return (a @ (b.t() if way == "forward" else b)).to(s["d"].dtype)
    if op == "grouped":
        r, n, k, way = case["rows"], case["n"], case["k"], case["direction"]
        index, exists = _group_rows(s["offsets"], r)
        if way == "weight":
            row = _row_blocks(s["offsets"], r)
            a, dy = s["a"].float() * s["sa"][row], s["dy"].float() * s["sdy"][row]
            return torch.bmm((dy[index] * exists[:, :, None]).transpose(1, 2), a[index]).to(s["d"].dtype)
        a = (s["a"].float() * _along(s["sa"], k).t())[index]
        b = s["b"].float() * _spread(s["sb"], *s["b"].shape[1:])
        d = torch.zeros_like(s["d"])
        d[index[exists]] = torch.bmm(a, b.transpose(1, 2) if way == "forward" else b)[exists].to(d.dtype)
        return d
    e, topk = case["experts"], case["topk"]
    chosen, slot = torch.unique(torch.where((s["expert"] >= 0) & (s["expert"] < e), s["expert"], e),
                                return_inverse=True)  # a dropped choice: behind the last expert
    weight = torch.zeros(case["tokens"], chosen.numel(), device="cuda").scatter_add_(1, slot, s["weight"])
    weight, chosen = weight * (chosen < e), chosen.clamp(max=e - 1).long()

    def matrices(name):
        w = s[name][chosen] if case["weights"] != "e4m3" else s[name].view(torch.uint8)[chosen].view(s[name].dtype)
        return w.float() * _spread(s["s" + name[1]][chosen], *w.shape[1:]) if case["weights"] == "e4m3" else w.float()

    x = s["x"].float()
    h = matrices("w1") @ x.t()
    h = h * torch.sigmoid(h)
    if case["gated"]:
        h = h * (matrices("w3") @ x.t())
    return ((matrices("w2") @ h) * weight.t()[:, None, :]).sum(0).t().to(s["y"].dtype)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------- exact

F64 = torch.float64


def _value(q):
    """The numbers that 8-bit codes stand for, from their bits."""
    wide = q.dtype is torch.float8_e5m2
    man_bits, bias = (2, 15) if wide else (3, 7)
    byte = torch.arange(256, device="cuda")
    sign = 1.0 - 2.0 * (byte >> 7).to(F64)
    exp, man = (byte & 127) >> man_bits, (byte & ((1 << man_bits) - 1)).to(F64) / (1 << man_bits)
    table = sign * torch.where(exp == 0, man * 2.0 ** (1 - bias), (1 + man) * torch.exp2((exp - bias).to(F64)))
    return table[q.contiguous().view(torch.uint8).int()]


def _round(v, fmt):
    """v rounded to the format's grid, ties to even."""
    man_bits, low = (2, -14) if fmt == "e5m2" else (3, -6)
    _, e = torch.frexp(v.abs())
    step = torch.exp2(((e - 1).clamp(min=low) - man_bits).to(F64))
    return torch.round(v / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        r, c, fmt = case["rows"], case["columns"], case["format"]
        x, top = s["x"].to(F64), LARGEST[fmt]
        q, scale = torch.zeros(r, c, dtype=F64, device="cuda"), s["scale"].to(F64)

        def one(xs):  # blocks in the rows of xs
            amax = xs.abs().amax(1)
            sf = amax / top
            if case["pow2"]:
                man, ex = torch.frexp(sf)
                sf = torch.exp2(torch.where(man == 0.5, ex - 1, ex).to(F64))
            sf = torch.where(amax > 0, sf, 1.0)
            # x top / amax keeps exact ties, which x / (amax / top) would break
            unit = xs / sf[:, None] if case["pow2"] else xs * top / torch.where(amax > 0, amax, 1.0)[:, None]
            return _round(unit, fmt), sf

        if case["blocks"] == "row":
            for b in range(_blocks(c)):
                cut = slice(b * BLOCK, min(c, (b + 1) * BLOCK))
                q[:, cut], scale[b] = one(x[:, cut])
        elif case["blocks"] == "column":
            bounds = s["offsets"].tolist() if case["groups"] else [0, r]
            for g in range(len(bounds) - 1):
                for j, lo in enumerate(range(bounds[g], bounds[g + 1], BLOCK)):
                    cut = slice(lo, min(bounds[g + 1], lo + BLOCK))
                    values, sf = one(x[cut].t())
                    q[cut], scale[bounds[g] // BLOCK + g + j] = values.t(), sf
        else:
            for b in range(_blocks(r)):
                for d in range(_blocks(c)):
                    rows, cut = slice(b * BLOCK, min(r, (b + 1) * BLOCK)), slice(d * BLOCK, min(c, (d + 1) * BLOCK))
                    values, sf = one(x[rows, cut].reshape(1, -1))
                    q[rows, cut], scale[b, d] = values.view(q[rows, cut].shape), sf[0]
        return [q, scale]
    if op == "product":
        m, n, k, way = case["m"], case["n"], case["k"], case["direction"]
        a, b = _value(s["a"]), _value(s["b"])
        if way == "weight":
            a = a.t()
        if way != "forward":
            b = b.t()  # [n][k]
        d = torch.zeros(m, n, dtype=F64, device="cuda")
        for j in range(_blocks(k)):
            cut = slice(j * BLOCK, min(k, (j + 1) * BLOCK))
            if way == "weight":
                sb = s["sb"][j].to(F64)
            else:
                sb = (s["sb"][:, j] if way == "forward" else s["sb"][j]).to(F64)
                sb = sb[torch.arange(n, device="cuda") // BLOCK]
            d += torch.einsum("mk,nk->mn", a[:, cut], b[:, cut]) * s["sa"][j].to(F64)[:, None] * sb[None, :]
        return d
    if op == "grouped":
        r, g, n, k, way = case["rows"], case["groups"], case["n"], case["k"], case["direction"]
        bounds = s["offsets"].tolist()
        d = torch.zeros(s["d"].shape, dtype=F64, device="cuda")
        for i in range(g):
            lo, hi = bounds[i], bounds[i + 1]
            if way == "weight":
                for j, at in enumerate(range(lo, hi, BLOCK)):
                    rows, sf = slice(at, min(hi, at + BLOCK)), lo // BLOCK + i + j
                    d[i] += torch.einsum("rn,rk->nk", _value(s["dy"][rows]) * s["sdy"][sf].to(F64),
                                         _value(s["a"][rows]) * s["sa"][sf].to(F64))
                continue
            if lo == hi:
                continue
            sa = s["sa"][torch.arange(k, device="cuda") // BLOCK, lo:hi].to(F64)
            b = _value(s["b"][i])
            b = b * s["sb"][i].to(F64)[torch.arange(b.shape[0], device="cuda")[:, None] // BLOCK,
                                       torch.arange(b.shape[1], device="cuda")[None, :] // BLOCK]
            d[lo:hi] = torch.einsum("rk,nk->rn" if way == "forward" else "rk,kn->rn", _value(s["a"][lo:hi]) * sa.t(), b)
        return d
    t, e = case["tokens"], case["experts"]

    def matrix(name, i):
        if case["weights"] != "e4m3":
            return s[name][i].to(F64)
        w = _value(s[name][i])
        return w * s["s" + name[1]][i].to(F64)[torch.arange(w.shape[0], device="cuda")[:, None] // BLOCK,
                                               torch.arange(w.shape[1], device="cuda")[None, :] // BLOCK]

    y = torch.zeros(t, case["hidden"], dtype=F64, device="cuda")
    x, choice = s["x"].to(F64), s["expert"].tolist()
    for i in range(e):
        rows = [(a, b) for a in range(t) for b in range(case["topk"]) if choice[a][b] == i]
        if not rows:
            continue
        token = torch.tensor([a for a, _ in rows], device="cuda")
        h = torch.einsum("th,ih->ti", x[token], matrix("w1", i))
        h = h / (1 + torch.exp(-h))
        if case["gated"]:
            h = h * torch.einsum("th,ih->ti", x[token], matrix("w3", i))
        w = torch.stack([s["weight"][a, b] for a, b in rows]).to(F64)
        y.index_add_(0, token, torch.einsum("ti,hi->th", h, matrix("w2", i)) * w[:, None])
    return y


# ----------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    size = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1, "e5m2": 1}
    if op == "quantize":
        r, c, g = case["rows"], case["columns"], case["groups"]
        scales = {"row": r * _blocks(c), "column": (_blocks(r) + g // 2) * c, "square": _blocks(r) * _blocks(c)}
        return {"bytes": r * c * (size[case["dtype"]] + 1) + 4 * scales[case["blocks"]], "flops": 0}
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        sb = _blocks(k) * (n if case["direction"] == "weight" else _blocks(n))
        return {"bytes": m * k + n * k + 4 * (m * _blocks(k) + sb) + size[case["out"]] * m * n, "flops": 2 * m * n * k}
    if op == "grouped":
        r, g, n, k, o = case["rows"], case["groups"], case["n"], case["k"], size[case["out"]]
        if case["direction"] == "weight":
            return {"bytes": r * (n + k) + 4 * (r // BLOCK + g // 2) * (n + k) + o * g * n * k, "flops": 2 * r * n * k}
        # matrices that have rows: their expected number under an even choice
        used = g * (1 - (1 - 1 / g) ** r)
        return {"bytes": r * k + 4 * r * _blocks(k) + used * (n * k + 4 * _blocks(n) * _blocks(k)) + o * r * n,
                "flops": 2 * r * n * k}
    t, e, h, i = case["tokens"], case["experts"], case["hidden"], case["inner"]
    used = e * (1 - (1 - case["topk"] / e) ** (t * (1 - case["masked"])))
    parts = 3 if case["gated"] else 2
    scales = 4 * _blocks(h) * _blocks(i) if case["weights"] == "e4m3" else 0
    return {"bytes": used * parts * (h * i * size[case["weights"]] + scales) + 2 * 2 * t * h + 8 * t * case["topk"],
            "flops": 2 * parts * t * case["topk"] * h * i}
