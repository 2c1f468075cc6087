"""Performance cases of the mixture-of-experts operators: token routing,
products grouped by expert, and products with 4-bit weights.

Each case runs either the plain form (``own`` false: elementary torch
operations in 32 bits, rounded once at the end) or the library's operators
(``own`` true).  ``prepare`` makes what a program has in hand before the call,
``run`` is one pass, ``exact`` the same outputs from the definition in 64 bits.

Operators
    dispatch  T tokens chose `topk` of E experts each: order the T * topk
              choices by expert (offsets, position, source) and copy every
              token's row to its sorted positions.  Choices outside [0, E)
              are dropped: they sort after the last expert, their position is
              stored inverted (-1 - p) and their rows are zero.
    combine   forward: Y[t] = sum_j w[t, j] Ys[position[t, j]] over the kept
              choices; backward: dYs[position[t, j]] = w[t, j] dY[t] (zero
              for dropped ones) and dw[t, j] = <dY[t], Ys[position[t, j]]>.
    grouped   rows [offsets[g], offsets[g+1]) use matrix g.
              forward: D[r, n] = sum_k A[r, k] B[g][n, k];
              input (the gradient of the rows): B[g] stored [k][n];
              weight (the gradient of the matrices):
              DW[g][n, k] = sum over the group's rows of DY[r, n] A[r, k].
    w4        D[r, n] = alpha[g] sum_k A[r, k] s[g][n, k / group] c[g][n, k],
              c the value of a 4-bit code: E2M1 (mxf4: e8m0 scales per 32;
              nvf4: unsigned E4M3 scales per 16) or code - zero (int4).
"""
import math

import torch

own = False

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one token of a decoding step finds its experts: pure latency
        {"name": "dispatch_token", "op": "dispatch", "tokens": 1, "topk": 8, "experts": 128, "hidden": 4096,
         "dtype": "bf16", "masked": 0.0},
        # a prefill or training batch, a few padding tokens masked
        {"name": "dispatch_batch", "op": "dispatch", "tokens": 16384, "topk": 4, "experts": 64, "hidden": 4096,
         "dtype": "bf16", "masked": 0.02},
        # the outputs of a small decoding batch are summed back, rows of odd length
        {"name": "combine_few", "op": "combine", "direction": "forward", "tokens": 24, "topk": 6, "experts": 64,
         "hidden": 4101, "dtype": "f16", "masked": 0.1},
        # a training step's way back through the weighted sum
        {"name": "combine_backward", "op": "combine", "direction": "backward", "tokens": 8191, "topk": 8,
         "experts": 128, "hidden": 4096, "dtype": "bf16", "masked": 0.0},
        # a decoding batch: a few rows for each expert, bound by reading the matrices
        {"name": "grouped_few", "op": "grouped", "direction": "forward", "rows": 37, "groups": 16, "n": 1032,
         "k": 2048, "dtype": "bf16", "out": "bf16", "skew": 1.0},
        # a large batch over few experts: bound by the tensor cores
        {"name": "grouped_forward", "op": "grouped", "direction": "forward", "rows": 32768, "groups": 16, "n": 4096,
         "k": 4096, "dtype": "bf16", "out": "bf16", "skew": 0.5},
        # the rows' gradient of a training step over many experts, ragged
        {"name": "grouped_input_gradient", "op": "grouped", "direction": "input", "rows": 12289, "groups": 64,
         "n": 4096, "k": 2048, "dtype": "f16", "out": "f16", "skew": 1.0},
        # the matrices' gradient of a training step, kept in 32 bits
        {"name": "grouped_weight_gradient", "op": "grouped", "direction": "weight", "rows": 16385, "groups": 32,
         "n": 2048, "k": 4096, "dtype": "bf16", "out": "f32", "skew": 0.5},
        # a small projection of a small batch, odd number of outputs
        {"name": "w4_small", "op": "w4", "format": "int4", "rows": 3, "groups": 1, "n": 1001, "k": 1056, "group": 32,
         "zeros": False, "dtype": "f16"},
        # one decoded token through a large matrix
        {"name": "w4_token", "op": "w4", "format": "mxf4", "rows": 1, "groups": 1, "n": 8192, "k": 8192, "group": 32,
         "zeros": False, "dtype": "bf16"},
        # a decoding batch through a large matrix with zero points
        {"name": "w4_batch", "op": "w4", "format": "int4", "rows": 16, "groups": 1, "n": 16384, "k": 8192,
         "group": 128, "zeros": True, "dtype": "f16"},
        # four tokens decoded through eight experts each
        {"name": "w4_experts", "op": "w4", "format": "nvf4", "rows": 32, "groups": 64, "n": 4096, "k": 4096,
         "group": 16, "zeros": False, "dtype": "bf16"},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("dispatch", "combine", "grouped", "w4"))
    if op in ("dispatch", "combine"):
        while True:
            c = {"op": op, "tokens": log(1, 16384), "topk": rng.randint(1, 8), "experts": log(8, 256),
                 "hidden": log(256, 8192), "dtype": rng.choice(("bf16", "f16", "f32")),
                 "masked": rng.choice((0.0, 0.0, 0.05))}
            if rng.random() < 0.7:
                c["hidden"] = c["hidden"] // 8 * 8
            size = 4 if c["dtype"] == "f32" else 2
            if c["tokens"] * c["topk"] * c["hidden"] * size <= 16384 * 4 * 4096 * 2 and c["topk"] <= c["experts"]:
                break
        if op == "combine":
            c["direction"] = rng.choice(("forward", "backward"))
        return c
    if op == "grouped":
        while True:
            c = {"op": op, "direction": rng.choice(("forward", "input", "weight")), "rows": log(1, 32768),
                 "groups": log(1, 128), "n": log(32, 512) * 8, "k": log(32, 512) * 8,
                 "dtype": rng.choice(("bf16", "f16")), "skew": rng.choice((0.0, 0.5, 1.0))}
            c["out"] = rng.choice((c["dtype"], "f32"))
            if c["groups"] * c["n"] * c["k"] <= 512 * 1024 * 1024:
                return c
    fmt = rng.choice(("int4", "mxf4", "nvf4"))
    c = {"op": op, "format": fmt, "zeros": fmt == "int4" and rng.random() < 0.5, "dtype": rng.choice(("bf16", "f16"))}
    if rng.random() < 0.5:
        c.update(rows=log(1, 32), groups=1, n=log(256, 16384), k=log(8, 256) * 32)
    else:
        c.update(rows=log(1, 32), groups=log(8, 64), n=log(256, 4096), k=log(8, 128) * 32)
    c["group"] = {"mxf4": 32, "nvf4": 16}.get(fmt) or rng.choice([g for g in (32, 64, 128) if c["k"] % g == 0])
    return c


# --------------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _uniform(gen, *shape):
    return torch.rand(*shape, generator=gen, device="cuda")


def _normal(gen, dtype, scale, *shape):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


def _popularity(gen, count, skew):
    """Experts are not equally popular: log-normal weights, in no order."""
    return torch.randn(count, generator=gen, device="cuda") * skew


def _choices(gen, case):
    """Each token's topk distinct experts (int32 [T, topk]) and the softmax of
    their scores (f32); the choices of masked tokens are -1."""
    t, e, k = case["tokens"], case["experts"], case["topk"]
    noise = -torch.log(-torch.log(_uniform(gen, t, e).clamp(1e-6, 1 - 1e-6)))
    score, expert = torch.topk(noise + _popularity(gen, e, 0.5), k, dim=1)
    masked = _uniform(gen, t, 1) < case["masked"]
    expert = torch.where(masked, -1, expert).to(torch.int32).contiguous()
    return expert, torch.softmax(score, dim=1).contiguous()


def _order(expert, experts):
    """offsets, position and source of the choices, by a stable sort."""
    flat = expert.reshape(-1)
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    source = torch.sort(key, stable=True).indices
    rank = torch.empty_like(source)
    rank[source] = torch.arange(flat.numel(), device=flat.device)
    position = torch.where(key < experts, rank, -1 - rank)
    counts = (key[:, None] == torch.arange(experts, device=flat.device)).sum(0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    return offsets.to(torch.int32), position.to(torch.int32), source.to(torch.int32)


def _offsets(gen, case):
    g, r = case["groups"], case["rows"]
    share = torch.softmax(_popularity(gen, g, case.get("skew", 1.0)), 0).double()
    group = torch.bucketize(_uniform(gen, r).double(), share.cumsum(0)[:-1].contiguous(), right=True)
    counts = torch.bincount(group, minlength=g)
    return torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)


def _inputs(case, seed):
    gen = _generator(seed)
    op = case["op"]
    s = {"case": case}
    if op == "dispatch":
        s["expert"], _ = _choices(gen, case)
        s["x"] = _normal(gen, TORCH[case["dtype"]], 1.0, case["tokens"], case["hidden"])
    elif op == "combine":
        s["expert"], s["weight"] = _choices(gen, case)
        _, s["position"], _ = _order(s["expert"], case["experts"])
        s["ys"] = _normal(gen, TORCH[case["dtype"]], 1.0, case["tokens"] * case["topk"], case["hidden"])
        if case["direction"] == "backward":
            s["dy"] = _normal(gen, TORCH[case["dtype"]], 0.1, case["tokens"], case["hidden"])
    elif op == "grouped":
        dt, r, g, n, k = TORCH[case["dtype"]], case["rows"], case["groups"], case["n"], case["k"]
        s["offsets"] = _offsets(gen, case)
        s["a"] = _normal(gen, dt, 1.0, r, k)
        if case["direction"] == "weight":
            s["dy"] = _normal(gen, dt, 0.1, r, n)
        else:
            s["b"] = torch.empty((g, n, k) if case["direction"] == "forward" else (g, k, n), dtype=dt, device="cuda")
            for i in range(g):
                s["b"][i] = _normal(gen, dt, k ** -0.5, *s["b"].shape[1:])
    else:
        dt, r, g, n, k = TORCH[case["dtype"]], case["rows"], case["groups"], case["n"], case["k"]
        s["offsets"] = _offsets(gen, case)
        s["a"] = _normal(gen, dt, 1.0, r, k)
        s["b"] = torch.randint(0, 256, (g, n, k // 2), generator=gen, device="cuda", dtype=torch.uint8)
        blocks = (g, n, k // case["group"])
        if case["format"] == "int4":
            s["scale"] = ((0.5 + _uniform(gen, *blocks)) * (0.2 * k ** -0.5)).to(dt)
        elif case["format"] == "mxf4":
            s["scale"] = torch.randint(118, 123, blocks, generator=gen, device="cuda", dtype=torch.uint8)
        else:
            s["scale"] = torch.randint(0x28, 0x50, blocks, generator=gen, device="cuda", dtype=torch.uint8)
        if case["zeros"]:
            s["zero"] = torch.randint(5, 12, blocks, generator=gen, device="cuda", dtype=torch.uint8)
        s["alpha"] = (0.5 + _uniform(gen, g)) * (0.3 * k ** -0.5 if case["format"] == "nvf4" else 1.0)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if not own:
        return s
    # the buffers a program keeps for the outputs
    op, t = case["op"], lambda dt, *sh: torch.empty(*sh, dtype=dt, device="cuda")
    if op == "dispatch":
        m = case["tokens"] * case["topk"]
        s["out"] = [t(torch.int32, case["experts"] + 1), t(torch.int32, case["tokens"], case["topk"]),
                    t(torch.int32, m), t(s["x"].dtype, m, case["hidden"])]
    elif op == "combine" and case["direction"] == "forward":
        s["out"] = t(s["ys"].dtype, case["tokens"], case["hidden"])
    elif op == "combine":
        s["out"] = [torch.empty_like(s["ys"]), torch.empty_like(s["weight"])]
    elif op == "grouped" and case["direction"] == "weight":
        s["out"] = t(TORCH[case["out"]], case["groups"], case["n"], case["k"])
    else:
        s["out"] = t(TORCH[case.get("out", case["dtype"])], case["rows"], case["n"])
    return s


# ----------------------------------------------------------------------- runs

def _run_own(s):
    import blackwell_tensor_core_swizzled_gb300 as tcg

    case, op = s["case"], s["case"]["op"]
    dtype = {"f32": tcg.F32, "f16": tcg.F16, "bf16": tcg.BF16}
    intype = {"f16": tcg.IN_F16, "bf16": tcg.IN_BF16}
    if op == "dispatch":
        t, k, h = case["tokens"], case["topk"], case["hidden"]
        offsets, position, source, xs = s["out"]
        tcg.moe_sort(t, k, case["experts"], s["expert"], offsets, position, source)
        tcg.moe_dispatch(dtype[case["dtype"]], t, k, h, s["x"], h, position, xs, h)
        return s["out"]
    if op == "combine":
        t, k, h = case["tokens"], case["topk"], case["hidden"]
        if case["direction"] == "forward":
            tcg.moe_combine(dtype[case["dtype"]], t, k, h, s["ys"], h, s["position"], s["weight"], s["out"], h)
        else:
            tcg.moe_combine_grad(dtype[case["dtype"]], t, k, h, s["dy"], h, s["ys"], h, s["position"], s["weight"],
                                 s["out"][0], h, s["out"][1])
        return s["out"]
    r, g, n, k = case["rows"], case["groups"], case["n"], case["k"]
    if op == "grouped":
        if case["direction"] == "weight":
            tcg.gemm_grouped_wgrad(intype[case["dtype"]], r, n, k, g, s["dy"], n, s["a"], k, s["offsets"], s["out"],
                                   dtype[case["out"]], k, n * k)
        elif case["direction"] == "forward":
            tcg.gemm_grouped(intype[case["dtype"]], r, n, k, g, s["a"], k, s["offsets"], s["b"], tcg.K_MAJOR, k,
                             n * k, s["out"], dtype[case["out"]], n)
        else:
            tcg.gemm_grouped(intype[case["dtype"]], r, n, k, g, s["a"], k, s["offsets"], s["b"], tcg.MN_MAJOR, n,
                             n * k, s["out"], dtype[case["out"]], n)
        return s["out"]
    fmt = {"int4": tcg.W4_INT4, "mxf4": tcg.W4_MXF4, "nvf4": tcg.W4_NVF4}[case["format"]]
    tcg.gemv_w4(fmt, intype[case["dtype"]], r, n, k, s["a"], k, s["b"], s["scale"], s["out"], dtype[case["dtype"]], n,
                group=case["group"], zero=s.get("zero"), groups=g, offsets=s["offsets"], alpha=s["alpha"])
    return s["out"]


def _segments(offsets):
    o = offsets.tolist()
    return [(g, o[g], o[g + 1]) for g in range(len(o) - 1)]


def _weights(s, g, dtype):
    """Matrix g of a 4-bit case, decoded without alpha: [n, k] in `dtype`."""
    case, b = s["case"], s["b"][g]
    code = torch.stack([b & 15, b >> 4], dim=-1).reshape(case["n"], case["k"]).long()
    group = case["group"]
    if case["format"] == "int4":
        zero = s["zero"][g].to(dtype).repeat_interleave(group, 1) if case["zeros"] else 8
        return (code.to(dtype) - zero) * s["scale"][g].to(dtype).repeat_interleave(group, 1)
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=dtype, device="cuda")
    sf = s["scale"][g].to(dtype)
    if case["format"] == "mxf4":
        sf = torch.exp2(sf - 127)
    else:
        sf = s["scale"][g].view(torch.float8_e4m3fn).to(dtype)
    return table[code] * sf.repeat_interleave(group, 1)


def _run_plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "dispatch":
        offsets, position, source = _order(s["expert"], case["experts"])
        xs = s["x"][(source // case["topk"]).long()]
        xs[int(offsets[-1]):] = 0
        return [offsets, position.view(case["tokens"], case["topk"]), source, xs]
    if op == "combine":
        t, k = case["tokens"], case["topk"]
        position = s["position"].view(t, k).long()
        kept = (position >= 0)
        rows = torch.where(kept, position, -1 - position)
        w = s["weight"] * kept
        if case["direction"] == "forward":
            y = torch.zeros(t, case["hidden"], device="cuda")
            for j in range(k):
                y += w[:, j, None] * torch.where(kept[:, j, None], s["ys"][rows[:, j]].float(), 0)
            return y.to(s["ys"].dtype)
        dys, dw = torch.empty_like(s["ys"]), torch.empty_like(s["weight"])
        dy = s["dy"].float()
        for j in range(k):
            dys[rows[:, j]] = (w[:, j, None] * dy).to(dys.dtype)
            dw[:, j] = (dy * s["ys"][rows[:, j]].float()).sum(1) * kept[:, j]
        return [dys, dw]
    r, g, n, k = case["rows"], case["groups"], case["n"], case["k"]
    if op == "grouped" and case["direction"] == "weight":
        out = torch.empty(g, n, k, dtype=TORCH[case["out"]], device="cuda")
        for i, lo, hi in _segments(s["offsets"]):
            out[i] = (s["dy"][lo:hi].float().t() @ s["a"][lo:hi].float()).to(out.dtype)
        return out
    out = torch.zeros(r, n, dtype=TORCH[case.get("out", case["dtype"])], device="cuda")
    for i, lo, hi in _segments(s["offsets"]):
        if lo == hi:
            continue
        if op == "grouped":
            b = s["b"][i].float()
            out[lo:hi] = (s["a"][lo:hi].float() @ (b.t() if case["direction"] == "forward" else b)).to(out.dtype)
        else:
            out[lo:hi] = ((s["a"][lo:hi].float() @ _weights(s, i, torch.float32).t()) * s["alpha"][i]).to(out.dtype)
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------- exact

def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op in ("dispatch", "combine"):
        t, k, e = case["tokens"], case["topk"], case["experts"]
        flat = s["expert"].reshape(-1).long()
        bucket = torch.where((flat < 0) | (flat >= e), e, flat)
        # rank by counting: entries of smaller buckets, then earlier entries of the same one
        onehot = torch.nn.functional.one_hot(bucket, e + 1).to(torch.int32)
        total = onehot.sum(0)
        start = total.cumsum(0) - total
        earlier = onehot.cumsum(0).gather(1, bucket[:, None])[:, 0] - 1
        rank = start[bucket] + earlier
        dropped = bucket == e
    if op == "dispatch":
        source = torch.zeros(t * k, dtype=torch.int64, device="cuda")
        source.scatter_(0, rank, torch.arange(t * k, device="cuda"))
        xs = torch.zeros(t * k, case["hidden"], dtype=f64, device="cuda")
        keep = (~dropped).nonzero()[:, 0]
        xs[rank[keep]] = s["x"].to(f64)[keep // k]
        return [start.to(torch.int32), torch.where(dropped, -1 - rank, rank).to(torch.int32).view(t, k),
                source.to(torch.int32), xs]
    if op == "combine":
        w = s["weight"].to(f64).reshape(-1)
        if case["direction"] == "forward":
            y = torch.zeros(t, case["hidden"], dtype=f64, device="cuda")
            keep = (~dropped).nonzero()[:, 0]
            y.index_add_(0, keep // k, s["ys"].to(f64)[rank[keep]] * w[keep, None])
            return y
        dys = torch.zeros(t * k, case["hidden"], dtype=f64, device="cuda")
        dw = torch.zeros(t * k, dtype=f64, device="cuda")
        for lo in range(0, t * k, 8192):
            i = torch.arange(lo, min(lo + 8192, t * k), device="cuda")
            i = i[~dropped[i]]
            d = s["dy"][i // k].to(f64)
            dys[rank[i]] = d * w[i, None]
            dw[i] = torch.einsum("ih,ih->i", d, s["ys"][rank[i]].to(f64))
        return [dys, dw.view(t, k)]
    r, g, n, k = case["rows"], case["groups"], case["n"], case["k"]
    bounds = s["offsets"].tolist()
    if op == "grouped" and case["direction"] == "weight":
        out = torch.zeros(g, n, k, dtype=f64, device="cuda")
        for i in range(g):
            rows = slice(bounds[i], bounds[i + 1])
            out[i] = torch.einsum("rn,rk->nk", s["dy"][rows].to(f64), s["a"][rows].to(f64))
        return out
    out = torch.zeros(r, n, dtype=f64, device="cuda")
    for i in range(g):
        rows = slice(bounds[i], bounds[i + 1])
        if bounds[i] == bounds[i + 1]:
            continue
        a = s["a"][rows].to(f64)
        if op == "grouped":
            out[rows] = torch.einsum("rk,nk->rn" if case["direction"] == "forward" else "rk,kn->rn", a,
                                     s["b"][i].to(f64))
            continue
        # codes from the bytes: low nibble first
        byte = s["b"][i].to(torch.int64)
        code = torch.empty(n, k, dtype=torch.int64, device="cuda")
        code[:, 0::2], code[:, 1::2] = byte % 16, byte // 16
        blocks = k // case["group"]
        if case["format"] == "int4":
            zero = s["zero"][i].to(f64) if case["zeros"] else torch.full((n, blocks), 8.0, dtype=f64, device="cuda")
            value = code.to(f64).view(n, blocks, -1) - zero[:, :, None]
            sf = s["scale"][i].to(f64)
        else:
            sign = 1.0 - 2.0 * (code // 8).to(f64)
            exp, man = (code % 8) // 2, (code % 2).to(f64)
            value = torch.where(exp == 0, 0.5 * man, (1 + 0.5 * man) * 2.0 ** (exp - 1).to(f64)) * sign
            value = value.view(n, blocks, -1)
            sb = s["scale"][i].to(torch.int64)
            if case["format"] == "mxf4":
                sf = 2.0 ** (sb - 127).to(f64)
            else:
                se, sm = sb // 8, (sb % 8).to(f64)
                sf = torch.where(se == 0, sm / 8 * 2.0 ** -6, (1 + sm / 8) * 2.0 ** (se - 7).to(f64))
        w = (value * sf[:, :, None]).view(n, k)
        out[rows] = torch.einsum("rk,nk->rn", a, w) * s["alpha"][i].to(f64)
    return out


# ----------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    size = {"f32": 4, "f16": 2, "bf16": 2}
    if op in ("dispatch", "combine"):
        t, k, h, b = case["tokens"], case["topk"], case["hidden"], size[case["dtype"]]
        if op == "dispatch":
            return {"bytes": 4 * t * k * 3 + 4 * (case["experts"] + 1) + b * h * t * (1 + k), "flops": 0}
        if case["direction"] == "forward":
            return {"bytes": 8 * t * k + b * h * t * (1 + k), "flops": 2 * t * k * h}
        return {"bytes": 12 * t * k + b * h * t * (1 + 2 * k), "flops": 3 * t * k * h}
    r, g, n, k = case["rows"], case["groups"], case["n"], case["k"]
    # matrices that have rows: their expected number under an even choice
    used = g * (1 - (1 - 1 / g) ** r)
    if op == "grouped":
        b, o = size[case["dtype"]], size[case["out"]]
        if case["direction"] == "weight":
            return {"bytes": b * r * (n + k) + o * g * n * k, "flops": 2 * r * n * k}
        return {"bytes": b * r * k + b * used * n * k + o * r * n, "flops": 2 * r * n * k}
    per = {"int4": 2 + (1 if case["zeros"] else 0)}.get(case["format"], 1)
    return {"bytes": 2 * r * (n + k) + used * n * (k / 2 + per * (k // case["group"])), "flops": 2 * r * n * k}
