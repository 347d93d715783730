"""Operators of a mixture-of-experts layer and of 4-bit weights, as work to measure.

Three operators and their directions:

- tokens sorted by expert and back (``sort_tokens``, ``gather_rows``, ``combine_rows`` and the gradients of
  the last two);
- the experts' products over the sorted rows (``grouped_matmul`` and the gradients of both operands);
- products with 4-bit weights and group scales, for one weight matrix or one per expert
  (``pack_w4``, ``w4_matmul``).

``run`` computes a pass in elementary torch operations where ``own`` is false, and makes the package's
calls where it is true. ``exact`` computes the same outputs in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def _spt():
    import software_pipelined_tiled_amd as spt

    return spt


# ------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # 16 sequences decoding one token each, two experts of eight a token: launch latency
        dict(name="dispatch decode", op="dispatch", tokens=16, top_k=2, experts=8, width=4096, pad=0, dtype="bf16"),
        # a prompt, padded at its end (the padding has no expert), many experts
        dict(name="dispatch prompt", op="dispatch", tokens=8191, top_k=6, experts=64, width=2048, pad=120, dtype="f16"),
        # experts' outputs of a small batch brought back to its tokens; an odd row width
        dict(name="combine decode", op="combine", tokens=37, top_k=8, experts=128, width=4097, pad=1, dtype="bf16"),
        # a training step's way back: weighted sums, and the gradients of rows, weights and tokens
        dict(name="combine training", op="combine_train", tokens=8192, top_k=4, experts=32, width=4096, pad=0, dtype="bf16"),
        # experts' products of a decoding batch: every expert's weights are read for a few rows each
        dict(name="grouped decode", op="grouped", rows=64, experts=8, n=4096, k=4096, pad=0, dtype="bf16", out="bf16"),
        # experts' products of a long prompt
        dict(name="grouped prompt", op="grouped", rows=16384, experts=8, n=8192, k=4096, pad=0, dtype="bf16", out="bf16"),
        # many small experts, ragged sizes, rows behind the last expert's
        dict(name="grouped ragged", op="grouped", rows=5003, experts=64, n=1409, k=2044, pad=33, dtype="f16", out="f32"),
        # both gradients of a training step
        dict(name="grouped training", op="grouped_train", rows=8190, experts=16, n=4096, k=2048, pad=0, dtype="bf16", out="f32"),
        # one token against a square 4-bit weight
        dict(name="w4 one token", op="w4", rows=1, experts=0, n=8192, k=8192, group=128, zeros=False, pad=0, dtype="bf16", out="bf16"),
        # a decoding batch against a wide 4-bit weight with zero points
        dict(name="w4 batch", op="w4", rows=16, experts=0, n=28672, k=8192, group=64, zeros=True, pad=0, dtype="f16", out="f16"),
        # a short prompt; small groups, rows and columns off the tile sizes
        dict(name="w4 prompt", op="w4", rows=301, experts=0, n=1025, k=8190, group=32, zeros=True, pad=0, dtype="bf16", out="f32"),
        # a decoding batch over 4-bit experts
        dict(name="w4 experts", op="w4", rows=32, experts=8, n=4096, k=4096, group=128, zeros=False, pad=0, dtype="bf16", out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """Half of the sizes are multiples of 64, the others any."""
    v = _log(rng, lo, hi)
    return max(64, v // 64 * 64) if rng.random() < 0.5 else v


def draw(rng):
    op = rng.choice(["dispatch", "combine", "combine_train", "grouped", "grouped", "grouped_train", "w4", "w4", "w4"])
    dtype = rng.choice(["bf16", "f16"])
    if op in ("dispatch", "combine", "combine_train"):
        experts = _log(rng, 2, 256)
        top_k = rng.randint(1, min(8, experts))
        width = _size(rng, 100, 8192)
        most = 1 << 27  # elements of the sorted rows
        tokens = _log(rng, 1, min(32768, most // (width * top_k)))
        return dict(op=op, tokens=tokens, top_k=top_k, experts=experts, width=width,
                    pad=rng.choice([0, tokens // 16]), dtype=dtype)
    if op in ("grouped", "grouped_train"):
        experts = _log(rng, 1, 128)
        n, k = _size(rng, 100, 8192), _size(rng, 100, 8192)
        n = max(1, min(n, (1 << 29) // (experts * k)))
        most = int(5.0e11) // (n * k * (2 if op == "grouped_train" else 1))
        rows = _log(rng, 1, max(2, min(16384, most)))
        return dict(op=op, rows=rows, experts=experts, n=n, k=k, pad=rng.choice([0, rows // 16]), dtype=dtype,
                    out=rng.choice([dtype, "f32"]))
    experts = rng.choice([0, 0, _log(rng, 2, 64)])
    n, k = _size(rng, 100, 28672), _size(rng, 100, 8192)
    n = max(1, min(n, (1 << 28) // (max(experts, 1) * k)))
    rows = _log(rng, 1, 512)
    return dict(op=op, rows=rows, experts=experts, n=n, k=k, group=rng.choice([32, 64, 128]),
                zeros=rng.random() < 0.5, pad=rng.choice([0, rows // 16]) if experts else 0, dtype=dtype,
                out=rng.choice([dtype, dtype, "f32"]))


def _w4_groups(case):
    return -(-case["k"] // case["group"])


def work(case):
    op = case["op"]
    if op in ("dispatch", "combine", "combine_train"):
        t, k, h = case["tokens"], case["top_k"], case["width"]
        r = t * k
        if op == "dispatch":  # ids in, two index lists and the offsets out, tokens in, rows out
            return {"bytes": 8 * r + 8 * r + 4 * (case["experts"] + 1) + 2 * h * (t + r), "flops": 0}
        if op == "combine":
            return {"bytes": 8 * r + 2 * h * (t + r), "flops": 2 * r * h}
        # out; dY and dW from dOut and Y; dX from the sorted rows' gradient. Y is read once.
        return {"bytes": 12 * r + 2 * h * (t + r) + 2 * h * (t + r) + 2 * h * (r + t), "flops": 2 * r * h + 3 * r * h + r * h}
    if op in ("grouped", "grouped_train"):
        r, e, n, k = case["rows"], case["experts"], case["n"], case["k"]
        o = 4 if case["out"] == "f32" else 2
        used = min(e, max(r - case["pad"], 0))  # experts with rows, at most
        flops = 2 * (r - case["pad"]) * n * k
        if op == "grouped":
            return {"bytes": 2 * r * k + 2 * used * n * k + o * r * n, "flops": flops}
        # dA (in the operands' type) from dC and B; dB from dC and A
        return {"bytes": 2 * r * n + 2 * used * n * k + 2 * r * k + 2 * r * k + o * e * n * k, "flops": 2 * flops}
    m, n, k = case["rows"], case["n"], case["k"]
    e = max(case["experts"], 1)
    used = min(e, max(m - case["pad"], 0))
    o = 4 if case["out"] == "f32" else 2
    per_group = 2 + (0.5 if case["zeros"] else 0)
    return {"bytes": int(used * n * (k / 2 + per_group * _w4_groups(case)) + 2 * m * k + o * m * n),
            "flops": 2 * (m - case["pad"]) * n * k}


# ----------------------------------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)


def _normal(shape, g, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _route(tokens, top_k, experts, pad, g):
    """Expert ids [tokens, top_k] (distinct per token, some experts preferred; the last `pad` tokens have
    none: -1) and their weights, as a softmax router over the experts leaves them."""
    logits = torch.randn((tokens, experts), generator=g, device="cuda")
    logits += torch.randn((experts,), generator=g, device="cuda") * 0.5
    val, ids = torch.topk(torch.softmax(logits, dim=1), top_k, dim=1)
    val = val / val.sum(dim=1, keepdim=True)
    if pad:
        ids[tokens - pad:] = -1
    return ids, val


def _plain_sort(ids, experts):
    """offsets [experts + 1], slots [rows] (sorted position -> slot) and position of each slot."""
    flat = ids.reshape(-1)
    key = torch.where((flat >= 0) & (flat < experts), flat, torch.full_like(flat, experts))
    slots = torch.argsort(key, stable=True)
    edges = torch.arange(experts + 1, device=flat.device)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=flat.device),
                         torch.cumsum((key[:, None] == edges[None, :experts]).sum(dim=0), dim=0)])
    rows = torch.empty_like(slots)
    rows[slots] = torch.arange(slots.numel(), device=flat.device)
    return offsets.to(torch.int32), slots.to(torch.int32), rows.to(torch.int32).reshape(ids.shape)


def _expert_offsets(rows, experts, pad, g):
    """Offsets of `rows - pad` rows spread unevenly over the experts (some may get none)."""
    kept = rows - pad
    share = torch.softmax(torch.randn((experts,), generator=g, device="cuda") * 0.7, dim=0)
    ids = torch.multinomial(share, max(kept, 1), replacement=True, generator=g)[:kept]
    counts = torch.bincount(ids, minlength=experts)
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(counts, dim=0).to(torch.int32)
    return offsets


def _inputs(case, seed):
    g = _generator(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    s = {"op": op, "case": case}
    if op in ("dispatch", "combine", "combine_train"):
        t, k, h = case["tokens"], case["top_k"], case["width"]
        s["ids"], s["weights"] = _route(t, k, case["experts"], case["pad"], g)
        if op == "dispatch":
            s["x"] = _normal((t, h), g, dt)
        else:
            s["y"] = _normal((t * k, h), g, dt)
        if op == "combine_train":
            s["dout"] = _normal((t, h), g, dt)
            s["dsorted"] = _normal((t * k, h), g, dt)
        return s
    r, n, k, e = case["rows"], case["n"], case["k"], case["experts"]
    if op in ("grouped", "grouped_train"):
        s["offsets"] = _expert_offsets(r, e, case["pad"], g)
        s["a"] = _normal((r, k), g, dt)
        s["b"] = _normal((e, n, k), g, dt, k ** -0.5)
        if op == "grouped_train":
            s["dc"] = _normal((r, n), g, dt)
        return s
    shape = (e, n) if e else (n,)
    gs = _w4_groups(case)
    s["offsets"] = _expert_offsets(r, e, case["pad"], g) if e else None
    s["x"] = _normal((r, k), g, dt)
    s["q"] = (torch.randn((*shape, k), generator=g, device="cuda") * 2.5 + 8.0).round_().clamp_(0, 15).to(torch.uint8)
    s["scales"] = ((0.5 + torch.rand((*shape, gs), generator=g, device="cuda")) * (0.4 * k ** -0.5)).to(dt)
    s["zeros"] = (torch.randint(5, 11, (*shape, gs), generator=g, device="cuda").to(torch.uint8)
                  if case["zeros"] else None)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op in ("combine", "combine_train"):
        if own:  # the order the forward's dispatch left
            s["order"] = _spt().sort_tokens(s["ids"], case["experts"])
        else:
            s["order"] = _plain_sort(s["ids"], case["experts"])
    elif op != "dispatch" and s["offsets"] is not None:
        if not own:  # the plain form walks the experts on the host
            s["bounds"] = s["offsets"].tolist()
    if op == "w4" and own:  # a model's 4-bit weights, laid out once
        s["packed"] = _spt().pack_w4(s.pop("q"), s.pop("scales"), s.pop("zeros"), case["group"])
    return s


# ------------------------------------------------------------------------------------- plain forms

def _dequant(q, scales, zeros, group, dtype):
    k = q.shape[-1]
    z = zeros.to(dtype) if zeros is not None else torch.full_like(scales, 8.0, dtype=dtype)
    z = z.repeat_interleave(group, dim=-1)[..., :k]
    sc = scales.to(dtype).repeat_interleave(group, dim=-1)[..., :k]
    return (q.to(dtype) - z) * sc


def _plain(s):
    case, op = s["case"], s["op"]
    dt = DTYPES[case["dtype"]]
    f32 = torch.float32
    if op == "dispatch":
        offsets, slots, rows = _plain_sort(s["ids"], case["experts"])
        kept = torch.arange(slots.numel(), device=slots.device) < offsets[-1]
        return {"offsets": offsets, "slots": slots, "rows": rows,
                "sorted": torch.where(kept[:, None], s["x"][slots.long() // case["top_k"]], 0)}
    if op in ("combine", "combine_train"):
        offsets, slots, rows = s["order"]
        rl = rows.long()
        kept = rows < offsets[-1]
        w = s["weights"]
        y = torch.where(kept[:, :, None], s["y"].to(f32)[rl], 0)
        out = (w[:, :, None] * y).sum(dim=1).to(dt)
        if op == "combine":
            return out
        dout = s["dout"].to(f32)
        dy = torch.zeros_like(s["y"])
        dy[rl] = torch.where(kept[:, :, None], w[:, :, None] * dout[:, None, :], 0).to(dt)
        dw = (dout[:, None, :] * y).sum(dim=2)
        del y
        dx = torch.where(kept[:, :, None], s["dsorted"].to(f32)[rl], 0).sum(dim=1).to(dt)
        return {"out": out, "dy": dy, "dweights": dw, "dx": dx}
    od = DTYPES[case["out"]]
    if op == "grouped":
        c = torch.zeros((case["rows"], case["n"]), dtype=od, device="cuda")
        for e in range(case["experts"]):
            lo, hi = s["bounds"][e], s["bounds"][e + 1]
            if hi > lo:
                c[lo:hi] = (s["a"][lo:hi].to(f32) @ s["b"][e].to(f32).t()).to(od)
        return c
    if op == "grouped_train":
        da = torch.zeros((case["rows"], case["k"]), dtype=dt, device="cuda")
        db = torch.zeros((case["experts"], case["n"], case["k"]), dtype=od, device="cuda")
        for e in range(case["experts"]):
            lo, hi = s["bounds"][e], s["bounds"][e + 1]
            if hi > lo:
                dc = s["dc"][lo:hi].to(f32)
                da[lo:hi] = (dc @ s["b"][e].to(f32)).to(dt)
                db[e] = (dc.t() @ s["a"][lo:hi].to(f32)).to(od)
        return {"da": da, "db": db}
    if s["offsets"] is None:
        w = _dequant(s["q"], s["scales"], s["zeros"], case["group"], f32)
        return (s["x"].to(f32) @ w.t()).to(od)
    c = torch.zeros((case["rows"], case["n"]), dtype=od, device="cuda")
    for e in range(case["experts"]):
        lo, hi = s["bounds"][e], s["bounds"][e + 1]
        if hi > lo:
            w = _dequant(s["q"][e], s["scales"][e], None if s["zeros"] is None else s["zeros"][e], case["group"], f32)
            c[lo:hi] = (s["x"][lo:hi].to(f32) @ w.t()).to(od)
    return c


def _own(s):
    spt = _spt()
    case, op = s["case"], s["op"]
    if op == "dispatch":
        order = spt.sort_tokens(s["ids"], case["experts"])
        return {"offsets": order.offsets, "slots": order.slots, "rows": order.rows,
                "sorted": spt.gather_rows(s["x"], order)}
    if op == "combine":
        return spt.combine_rows(s["y"], s["order"], s["weights"])
    if op == "combine_train":
        out = spt.combine_rows(s["y"], s["order"], s["weights"])
        dy, dw = spt.combine_rows_grad(s["dout"], s["y"], s["order"], s["weights"])
        return {"out": out, "dy": dy, "dweights": dw, "dx": spt.gather_rows_grad(s["dsorted"], s["order"])}
    od = DTYPES[case["out"]]
    if op == "grouped":
        return spt.grouped_matmul(s["a"], s["b"], s["offsets"], out_dtype=od)
    if op == "grouped_train":
        return {"da": spt.grouped_matmul_grad_a(s["dc"], s["b"], s["offsets"]),
                "db": spt.grouped_matmul_grad_b(s["dc"], s["a"], s["offsets"], out_dtype=od)}
    return spt.w4_matmul(s["x"], s["packed"], offsets=s["offsets"], out_dtype=od)


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------------- the definition

def exact(case, seed):
    """The definitions in 64 bits, one sum per expert or token slot."""
    s = _inputs(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op in ("dispatch", "combine", "combine_train"):
        flat = s["ids"].reshape(-1).long()
        r, e, k = flat.numel(), case["experts"], case["top_k"]
        ok = (flat >= 0) & (flat < e)
        place = torch.where(ok, flat, e) * r + torch.arange(r, device=flat.device)  # unique keys
        slots = torch.sort(place).values % r
        rows = torch.argsort(slots).reshape(s["ids"].shape)
        counts = torch.bincount(flat[ok], minlength=e)
        offsets = torch.nn.functional.pad(torch.cumsum(counts, 0), (1, 0))
        kept = int(offsets[-1])
        if op == "dispatch":
            out = torch.zeros((r, case["width"]), dtype=f64, device="cuda")
            out[:kept] = s["x"].to(f64)[slots[:kept] // k]
            return {"offsets": offsets, "slots": slots, "rows": rows, "sorted": out}
        ok2 = ok.reshape(s["ids"].shape)
        w = s["weights"].to(f64)
        t, h = case["tokens"], case["width"]
        out = torch.zeros((t, h), dtype=f64, device="cuda")
        dx = torch.zeros((t, h), dtype=f64, device="cuda") if op == "combine_train" else None
        dy = torch.zeros((r, h), dtype=f64, device="cuda") if op == "combine_train" else None
        dw = torch.zeros((t, k), dtype=f64, device="cuda") if op == "combine_train" else None
        for j in range(k):
            m = ok2[:, j]
            at = rows[m, j]
            y = s["y"][at].to(f64)
            out[m] += w[m, j, None] * y
            if op == "combine_train":
                d = s["dout"][m].to(f64)
                dy[at] = w[m, j, None] * d
                dw[m, j] = (d * y).sum(dim=1)
                dx[m] += s["dsorted"][at].to(f64)
        if op == "combine":
            return out
        return {"out": out, "dy": dy, "dweights": dw, "dx": dx}
    r, n, k, e = case["rows"], case["n"], case["k"], case["experts"]
    bounds = s["offsets"].tolist() if s["offsets"] is not None else [0, r]
    if op == "grouped_train":
        da = torch.zeros((r, k), dtype=f64, device="cuda")
        db = torch.zeros((e, n, k), dtype=f64, device="cuda")
        for i in range(e):
            part = slice(bounds[i], bounds[i + 1])
            if bounds[i + 1] > bounds[i]:
                da[part] = s["dc"][part].to(f64) @ s["b"][i].to(f64)
                db[i] = s["dc"][part].to(f64).t() @ s["a"][part].to(f64)
        return {"da": da, "db": db}
    x = s["a"] if op == "grouped" else s["x"]
    c = torch.zeros((r, n), dtype=f64, device="cuda")
    for i in range(len(bounds) - 1):
        part = slice(bounds[i], bounds[i + 1])
        if bounds[i + 1] <= bounds[i]:
            continue
        if op == "grouped":
            weight = s["b"][i].to(f64)
        else:
            pick = (lambda t: t[i]) if e else (lambda t: t)
            group = torch.arange(k, device="cuda") // case["group"]
            weight = pick(s["q"]).to(f64)
            weight -= pick(s["zeros"]).to(f64)[:, group] if case["zeros"] else 8.0
            weight *= pick(s["scales"]).to(f64)[:, group]
        c[part] = x[part].to(f64) @ weight.t()
    return c
