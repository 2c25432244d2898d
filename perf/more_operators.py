"""Operators of a decoder layer beside the quantized linear layers, as cases to
measure: matrix-vector products with 4-bit weights, tokens sorted by expert and
back (with the gradient), norms of queries and keys with the rotation, and
attention over whole prompts.

`run` computes them in plain torch operations in 32 bits (`own` false) or through
the library's entry points (`own` true), `exact` from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

MX, NV = 0, 1
HALF, INTERLEAVED = 0, 1


def _lib():
    from nvfp4_mxfp4_w4a4_gb300 import fp4lin

    fp4lin.load()
    return fp4lin


# ------------------------------------------------------------------ cases


def listed():
    return [
        # one token through a 4096-wide projection (latency), three drafted tokens through
        # the decode workload's layer in the checkpoint's own format, and the largest batch
        # through the prefill workload's layer, with a ragged number of outputs
        dict(name="gemv_mx_one", op="gemv", fmt=MX, m=1, n=4096, k=4096),
        dict(name="gemv_nv_draft", op="gemv", fmt=NV, m=3, n=14336, k=4096),
        dict(name="gemv_mx_large", op="gemv", fmt=MX, m=8, n=18429, k=7168),
        # one token through the gate and up projections of its 8 of 64 experts
        dict(name="gemv_experts", op="experts", tokens=1, top=8, experts=64, n=2048, k=4096),
        # a decode batch's tokens to the rows of the grouped GEMM, and a prefill's
        dict(name="dispatch_decode", op="dispatch", tokens=32, top=8, experts=64, width=4096),
        dict(name="dispatch_prefill", op="dispatch", tokens=4096, top=8, experts=64, width=4096),
        # a decode batch back from the experts; a training step's forward and gradients
        dict(name="combine_decode", op="combine", tokens=32, top=8, experts=64, width=4096, grad=0),
        dict(name="combine_train", op="combine", tokens=4093, top=8, experts=64, width=4096, grad=1),
        # queries and keys of a decode batch, and of a long prefill
        dict(name="norm_rope_decode", op="norm", t=64, heads=32, kv=8, dim=128, rot=128, layout=HALF),
        dict(name="norm_rope_prefill", op="norm", t=16381, heads=56, kv=8, dim=128, rot=64, layout=INTERLEAVED),
        # a batch of short ragged prompts, and one long one
        dict(name="prompt_short", op="prompt", batch=16, n=509, ctx=0, heads=8, group=4, dim=64, causal=1),
        dict(name="prompt_long", op="prompt", batch=1, n=16381, ctx=0, heads=8, group=4, dim=128, causal=1),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gemv", "gemv", "experts", "dispatch", "combine", "norm", "prompt", "prompt", "prompt"])
    if op == "gemv":
        n = _log(rng, 8, 18432)
        return dict(op=op, fmt=rng.choice([MX, NV]), m=rng.randint(1, 8), n=n, k=32 * _log(rng, 4, min(576, 4128768 // n)))
    if op == "experts":
        experts = _log(rng, 4, 64)
        return dict(op=op, tokens=rng.randint(1, 4), top=rng.randint(1, min(8, experts)), experts=experts,
                    n=_log(rng, 64, 4096), k=32 * _log(rng, 8, 128))
    experts = _log(rng, 8, 256)
    if op in ("dispatch", "combine"):
        c = dict(op=op, tokens=_log(rng, 1, 4093), top=rng.randint(1, 8), experts=experts, width=8 * _log(rng, 8, 512))
        if op == "combine":
            c["grad"] = rng.choice([0, 1])
        return c
    dim = rng.choice([64, 128])
    if op == "norm":
        kv = rng.choice([1, 2, 4, 8])
        return dict(op=op, t=_log(rng, 1, 16381), heads=kv * rng.randint(1, 7), kv=kv, dim=dim,
                    rot=rng.choice([dim, dim // 2]), layout=rng.choice([HALF, INTERLEAVED]))
    batch, heads, group = _log(rng, 1, 32), rng.choice([1, 2, 4, 8]), rng.randint(1, 8)
    ctx = rng.choice([0, 0, 0, 1, -1])
    # (token, key) pairs, heads and sequences together stay below the long prompt's
    most = int(math.sqrt(32 * 128 * 16381.0 ** 2 / (batch * heads * group * dim)) / (1 if ctx <= 0 else 4))
    n = _log(rng, 1, min(most, 16381))
    if ctx > 0:
        ctx = _log(rng, 1, 7 * n)     # a chunk behind a context
    elif ctx < 0:
        ctx = -rng.randint(0, n)      # fewer keys than queries: the first rows see nothing
    return dict(op=op, batch=batch, n=n, ctx=ctx, heads=heads, group=group, dim=dim, causal=rng.choice([1, 1, 1, 0]))


def _lens(c):
    """(queries, keys) of each sequence: the first has the whole of both; of four or
    more the last has no tokens."""
    r = random.Random("%d %d %d" % (c["batch"], c["n"], c["ctx"]))
    got = [(c["n"], max(c["n"] + c["ctx"], 0))]
    for b in range(1, c["batch"]):
        n = 0 if b >= 3 and b == c["batch"] - 1 else r.randint((c["n"] + 3) // 4, c["n"])
        ctx = r.randint(0, c["ctx"]) if c["ctx"] > 0 else -r.randint(0, -c["ctx"])
        got.append((n, max(n + ctx, 0) if n else 0))
    return got


def _pairs(n, keys, causal):
    """(query, key) pairs that see each other: query i sees keys up to i + keys - n."""
    if not causal:
        return n * keys
    skip = max(n - keys, 0)
    return (n - skip) * (2 * keys - n + skip + 1) // 2


def work(case):
    c = case
    if c["op"] == "gemv":
        group = 32 if c["fmt"] == MX else 16
        return {"bytes": c["n"] * c["k"] * (0.5 + 1 / group) + 2 * c["m"] * c["k"] + 2 * c["n"] + 2 * c["m"] * c["n"],
                "flops": 2 * c["m"] * c["n"] * c["k"]}
    if c["op"] == "experts":
        met = c["experts"] * (1 - (1 - c["top"] / c["experts"]) ** c["tokens"])   # experts that some token chose
        rows = c["tokens"] * c["top"]
        return {"bytes": met * (c["n"] * c["k"] * 0.53125 + 2 * c["n"]) + 2 * c["tokens"] * c["k"] + 2 * rows * c["n"],
                "flops": 2 * rows * c["n"] * c["k"]}
    if c["op"] in ("dispatch", "combine"):
        t, rows, w = c["tokens"], c["tokens"] * c["top"], 2 * c["width"]
        if c["op"] == "dispatch":
            return {"bytes": (t + rows) * w + 8 * rows + 4 * c["experts"], "flops": 0}
        b, f = (t + rows) * w + 8 * rows, 2 * rows * c["width"]
        if c["grad"]:
            b, f = b + (t + rows) * w + 4 * rows, 5 * rows * c["width"]
        return {"bytes": b, "flops": f}
    if c["op"] == "norm":
        heads = c["heads"] + c["kv"]
        return {"bytes": c["t"] * (4 * heads * c["dim"] + 4 * c["rot"] + 4), "flops": c["t"] * heads * (4 * c["dim"] + 3 * c["rot"])}
    lens, heads, dim = _lens(c), c["heads"] * c["group"], c["dim"]
    pairs = sum(_pairs(n, k, c["causal"]) for n, k in lens)
    return {"bytes": sum(n for n, _ in lens) * heads * (4 * dim + 4) + sum(k for _, k in lens) * 4 * c["heads"] * dim,
            "flops": 4 * pairs * heads * dim}


# ----------------------------------------------------------------- inputs


def _quantize(w, fmt):
    """float32 [N, K] -> (codes [N, K / 2], scale bytes [N, K / group], global scale)."""
    if fmt == MX:
        b = w.unflatten(-1, (-1, 32))
        _, e = torch.frexp(b.abs().amax(-1))
        e = (e - 3).clamp(-127, 127)
        y, scales, g = torch.ldexp(b, -e.unsqueeze(-1)), (e + 127).to(torch.uint8), 1.0
    else:
        b = w.unflatten(-1, (-1, 16))
        g = float(w.abs().amax()) / 2688.0
        s = (b.abs().amax(-1) / (6.0 * g)).to(torch.float8_e4m3fn)
        y, scales = b / (s.float() * g).clamp(min=1e-30).unsqueeze(-1), s.view(torch.uint8)
    y = y.flatten(-2)
    a = y.abs()
    code = 8 * torch.signbit(y).to(torch.uint8)
    for at, up in ((0.25, 0), (0.75, 1), (1.25, 0), (1.75, 1), (2.5, 0), (3.5, 1), (5.0, 0)):
        code += (a >= at if up else a > at)
    return code[..., 0::2] | (code[..., 1::2] << 4), scales, g


def _swizzle(s):
    """Scale bytes [N, blocks] in the order of 128 rows x 4 blocks that the library's weights have."""
    n, kb = s.shape
    p = torch.nn.functional.pad(s, (0, -kb % 4, 0, -n % 128))
    return p.view(-1, 4, 32, p.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).flatten().contiguous()


def _weight(g, n, k, fmt):
    """A weight [n, k] of normal values, some input channels larger: codes, swizzled scales, global scale."""
    w = 0.02 * torch.randn(n, k, generator=g, device="cuda")
    w *= 1.0 + 7.0 * (torch.rand(k, generator=g, device="cuda") < 0.01)
    codes, scales, alpha = _quantize(w, fmt)
    return codes, _swizzle(scales), alpha


def _acts(g, *shape):
    """Activations: normal, one in 200 sixteen times as large."""
    x = torch.randn(*shape, generator=g, device="cuda")
    x *= 1.0 + 15.0 * (torch.rand(*shape, generator=g, device="cuda") < 0.005)
    return x.to(torch.bfloat16)


def _routing(g, tokens, top, experts, padded=True):
    """Expert of each choice [tokens, top] (different ones for a token, some experts
    more often) and its weight; one token in 64 is padding, without experts."""
    logits = torch.randn(tokens, experts, generator=g, device="cuda")
    logits += torch.randn(experts, generator=g, device="cuda") * 0.5
    best, ids = logits.topk(min(top, experts), -1)
    ids = ids.int()
    if padded:
        ids[torch.rand(tokens, generator=g, device="cuda") < 1 / 64] = -1
    return ids.contiguous(), torch.softmax(best, -1).contiguous()


def _rows(ids, experts):
    """The row of each choice when choices are sorted by expert, and the experts' first rows."""
    flat = ids.flatten().long()
    key = torch.where((flat >= 0) & (flat < experts), flat, torch.full_like(flat, experts))
    order = torch.sort(key, stable=True).indices
    row = torch.empty_like(key)
    row[order] = torch.arange(key.numel(), device="cuda")
    row = torch.where(key < experts, row, torch.full_like(row, -1))
    offsets = torch.zeros(experts + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.bincount(key, minlength=experts + 1)[:experts].cumsum(0)
    return row.int().view(ids.shape), offsets.int()


def _table(positions, rot):
    """cos and sin [positions, rot] of base 500000, rounded from 64 bits."""
    f = 500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(positions, dtype=torch.float64, device="cuda").unsqueeze(1) * f
    return torch.cat((a.cos(), a.sin()), -1).float()


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": c}
    if c["op"] == "gemv":
        m, n, k = c["m"], c["n"], c["k"]
        s["x"] = _acts(g, m, k)
        s["w"], s["sw"], s["alpha"] = _weight(g, n, k, c["fmt"])
        s["bias"] = (0.01 * torch.randn(n, generator=g, device="cuda")).to(torch.bfloat16)
        if own:
            s["out"] = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
        return s
    if c["op"] == "experts":
        s["x"] = _acts(g, c["tokens"], c["k"])
        parts = [_weight(g, c["n"], c["k"], MX) for _ in range(c["experts"])]
        s["w"] = torch.stack([p[0] for p in parts])
        s["sw"] = torch.stack([p[1] for p in parts])
        s["bias"] = (0.01 * torch.randn(c["experts"], c["n"], generator=g, device="cuda")).to(torch.bfloat16)
        s["ids"], _ = _routing(g, c["tokens"], c["top"], c["experts"], padded=False)
        if own:
            s["out"] = torch.empty(c["tokens"] * c["top"], c["n"], dtype=torch.bfloat16, device="cuda")
        return s
    if c["op"] in ("dispatch", "combine"):
        t, top, width = c["tokens"], c["top"], c["width"]
        s["ids"], s["weights"] = _routing(g, t, top, c["experts"])
        if c["op"] == "dispatch":
            s["x"] = _acts(g, t, width)
            s["sorted"] = torch.zeros(t * top, width, dtype=torch.bfloat16, device="cuda")
            if own:
                s["offsets"] = torch.empty(c["experts"] + 1, dtype=torch.int32, device="cuda")
                s["rows"] = torch.empty(t, top, dtype=torch.int32, device="cuda")
            return s
        s["rows"], _ = _rows(s["ids"], c["experts"])
        s["y"] = _acts(g, t * top, width)
        s["grad_y"] = torch.zeros(t * top, width, dtype=torch.bfloat16, device="cuda")
        if c["grad"]:
            s["grad"] = torch.randn(t, width, generator=g, device="cuda").to(torch.bfloat16)
        if own:
            s["out"] = torch.empty(t, width, dtype=torch.bfloat16, device="cuda")
            s["grad_w"] = torch.empty(t, top, dtype=torch.float32, device="cuda")
        return s
    if c["op"] == "norm":
        t, heads, kv, dim = c["t"], c["heads"], c["kv"], c["dim"]
        qkv = _acts(g, t, (heads + 2 * kv) * dim)     # the rows of one projection
        s["q"] = qkv[:, : heads * dim].unflatten(1, (heads, dim))
        s["k"] = qkv[:, heads * dim: (heads + kv) * dim].unflatten(1, (kv, dim))
        for name in ("q_weight", "k_weight"):
            s[name] = (1.0 + 0.2 * torch.randn(dim, generator=g, device="cuda")).to(torch.bfloat16)
        s["eps"] = 1e-6
        s["positions"] = torch.randint(0, 32768, (t,), generator=g, device="cuda", dtype=torch.int32)
        s["table"] = _table(32768, c["rot"])
        if own:
            s["rope"] = _lib().rope_params(s["table"], c["rot"], c["layout"])
            s["q_out"] = torch.empty(t, heads, dim, dtype=torch.bfloat16, device="cuda")
            s["k_out"] = torch.empty(t, kv, dim, dtype=torch.bfloat16, device="cuda")
        return s
    lens, heads, dim = _lens(c), c["heads"], c["dim"]
    n, keys = sum(a for a, _ in lens), sum(b for _, b in lens)
    s["q"] = torch.randn(n, heads * c["group"], dim, generator=g, device="cuda").to(torch.bfloat16)
    # keys and values: slices of the rows of one projection; a few channels are larger
    kv = torch.randn(keys, 2 * heads, dim, generator=g, device="cuda")
    kv *= 1.0 + 3.0 * (torch.arange(dim, device="cuda") % 61 == 5)
    kv = kv.to(torch.bfloat16)
    s["k"], s["v"] = kv[:, :heads], kv[:, heads:]
    cu, cu_k = [0], [0]
    for a, b in lens:
        cu.append(cu[-1] + a)
        cu_k.append(cu_k[-1] + b)
    s["lens"] = lens
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    s["cu_k"] = torch.tensor(cu_k, dtype=torch.int32, device="cuda")
    s["scale"] = dim ** -0.5
    if own:
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(n, heads * c["group"], dtype=torch.float32, device="cuda")
        need = _lib().fp4_prompt_attention_workspace_size(c["batch"], n, keys, heads * c["group"], heads, dim)
        s["ws"] = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    return s


# ----------------------------------------------------------------- passes


def _run_own(s):
    L, c = _lib(), s["case"]
    if c["op"] == "gemv":
        if c["fmt"] == MX:
            L.fp4_gemv_mxfp4(s["x"], s["w"], s["sw"], s["bias"], s["out"], c["m"], c["n"], c["k"])
        else:
            L.fp4_gemv_nvfp4(s["x"], s["w"], s["sw"], s["alpha"], s["bias"], s["out"], c["m"], c["n"], c["k"])
        return s["out"]
    if c["op"] == "experts":
        L.fp4_gemv_mxfp4_experts(s["x"], s["ids"], c["experts"], c["tokens"] * c["top"], c["top"], s["w"], s["sw"],
                                 s["bias"], s["out"], c["n"], c["k"])
        return s["out"]
    if c["op"] == "dispatch":
        L.fp4_moe_dispatch(s["x"], s["ids"], c["experts"], s["sorted"], s["offsets"], s["rows"])
        return {"sorted": s["sorted"], "offsets": s["offsets"], "rows": s["rows"]}
    if c["op"] == "combine":
        L.fp4_moe_combine(s["y"], s["rows"], s["weights"], s["out"])
        if not c["grad"]:
            return {"out": s["out"]}
        L.fp4_moe_combine_backward(s["grad"], s["y"], s["rows"], s["weights"], s["grad_y"], s["grad_w"])
        return {"out": s["out"], "grad_y": s["grad_y"], "grad_w": s["grad_w"]}
    if c["op"] == "norm":
        L.fp4_qk_norm_rope(s["q"], s["k"], s["q_out"], s["k_out"], s["q_weight"], s["k_weight"], s["eps"],
                           s["positions"], s["rope"])
        return {"q": s["q_out"], "k": s["k_out"]}
    L.fp4_prompt_attention(s["q"], s["k"], s["v"], s["out"], s["cu"], s["cu_k"], s["ws"], causal=bool(c["causal"]),
                           lse=s["lse"], softmax_scale=s["scale"])
    return {"out": s["out"], "lse": s["lse"]}


def _weight_values(codes, sw, fmt, alpha, n, k):
    """The float32 values [n, k] of a packed weight with swizzled scales."""
    group = 32 if fmt == MX else 16
    kb = k // group
    scales = sw.view(-(-n // 128), -(-kb // 4), 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-(-n // 128) * 128, -1)[:n, :kb]
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                        device=codes.device)
    v = grid[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()].unflatten(-1, (-1, group))
    if fmt == MX:
        return torch.ldexp(v, (scales.int() - 127).unsqueeze(-1)).flatten(-2)
    return (v * scales.contiguous().view(torch.float8_e4m3fn).float().unsqueeze(-1)).flatten(-2) * alpha


def _norm_rope(x, w, eps, positions, table, rot, layout):
    x = x.float()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w.float()
    cos, sin = table[positions.long()].unsqueeze(1).chunk(2, -1)
    r, rest = x[..., :rot], x[..., rot:]
    if layout == HALF:
        a, b = r.chunk(2, -1)
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    return torch.cat((r, rest), -1).to(torch.bfloat16)


def run(s):
    if own:
        return _run_own(s)
    c = s["case"]
    if c["op"] == "gemv":
        w = _weight_values(s["w"], s["sw"], c["fmt"], s["alpha"], c["n"], c["k"])
        return (s["x"].float() @ w.t() + s["bias"].float()).to(torch.bfloat16)
    if c["op"] == "experts":
        ids = s["ids"].flatten().long()
        w = torch.stack([_weight_values(a, b, MX, 1.0, c["n"], c["k"]) for a, b in
                         zip(s["w"].index_select(0, ids).unbind(), s["sw"].index_select(0, ids).unbind())])
        x = s["x"].float().repeat_interleave(c["top"], 0)
        return (torch.bmm(w, x.unsqueeze(-1)).squeeze(-1) + s["bias"][ids].float()).to(torch.bfloat16)
    if c["op"] == "dispatch":
        rows, offsets = _rows(s["ids"], c["experts"])
        flat = rows.flatten().long()
        live = flat >= 0
        token = torch.arange(flat.numel(), device="cuda") // c["top"]
        s["sorted"][flat[live]] = s["x"][token[live]]
        return {"sorted": s["sorted"], "offsets": offsets, "rows": rows}
    if c["op"] == "combine":
        rows = s["rows"].flatten().long()
        live = (rows >= 0).view(s["rows"].shape)
        y = s["y"][rows.clamp(min=0)].unflatten(0, s["rows"].shape).float()
        w = torch.where(live, s["weights"], torch.zeros_like(s["weights"]))
        got = {"out": (y * w.unsqueeze(-1)).sum(1).to(torch.bfloat16)}
        if c["grad"]:
            grad = s["grad"].float().unsqueeze(1)
            got["grad_w"] = torch.where(live, (y * grad).sum(-1), torch.zeros_like(w))
            s["grad_y"][rows[live.flatten()]] = (grad * w.unsqueeze(-1)).to(torch.bfloat16).flatten(0, 1)[live.flatten()]
            got["grad_y"] = s["grad_y"]
        return got
    if c["op"] == "norm":
        return {n: _norm_rope(s[n], s[n + "_weight"], s["eps"], s["positions"], s["table"], c["rot"], c["layout"])
                for n in ("q", "k")}
    return _attend(s)


def _attend(s):
    """Softmax attention of one sequence and key head at a time."""
    c, group = s["case"], s["case"]["group"]
    out = torch.zeros(s["q"].shape, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, device="cuda")
    row = at = 0
    for n, keys in s["lens"]:
        if n and keys:
            hidden = None
            if c["causal"]:
                i = torch.arange(n, device="cuda").unsqueeze(1) + (keys - n)
                hidden = torch.arange(keys, device="cuda") > i
            for h in range(c["heads"]):
                q = s["q"][row:row + n, h * group:(h + 1) * group].float().transpose(0, 1)
                x = torch.matmul(q, s["k"][at:at + keys, h].float().t()) * s["scale"]
                if hidden is not None:
                    x.masked_fill_(hidden, -math.inf)
                m = x.amax(-1, keepdim=True)
                m = torch.where(m == -math.inf, torch.zeros_like(m), m)
                x = torch.exp(x - m)
                total = x.sum(-1, keepdim=True)
                o = torch.matmul(x, s["v"][at:at + keys, h].float()) / torch.where(total == 0, torch.ones_like(total), total)
                out[row:row + n, h * group:(h + 1) * group] = o.transpose(0, 1).to(torch.bfloat16)
                lse[row:row + n, h * group:(h + 1) * group] = (m + torch.log(total)).squeeze(-1).t()
        row, at = row + n, at + keys
    return {"out": out, "lse": lse}


# ------------------------------------------------------------- in 64 bits


def _elements64(codes, bytes_, fmt, alpha, n, k):
    """Values [n, k] of a packed weight from the bit fields of its formats, in 64 bits."""
    r, b = torch.arange(n, device="cuda").unsqueeze(1), torch.arange(k // (32 if fmt == MX else 16), device="cuda")
    wide = -(-b.numel() // 4)
    raw = bytes_[((r // 128) * wide + b // 4) * 512 + (r % 32) * 16 + ((r % 128) // 32) * 4 + b % 4].int()
    if fmt == MX:
        scale = torch.exp2(raw.double() - 127)
    else:
        e, f = (raw >> 3) & 15, (raw & 7).double()
        scale = torch.where(e == 0, f * 2.0 ** -9, (1 + f / 8) * torch.exp2(e.double() - 7)) * alpha
    nib = torch.empty(n, k, dtype=torch.int16, device="cuda")
    nib[:, 0::2], nib[:, 1::2] = (codes % 16).short(), (codes // 16).short()
    e, f = (nib >> 1) & 3, (nib & 1).double()
    mag = torch.where(e == 0, f / 2, (1 + f / 2) * torch.exp2(e.double() - 1))
    return torch.where(nib >= 8, -mag, mag) * scale.repeat_interleave(k // b.numel(), 1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "gemv":
        return s["x"].double() @ _elements64(s["w"], s["sw"], c["fmt"], s["alpha"], c["n"], c["k"]).T + s["bias"].double()
    if c["op"] == "experts":
        rows = []
        for r, e in enumerate(s["ids"].flatten().tolist()):
            w = _elements64(s["w"][e], s["sw"][e], MX, 1.0, c["n"], c["k"])
            rows.append(w @ s["x"][r // c["top"]].double() + s["bias"][e].double())
        return torch.stack(rows)
    if c["op"] == "dispatch":
        ids = s["ids"].flatten().cpu().tolist()
        rows, offsets = [-1] * len(ids), [0]
        for e in range(c["experts"]):
            offsets.append(offsets[-1])
        of = [[] for _ in range(c["experts"])]
        for i, e in enumerate(ids):
            if 0 <= e < c["experts"]:
                of[e].append(i)
        at, got = 0, s["sorted"].double()
        for e, members in enumerate(of):
            for i in members:
                rows[i] = at
                at += 1
            offsets[e + 1] = at
        order = [i // c["top"] for members in of for i in members]
        got[:at] = s["x"].double()[torch.tensor(order, dtype=torch.int64, device="cuda")]
        return {"sorted": got, "offsets": torch.tensor(offsets, dtype=torch.int32, device="cuda"),
                "rows": torch.tensor(rows, dtype=torch.int32, device="cuda").view(s["ids"].shape)}
    if c["op"] == "combine":
        out = torch.zeros(c["tokens"], c["width"], dtype=torch.float64, device="cuda")
        grad_y = s["grad_y"].double()
        grad_w = torch.zeros(s["rows"].shape, dtype=torch.float64, device="cuda")
        for j in range(s["rows"].shape[1]):
            live = torch.nonzero(s["rows"][:, j] >= 0).squeeze(1)
            at = s["rows"][live, j].long()
            y, w = s["y"][at].double(), s["weights"][live, j].double().unsqueeze(1)
            out[live] += w * y
            if c["grad"]:
                g = s["grad"][live].double()
                grad_y[at] = w * g
                grad_w[live, j] = (g * y).sum(1)
        return {"out": out, "grad_y": grad_y, "grad_w": grad_w} if c["grad"] else {"out": out}
    if c["op"] == "norm":
        got, half = {}, c["rot"] // 2
        i = torch.arange(half, device="cuda")
        first, second = (i, i + half) if c["layout"] == HALF else (2 * i, 2 * i + 1)
        t = s["table"].double()[s["positions"].long()][:, None]
        for name in ("q", "k"):
            x = s[name].double()
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / c["dim"] + s["eps"]) * s[name + "_weight"].double()
            turned = torch.complex(x[..., first], x[..., second]) * torch.complex(t[..., :half], t[..., half:])
            x[..., first], x[..., second] = turned.real, turned.imag
            got[name] = x
        return got
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    row = at = 0
    for n, keys in s["lens"]:
        for h in range(c["heads"] * c["group"] if n and keys else 0):
            k, v = s["k"][at:at + keys, h // c["group"]].double(), s["v"][at:at + keys, h // c["group"]].double()
            x = (s["q"][row:row + n, h].double() @ k.T) * s["scale"]
            if c["causal"]:
                x += torch.full((n, keys), -math.inf, dtype=torch.float64, device="cuda").triu(keys - n + 1)
            total = torch.logsumexp(x, -1)
            p = torch.where(total.isfinite().unsqueeze(1), torch.exp(x - total.unsqueeze(1)), torch.zeros_like(x))
            out[row:row + n, h], lse[row:row + n, h] = p @ v, total
        row, at = row + n, at + keys
    return {"out": out, "lse": lse}
