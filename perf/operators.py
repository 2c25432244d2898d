"""The operators around the FP4 linear layer that a decoder layer needs, as cases
to measure: the FP8 linear layer with a scale per block of 128 (the layers a
mixed-precision checkpoint keeps out of FP4), rotary positions, the MX-quantized
paged key/value cache (written and read back) and attention of drafted tokens over
that cache.

`run` computes them in plain torch operations in 32 bits (`own` false) or through
the library's entry points (`own` true), `exact` from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

MXFP4, MXFP8 = 0, 1   # the library's numbering of the MX formats
HALF, INTERLEAVED = 0, 1


def _lib():
    from nvfp4_mxfp4_w4a4_gb300 import fp4lin

    fp4lin.load()
    return fp4lin


# ------------------------------------------------------------------ cases


def listed():
    return [
        # FP8 linear: one token through a 4096-wide projection, a decode batch through
        # the decode workload's layer, a ragged prefill chunk through the prefill layer
        dict(name="fp8_linear_m1", op="fp8", m=1, n=4096, k=4096),
        dict(name="fp8_linear_m64", op="fp8", m=64, n=14336, k=4096),
        dict(name="fp8_linear_m2041", op="fp8", m=2041, n=18432, k=7168),
        # rotary positions of the queries of a decode batch, and of a long prefill's
        # (interleaved pairs, half of each head rotated)
        dict(name="rope_decode", op="rope", t=64, heads=32, dim=128, rot=128, layout=HALF, gap=2048),
        dict(name="rope_prefill", op="rope", t=16381, heads=56, dim=128, rot=64, layout=INTERLEAVED, gap=0),
        # a decode batch's keys (rotated on the way) and values into the cache
        dict(name="kv_append_decode", op="append", fmt=MXFP8, batch=64, chunk=1, ctx=2000, heads=8, dim=128, page=64,
             layout=HALF, rot=128),
        # one step of a chunked prefill: the chunk goes into the cache, and the whole
        # context comes back in bf16 for the chunk's attention
        dict(name="kv_chunk_mxfp8", op="chunk", fmt=MXFP8, batch=4, chunk=1021, ctx=7000, heads=8, dim=128, page=64,
             layout=HALF, rot=128),
        dict(name="kv_chunk_mxfp4", op="chunk", fmt=MXFP4, batch=8, chunk=509, ctx=16000, heads=8, dim=128, page=32,
             layout=INTERLEAVED, rot=64),
        # one token of one short sequence (latency), a decode batch, a tree of drafted
        # tokens for each of a few sequences, and a few drafted tokens over one very long one
        dict(name="attn_one_token", op="attn", fmt=MXFP8, batch=1, draft=1, ctx=503, heads=8, group=4, dim=128, page=64,
             tree=0),
        dict(name="attn_decode_batch", op="attn", fmt=MXFP8, batch=64, draft=1, ctx=8190, heads=8, group=4, dim=128,
             page=64, tree=0),
        dict(name="attn_tree_mxfp4", op="attn", fmt=MXFP4, batch=8, draft=31, ctx=16001, heads=8, group=4, dim=128,
             page=32, tree=1),
        dict(name="attn_long_context", op="attn", fmt=MXFP8, batch=1, draft=4, ctx=262139, heads=8, group=8, dim=128,
             page=64, tree=1),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    case = _drawn(rng)
    return {key: value + 16 if value == 3072 else value for key, value in case.items()}


def _drawn(rng):
    op = rng.choice(["fp8", "fp8", "rope", "append", "chunk", "attn", "attn", "attn"])
    if op == "fp8":
        return dict(op=op, m=_log(rng, 1, 2041), n=8 * _log(rng, 64, 2304), k=16 * _log(rng, 16, 448))
    dim = rng.choice([64, 128])
    rot = rng.choice([dim, dim // 2])
    layout = rng.choice([HALF, INTERLEAVED])
    if op == "rope":
        return dict(op=op, t=_log(rng, 1, 16381), heads=rng.randint(1, 56), dim=dim, rot=rot, layout=layout,
                    gap=rng.choice([0, 128, 2048]))
    fmt = rng.choice([MXFP4, MXFP8])
    page = rng.choice([16, 32, 48, 64, 128])
    heads = rng.choice([1, 2, 4, 8])
    if op == "append":
        return dict(op=op, fmt=MXFP8, batch=_log(rng, 1, 128), chunk=_log(rng, 1, 64), ctx=_log(rng, 1, 2000),
                    heads=heads, dim=dim, page=page, layout=layout, rot=rot)
    if op == "chunk":
        return dict(op=op, fmt=fmt, batch=_log(rng, 1, 8), chunk=_log(rng, 1, 1021), ctx=_log(rng, 1, 7000),
                    heads=heads, dim=dim, page=page, layout=layout, rot=rot)
    batch = _log(rng, 1, 64)
    return dict(op=op, fmt=fmt, batch=batch, draft=_log(rng, 1, 64 if batch <= 8 else 8),
                ctx=_log(rng, 1, min(131072, 262139 // batch)), heads=heads, group=rng.randint(1, 8), dim=dim, page=page,
                tree=rng.choice([0, 1]))


def _lens(c):
    """Ragged per-sequence (context tokens, new tokens): the first sequence has the
    whole of both, and of four or more the last has no context."""
    r = random.Random("%d %d %d" % (c["batch"], c["ctx"], c.get("chunk", c.get("draft"))))
    new = c.get("chunk", c.get("draft"))
    got = [(c["ctx"], new)]
    for b in range(1, c["batch"]):
        got.append((0 if b >= 3 and b == c["batch"] - 1 else r.randint((c["ctx"] + 1) // 2, c["ctx"]), r.randint((new + 1) // 2, new)))
    return got


def _token_bytes(c):
    """Bytes of one token's keys (or values) in the cache: codes and a scale per 32."""
    return c["heads"] * (c["dim"] * (1 if c["fmt"] == MXFP8 else 0.5) + c["dim"] // 32)


def work(case):
    c = case
    if c["op"] == "fp8":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": 2 * m * k + n * k + 4 * -(-n // 128) * -(-k // 128) + 2 * n + 2 * m * n, "flops": 2 * m * n * k}
    if c["op"] == "rope":
        return {"bytes": c["t"] * (4 * c["heads"] * c["dim"] + 4 * c["rot"] + 4), "flops": 3 * c["t"] * c["heads"] * c["rot"]}
    lens = _lens(c)
    new, ctx = sum(n for _, n in lens), sum(l for l, _ in lens)
    if c["op"] in ("append", "chunk"):
        b = new * (2 * (2 * c["heads"] * c["dim"] + _token_bytes(c)) + 4 * c["rot"] + 12)
        if c["op"] == "chunk":
            b += (new + ctx) * 2 * (_token_bytes(c) + 2 * c["heads"] * c["dim"])
        return {"bytes": b, "flops": 3 * new * c["heads"] * c["rot"]}
    hq = c["heads"] * c["group"]
    pairs = sum(n * l + n * n for l, n in lens)
    return {"bytes": (ctx + new) * 2 * _token_bytes(c) + new * hq * (4 * c["dim"] + 4), "flops": 4 * pairs * hq * c["dim"]}


# ------------------------------------------------------- plain operations


def _e4m3(y):
    """The nearest E4M3 value (ties to even, saturating), as float8."""
    return y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _e2m1_code(y):
    """The code of the nearest E2M1 value (ties to the even code, saturating)."""
    a = y.abs()
    code = (a > 0.25).to(torch.uint8)
    code += a >= 0.75
    code += a > 1.25
    code += a >= 1.75
    code += a > 2.5
    code += a >= 3.5
    code += a > 5.0
    return code + 8 * torch.signbit(y).to(torch.uint8)


def _mx_quantize(x, fmt):
    """x [..., D] float32 -> (codes, E8M0 bytes): a power of two for each 32 elements."""
    blocks = x.unflatten(-1, (-1, 32))
    _, e = torch.frexp(blocks.abs().amax(-1))
    e = (e - 1 - (8 if fmt == MXFP8 else 2)).clamp(-127, 127)
    e = torch.where(blocks.abs().amax(-1) > 0, e, torch.full_like(e, -127))
    y = torch.ldexp(blocks, -e.unsqueeze(-1)).flatten(-2)
    if fmt == MXFP8:
        codes = _e4m3(y).view(torch.uint8)
    else:
        n = _e2m1_code(y).unflatten(-1, (-1, 2))
        codes = n[..., 0] | (n[..., 1] << 4)
    return codes, (e + 127).to(torch.uint8)


def _mx_values(codes, scales, fmt):
    """The float32 values of MX codes [..., bytes] with scales [..., D / 32]."""
    if fmt == MXFP8:
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                            device=codes.device)
        v = grid[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()]
    return torch.ldexp(v.unflatten(-1, (-1, 32)), (scales.int() - 127).unsqueeze(-1)).flatten(-2)


def _rotate(x, positions, table, rot, layout):
    """x [T, H, D] float32 with the first `rot` of each head rotated by its position."""
    cos, sin = table[positions.long()].unsqueeze(1).chunk(2, -1)
    r, rest = x[..., :rot], x[..., rot:]
    if layout == HALF:
        a, b = r.chunk(2, -1)
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    return torch.cat((r, rest), -1)


# ----------------------------------------------------------------- inputs


def _table(positions, rot):
    """cos and sin [positions, rot] of base 500000 interpolated by 4, rounded from 64 bits."""
    f = 500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot) / 4.0
    a = torch.arange(positions, dtype=torch.float64, device="cuda").unsqueeze(1) * f
    return torch.cat((a.cos(), a.sin()), -1).float()


def _heads(g, t, heads, dim, gap=0):
    """Projections [t, heads, dim] bf16, as a slice of rows with `gap` other elements;
    a few channels of each head are several times the others'."""
    x = torch.randn(t, heads * dim + gap, generator=g, device="cuda")
    big = 1.0 + 7.0 * (torch.arange(heads * dim + gap, device="cuda") % 61 == 5).float()
    return (x * big).to(torch.bfloat16)[:, : heads * dim].unflatten(1, (heads, dim))


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": c}
    if c["op"] == "fp8":
        m, n, k = c["m"], c["n"], c["k"]
        nb, kb = -(-n // 128), -(-k // 128)
        s["x"] = torch.randn(m, k, generator=g, device="cuda")
        s["x"] *= 1.0 + 15.0 * (torch.rand(m, k, generator=g, device="cuda") < 0.005)
        s["x"] = s["x"].to(torch.bfloat16)
        w = torch.zeros(nb * 128, kb * 128, device="cuda")
        w[:n, :k] = 0.02 * torch.randn(n, k, generator=g, device="cuda")
        w = w.view(nb, 128, kb, 128)
        s["sw"] = w.abs().amax((1, 3)) / 448.0
        s["w"] = _e4m3(w / s["sw"].view(nb, 1, kb, 1)).view(torch.uint8).view(nb * 128, kb * 128)[:n, :k].contiguous()
        s["bias"] = (0.01 * torch.randn(n, generator=g, device="cuda")).to(torch.bfloat16)
        if own:
            L = _lib()
            s["out"] = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
            s["ws"] = torch.zeros(L.fp4_linear_fp8_b128_workspace_size(m, n, k), dtype=torch.uint8, device="cuda")
        return s
    if c["op"] == "rope":
        s["x"] = _heads(g, c["t"], c["heads"], c["dim"], c["gap"])
        s["positions"] = torch.randint(0, 32768, (c["t"],), generator=g, device="cuda", dtype=torch.int32)
        s["table"] = _table(32768, c["rot"])
        if own:
            s["rope"] = _lib().rope_params(s["table"], c["rot"], c["layout"])
            s["out"] = torch.empty(c["t"], c["heads"], c["dim"], dtype=torch.bfloat16, device="cuda")
        return s

    # a pool of pages, twice as many as are needed, handed out in random order
    lens = _lens(c)
    page, heads, dim, fmt, batch = c["page"], c["heads"], c["dim"], c["fmt"], c["batch"]
    pages = [-(-(l + n) // page) for l, n in lens]
    pool = 2 * sum(pages)
    order = torch.randperm(pool, generator=g, device="cuda", dtype=torch.int64).int()
    starts = [sum(pages[:b]) for b in range(batch)]
    width = max(pages)
    index = torch.tensor([[starts[b] + min(i, pages[b] - 1) for i in range(width)] for b in range(batch)], device="cuda")
    s["table_pages"] = order[index]
    s["ctx"] = torch.tensor([l for l, _ in lens], dtype=torch.int32, device="cuda")
    cu = [0]
    for _, n in lens:
        cu.append(cu[-1] + n)
    s["cu_new"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    total = cu[-1]
    for name in ("k", "v"):
        x = torch.randn(pool, heads, page, dim, generator=g, device="cuda")
        x *= 1.0 + 7.0 * (torch.arange(dim, device="cuda") % 61 == 5)
        s[name + "_codes"], s[name + "_scales"] = _mx_quantize(x, fmt)
        del x
    if c["op"] == "attn":
        s["q"] = torch.randn(total, heads * c["group"], dim, generator=g, device="cuda").to(torch.bfloat16)
        s["mask"] = None
        if c["tree"]:
            # node j of a sequence's tree hangs on a random earlier one and sees its
            # ancestors and itself; the last node of every third tree is padding and
            # sees no drafted token
            words = -(-c["draft"] // 32)
            rows = torch.zeros(batch, c["draft"], words * 32, dtype=torch.bool)
            r = random.Random(seed)
            for b, (_, n) in enumerate(lens):
                for j in range(n):
                    if j:
                        rows[b, j] = rows[b, r.randint(max(0, j - 6), j - 1)]
                    rows[b, j, j] = True
                if b % 3 == 2:
                    rows[b, n - 1] = False
            rows = torch.cat([rows[b, :n] for b, (_, n) in enumerate(lens)])
            bits = rows.view(total, words, 32).long() << torch.arange(32)
            s["mask"] = bits.sum(-1).to(torch.int64).cuda().to(torch.uint32).view(torch.int32)
        s["scale"] = dim ** -0.5
        s["seq"] = torch.tensor([b for b, (_, n) in enumerate(lens) for _ in range(n)], device="cuda")
        s["node"] = torch.tensor([j for _, n in lens for j in range(n)], device="cuda")
        if own:
            L = _lib()
            s["cache"] = L.kv_cache(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], page, fmt)
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(total, heads * c["group"], dtype=torch.float32, device="cuda")
            need = L.fp4_kv_attention_workspace_size(batch, total, heads * c["group"], heads, dim, c["ctx"] + c["draft"],
                                                     c["draft"])
            s["ws"] = torch.zeros(max(need, 1), dtype=torch.uint8, device="cuda")
        return s
    kv = _heads(g, total, 2 * heads, dim)
    s["k"], s["v"] = kv[:, :heads], kv[:, heads:]
    s["positions"] = torch.tensor([l + j for l, n in lens for j in range(n)], dtype=torch.int32, device="cuda")
    seq = torch.tensor([b for b, (_, n) in enumerate(lens) for _ in range(n)], device="cuda")
    at = s["positions"].long()
    s["slots"] = s["table_pages"][seq, at // page].long() * page + at % page
    s["table"] = _table(c["ctx"] + c["chunk"], c["rot"])
    if c["op"] == "chunk":
        cl = [0]
        for l, n in lens:
            cl.append(cl[-1] + l + n)
        s["cu_all"] = torch.tensor(cl, dtype=torch.int32, device="cuda")
        s["row_seq"] = torch.repeat_interleave(torch.arange(batch, device="cuda"), s["cu_all"].diff().long())
        s["row_pos"] = torch.arange(cl[-1], device="cuda") - s["cu_all"].long()[s["row_seq"]]
    if own:
        L = _lib()
        s["cache"] = L.kv_cache(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], page, fmt)
        s["rope"] = L.rope_params(s["table"], c["rot"], c["layout"])
        if c["op"] == "chunk":
            s["k_out"] = torch.empty(cl[-1], heads, dim, dtype=torch.bfloat16, device="cuda")
            s["v_out"] = torch.empty(cl[-1], heads, dim, dtype=torch.bfloat16, device="cuda")
    return s


# ----------------------------------------------------------------- passes


def _run_own(s):
    L, c = _lib(), s["case"]
    if c["op"] == "fp8":
        L.fp4_linear_fp8_b128(s["x"], s["w"], s["sw"], s["bias"], s["out"], c["m"], c["n"], c["k"], s["ws"])
        return s["out"]
    if c["op"] == "rope":
        L.fp4_rope(s["x"], s["out"], s["positions"], s["rope"])
        return s["out"]
    if c["op"] == "attn":
        L.fp4_kv_attention(s["cache"], s["q"], s["out"], s["table_pages"], s["ctx"], s["cu_new"], c["ctx"] + c["draft"],
                           c["draft"], s["ws"], tree_mask=s["mask"], lse=s["lse"], softmax_scale=s["scale"])
        return {"out": s["out"], "lse": s["lse"]}
    L.fp4_kv_append(s["cache"], s["k"], s["v"], s["slots"], rope=s["rope"], positions=s["positions"])
    if c["op"] == "chunk":
        L.fp4_kv_read(s["cache"], s["table_pages"], s["cu_all"], s["k_out"], s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"]}
    return _append_outputs(s)


def _append_outputs(s):
    """The cache as the 8-bit values that its bytes stand for."""
    return {"k": s["k_codes"].view(torch.float8_e4m3fn), "ks": s["k_scales"].view(torch.float8_e8m0fnu),
            "v": s["v_codes"].view(torch.float8_e4m3fn), "vs": s["v_scales"].view(torch.float8_e8m0fnu)}


def run(s):
    if own:
        return _run_own(s)
    c = s["case"]
    if c["op"] == "fp8":
        m, n, k = c["m"], c["n"], c["k"]
        kb = -(-k // 128)
        x = torch.nn.functional.pad(s["x"].float(), (0, kb * 128 - k)).view(m, kb, 128)
        amax = x.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -110)
        x = (_e4m3(x * (448.0 / amax)).float() * (amax / 448.0)).view(m, kb * 128)[:, :k]
        w = s["w"].view(torch.float8_e4m3fn).float()
        w = w * s["sw"].repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
        return (x @ w.t() + s["bias"].float()).to(torch.bfloat16)
    if c["op"] == "rope":
        return _rotate(s["x"].float(), s["positions"], s["table"], c["rot"], c["layout"]).to(torch.bfloat16)
    if c["op"] == "attn":
        return _attend(s, torch.float32)
    page = c["page"]
    p, o = s["slots"] // page, s["slots"] % page
    for name in ("k", "v"):
        x = s[name].float()
        if name == "k":
            x = _rotate(x, s["positions"], s["table"], c["rot"], c["layout"])
        codes, scales = _mx_quantize(x, c["fmt"])
        s[name + "_codes"][p, :, o] = codes
        s[name + "_scales"][p, :, o] = scales
    if c["op"] == "append":
        return _append_outputs(s)
    p, o = s["table_pages"].long()[s["row_seq"], s["row_pos"] // page], s["row_pos"] % page
    return {name: _mx_values(s[name + "_codes"][p, :, o], s[name + "_scales"][p, :, o], c["fmt"]).to(torch.bfloat16)
            for name in ("k", "v")}


def _attend(s, kind):
    """Softmax attention of the drafted tokens over context and tree, padded to the longest sequence."""
    c, pages = s["case"], s["table_pages"].long()
    batch, draft, heads, group, dim = c["batch"], c["draft"], c["heads"], c["group"], c["dim"]
    width = pages.shape[1] * c["page"]
    k, v = (_mx_values(s[n + "_codes"][pages], s[n + "_scales"][pages], c["fmt"]).to(kind).transpose(2, 3)
            .reshape(batch, width, heads, dim) for n in ("k", "v"))
    q = torch.zeros(batch, draft, heads, group, dim, dtype=kind, device="cuda")
    q[s["seq"], s["node"]] = s["q"].to(kind).unflatten(1, (heads, group))
    at = torch.arange(width, device="cuda") - s["ctx"].long()[s["seq"]].unsqueeze(1)   # [T, width]: drafted index
    if s["mask"] is None:
        seen = at <= s["node"].unsqueeze(1)
    else:
        inside = (at >= 0) & (at < draft)
        i = torch.where(inside, at, torch.zeros_like(at))
        seen = (at < 0) | (inside & ((s["mask"].long().gather(1, i // 32) >> (i % 32)) & 1).bool())
    visible = torch.zeros(batch, draft, width, dtype=torch.bool, device="cuda")
    visible[s["seq"], s["node"]] = seen
    x = torch.einsum("bnhgd,bthd->bhgnt", q, k) * s["scale"]
    x = x.masked_fill(~visible[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    x = torch.exp(x - m)
    total = x.sum(-1, keepdim=True)
    out = torch.einsum("bhgnt,bthd->bhgnd", x, v) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (m + torch.log(total)).squeeze(-1)
    out = out.permute(0, 3, 1, 2, 4)[s["seq"], s["node"]].flatten(1, 2)
    lse = lse.permute(0, 3, 1, 2)[s["seq"], s["node"]].flatten(1, 2)
    return {"out": out.to(torch.bfloat16) if kind == torch.float32 else out, "lse": lse}


# ------------------------------------------------------------- in 64 bits


def _mx_values64(codes, scales, fmt):
    """Values of MX codes from the bit fields of the element formats, in 64 bits."""
    if fmt == MXFP8:
        b = codes.int()
        e, f = (b >> 3) & 15, (b & 7).double()
        mag = torch.where(e == 0, f * 2.0 ** -9, (1 + f / 8) * torch.exp2(e.double() - 7))
        sign = b >> 7
    else:
        b = torch.stack((codes % 16, codes // 16), -1).reshape(*codes.shape[:-1], -1).int()
        e, f = (b >> 1) & 3, (b & 1).double()
        mag = torch.where(e == 0, f / 2, (1 + f / 2) * torch.exp2(e.double() - 1))
        sign = b >> 3
    return torch.where(sign == 1, -mag, mag) * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def _nearest64(y, fmt):
    """The nearest value of the element format, ties to the even mantissa, saturating."""
    top, low, bits = (448.0, -6, 3) if fmt == MXFP8 else (6.0, 0, 1)
    _, e = torch.frexp(y)
    step = torch.exp2((e - 1).clamp(min=low).double() - bits)
    return (torch.round(y / step) * step).clamp(-top, top)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "fp8":
        m, n, k = c["m"], c["n"], c["k"]
        x = s["x"].double()
        for at in range(0, k, 128):
            scale = x[:, at:at + 128].abs().amax(1, keepdim=True) / 448
            scale = torch.where(scale == 0, torch.ones_like(scale), scale)
            x[:, at:at + 128] = _nearest64(x[:, at:at + 128] / scale, MXFP8) * scale
        one = torch.full((n, -(-k // 32)), 127, device="cuda")
        w = _mx_values64(torch.nn.functional.pad(s["w"], (0, -k % 32)), one, MXFP8)[:, :k].contiguous()
        row, col = torch.arange(n, device="cuda") // 128, torch.arange(k, device="cuda") // 128
        w *= s["sw"].double()[row][:, col]
        return x @ w.T + s["bias"].double()

    def rotate(x, positions):
        x = x.double()
        half = c["rot"] // 2
        i = torch.arange(half, device="cuda")
        first, second = (i, i + half) if c["layout"] == HALF else (2 * i, 2 * i + 1)
        t = s["table"].double()[positions.long()][:, None]
        turned = torch.complex(x[..., first], x[..., second]) * torch.complex(t[..., :half], t[..., half:])
        out = x.clone()
        out[..., first], out[..., second] = turned.real, turned.imag
        return out

    if c["op"] == "rope":
        return rotate(s["x"], s["positions"])
    if c["op"] in ("append", "chunk"):
        page, fmt = c["page"], c["fmt"]
        got = {}
        for name in ("k", "v"):
            x = rotate(s[name], s["positions"]) if name == "k" else s[name].double()
            x = x.reshape(*x.shape[:-1], -1, 32)
            _, e = torch.frexp(x.abs().amax(-1))
            e = (e - 1 - (8 if fmt == MXFP8 else 2)).clamp(-127, 127).double()
            y = _nearest64(x / torch.exp2(e).unsqueeze(-1), fmt)
            p, o = s["slots"] // page, s["slots"] % page
            if c["op"] == "append":
                one = torch.full_like(s[name + "_scales"], 127)
                codes, scales = _mx_values64(s[name + "_codes"], one, fmt), torch.exp2(s[name + "_scales"].double() - 127)
                codes[p, :, o], scales[p, :, o] = y.flatten(-2), torch.exp2(e)
                got |= {name: codes, name + "s": scales}
            else:
                whole = _mx_values64(s[name + "_codes"], s[name + "_scales"], fmt)
                whole[p, :, o] = (y * torch.exp2(e).unsqueeze(-1)).flatten(-2)
                row = s["row_pos"]
                got[name] = whole[s["table_pages"].long()[s["row_seq"], row // page], :, row % page]
        return got

    # attention, one sequence at a time
    outs, lses, row = [], [], 0
    for b, (ctx, n) in enumerate(_lens(c)):
        pages = s["table_pages"][b, : -(-(ctx + n) // c["page"])].long()
        k, v = (_mx_values64(s[x + "_codes"][pages], s[x + "_scales"][pages], c["fmt"]).movedim(1, 0).flatten(1, 2)[:, : ctx + n]
                for x in ("k", "v"))
        q = s["q"][row:row + n].double().reshape(n, c["heads"], c["group"], -1).permute(1, 2, 0, 3).flatten(1, 2)
        sees = torch.ones(n, ctx + n, dtype=torch.bool, device="cuda")
        if s["mask"] is None:
            sees[:, ctx:] = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
        else:
            words = s["mask"][row:row + n].cpu().tolist()
            sees[:, ctx:] = torch.tensor([[(words[i][j // 32] >> (j % 32)) & 1 for j in range(n)] for i in range(n)],
                                         dtype=torch.bool, device="cuda").view(n, n)
        x = (q @ k.transpose(1, 2)) * s["scale"]
        x = x.masked_fill(~sees.repeat(c["group"], 1), -math.inf)
        lse = torch.logsumexp(x, -1)
        p = torch.where(lse.isfinite().unsqueeze(-1), torch.exp(x - lse.unsqueeze(-1)), torch.zeros_like(x))
        shape = (c["heads"], c["group"], n)
        outs.append((p @ v).reshape(*shape, -1).permute(2, 0, 1, 3).flatten(1, 2))
        lses.append(lse.reshape(shape).permute(2, 0, 1).flatten(1, 2))
        row += n
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
