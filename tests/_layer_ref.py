"""64-bit references of the operators around the FP4 linear layer, written from
their formulas (shares no code with the library)."""
from __future__ import annotations

import math

import numpy as np

MXFP4, MXFP8 = 0, 1


def element_grid(fmt):
    """(values, codes) of the non-negative finite elements of E2M1 / E4M3, ascending."""
    if fmt == MXFP4:
        v = [0.5 * m if e == 0 else (1 + m / 2) * 2.0 ** (e - 1) for e in range(4) for m in range(2)]
    else:
        v = [m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127]
    return np.array(v), np.arange(len(v))


def nearest_codes(y, fmt):
    """Code (sign bit included) of the nearest element, ties to the even code, saturating."""
    v, codes = element_grid(fmt)
    a = np.abs(y)
    hi = np.clip(np.searchsorted(v, a), 0, len(v) - 1)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - v[lo], v[hi] - a
    pick = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    pick = np.where(a >= v[-1], len(v) - 1, pick)
    return (pick + np.signbit(y) * (8 if fmt == MXFP4 else 128)).astype(np.uint8)


def element_values(codes, fmt):
    v, _ = element_grid(fmt)
    bit = 8 if fmt == MXFP4 else 128
    table = np.concatenate([v, [np.nan]]) if fmt == MXFP8 else v
    return np.where(codes & bit, -1.0, 1.0) * table[codes & (bit - 1)]


def mx_quantize(x, fmt):
    """float32 [..., D] -> (elements' codes [..., D], scale bytes [..., D / 32])."""
    b = np.asarray(x, np.float32).astype(np.float64).reshape(*x.shape[:-1], -1, 32)
    amax = np.abs(b).max(-1)
    bad = ~np.isfinite(b).all(-1)
    with np.errstate(divide="ignore"):
        e = np.floor(np.log2(np.where((amax > 0) & ~bad, amax, 1.0)))
    # log2 of a value just under a power of two may round up to it
    e = np.where(2.0 ** e > np.where(amax > 0, amax, 1.0), e - 1, e)
    e = np.where(amax > 0, e - (8 if fmt == MXFP8 else 2), -127).clip(-127, 127)
    y = np.where(bad[..., None], 0.0, b) / 2.0 ** e[..., None]
    codes = np.where(bad[..., None], 0, nearest_codes(y, fmt))
    return codes.reshape(x.shape).astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def mx_values(codes, scales, fmt):
    v = element_values(codes, fmt).reshape(*codes.shape[:-1], -1, 32)
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return (v * s[..., None]).reshape(codes.shape)


def pack(codes, fmt):
    return codes if fmt == MXFP8 else (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(packed, fmt):
    if fmt == MXFP8:
        return packed
    return np.stack((packed & 15, packed >> 4), -1).reshape(*packed.shape[:-1], -1)


def pairs(rot, layout):
    i = np.arange(rot // 2)
    return (i, i + rot // 2) if layout == 0 else (2 * i, 2 * i + 1)


def rotate(x, cos, sin, rot, layout, kind=np.float64):
    """x [T, H, D]; cos, sin [T, rot / 2]; one operation at a time in `kind`."""
    x = np.asarray(x).astype(kind)
    c, s = cos[:, None].astype(kind), sin[:, None].astype(kind)
    a, b = pairs(rot, layout)
    out = x.copy()
    out[..., a] = x[..., a] * c - x[..., b] * s
    out[..., b] = x[..., b] * c + x[..., a] * s
    return out


def attend(q, k, v, seen, scale):
    """q [R, D], k, v [T, D], seen [R, T] -> (out, lse, sum of softmax |v|, score magnitude bound)."""
    x = np.where(seen, (q @ np.where(seen.any(0)[:, None], k, 0.0).T) * scale, -np.inf)
    m = x.max(-1, initial=-np.inf)
    z = np.where(np.isneginf(m), 0.0, m)
    p = np.exp(x - z[:, None])
    total = p.sum(-1)
    with np.errstate(divide="ignore", invalid="ignore"):
        w = np.where(total[:, None] == 0, 0.0, p / total[:, None])
        lse = z + np.log(total)
    vv = np.where(seen[:, :, None], v[None], 0.0)
    out = np.einsum("rt,rtd->rd", w, vv)
    mag = (np.abs(q) @ np.where(seen.any(0)[:, None], np.abs(k), 0.0).T * scale)
    return out, lse, np.einsum("rt,rtd->rd", w, np.abs(vv)), np.where(seen, mag, 0.0).max(-1, initial=0.0)


def fp8_quantize(x, rows_per_scale):
    """float64 [R, K] -> (codes, scales float32): one scale per rows_per_scale x 128 block."""
    R, K = x.shape
    nb, kb = -(-R // rows_per_scale), -(-K // 128)
    codes, scales = np.zeros((R, K), np.uint8), np.zeros((nb, kb), np.float32)
    for i in range(nb):
        for j in range(kb):
            at = np.s_[i * rows_per_scale:(i + 1) * rows_per_scale, j * 128:(j + 1) * 128]
            b = x[at].astype(np.float32)
            if not np.isfinite(b).all():
                scales[i, j] = np.nan
                continue
            a = np.maximum(np.abs(b).max(), np.float32(2.0 ** -110))
            scales[i, j] = a / np.float32(448.0)
            codes[at] = nearest_codes((b * (np.float32(448.0) / a)).astype(np.float64), MXFP8)
    return codes, scales


def fp8_values(codes, scales, rows_per_scale):
    s = scales.astype(np.float64).repeat(rows_per_scale, 0)[: codes.shape[0]].repeat(128, 1)[:, : codes.shape[1]]
    return element_values(codes, MXFP8) * s


def rope_frequencies(rot, base, kind=0, factor=1.0, original=0, fast=32.0, slow=1.0):
    half = rot // 2
    w = [base ** (-2.0 * i / rot) for i in range(half)]
    if kind == 1:
        w = [f / factor for f in w]
    if kind == 2:
        def index(turns):
            return half * math.log(original / (turns * 2 * math.pi)) / math.log(base)
        low, high = max(math.floor(index(fast)), 0), min(math.ceil(index(slow)), half - 1)
        got = []
        for i, f in enumerate(w):
            t = (i - low) / (high - low) if high > low else float(i >= low)
            t = min(max(t, 0.0), 1.0)
            got.append(f * (1 - t) + f / factor * t)
        w = got
    return np.array(w)
