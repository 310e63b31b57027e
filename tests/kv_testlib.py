"""A plain statement of the attention-layer operators in numpy (64 bits, the quantizer's fp32 roundings apart), written from
include/pace_kv.h and sharing no code with the CUDA path."""
from __future__ import annotations

import numpy as np

FLT_MIN = np.float32(1.17549435e-38)


def bf16(x):
    """Nearest bf16 (ties to even) of fp32 values, as fp32."""
    u = np.asarray(x, np.float32).view(np.uint32)
    r = (u + 0x7FFF + ((u >> 16) & 1)) & np.uint32(0xFFFF0000)
    return r.astype(np.uint32).view(np.float32)


def quantize(x, bits):
    """x [..., d] fp32 -> (codes int, scale fp32, zero int), per group of 64."""
    g = np.asarray(x, np.float32).reshape(*x.shape[:-1], x.shape[-1] // 64, 64)
    g = np.where(np.isnan(g), np.float32(0), np.clip(g, -np.float32(2.0 ** 120), np.float32(2.0 ** 120)))
    if bits == 8:
        s = bf16(np.abs(g).max(-1) / np.float32(127))
    else:
        lo, hi = np.minimum(g.min(-1), np.float32(0)), np.maximum(g.max(-1), np.float32(0))
        s = bf16((hi - lo) / np.float32(15))
    live = s >= FLT_MIN
    s = np.where(live, s, np.float32(0))
    r = np.where(live, np.float32(1) / np.where(live, s, np.float32(1)), np.float32(0)).astype(np.float32)
    if bits == 8:
        z = np.zeros(s.shape, np.int64)
        c = np.clip(np.rint(g * r[..., None]), -127, 127).astype(np.int64)
    else:
        z = np.where(live, np.clip(np.rint(-lo * r), 0, 15), 0).astype(np.int64)
        c = np.clip(np.rint(g * r[..., None]).astype(np.int64) + z[..., None], 0, 15)
    return c, s, z


def held(x, bits):
    """The values the cache holds for x, in 64 bits (each product s * (code - z) is exact in fp32)."""
    c, s, z = quantize(x, bits)
    return (s[..., None].astype(np.float64) * (c - z[..., None])).reshape(x.shape)


def thetas(rot, base=10000.0, scaling="none", factor=1.0, orig_pos=0, beta_fast=32.0, beta_slow=1.0, mscale=0.0):
    i = np.arange(rot // 2)
    m = mscale or 1.0
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    th = base ** (-2.0 * i / rot)
    if scaling == "linear":
        th = th / factor
    if scaling == "parts":
        turns = orig_pos * th / (2 * np.pi)
        g = np.clip((turns - beta_slow) / (beta_fast - beta_slow), 0, 1)
        th = th * (g + (1 - g) / factor)
        m = mscale or 0.1 * np.log(factor) + 1.0
    return th, m


def rotate(x, pos, rot, layout="half", inverse=False, dtype=np.float64, **kw):
    """x [..., heads, d], pos [...]. dtype float32: the library's own roundings (table, products and sums once each)."""
    th, m = thetas(rot, **kw)
    ang = np.asarray(pos, np.float64)[..., None, None] * th
    c, s = (m * np.cos(ang)).astype(dtype), (m * np.sin(ang)).astype(dtype)
    if inverse:
        s = -s
    x = np.asarray(x, dtype)
    y = x.copy()
    h = rot // 2
    ia, ib = (np.arange(h), np.arange(h) + h) if layout == "half" else (2 * np.arange(h), 2 * np.arange(h) + 1)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return y


def attend(q, k, v, see, scale):
    """q [T, H, d], k, v [L, Hkv, d], see [T, L] -> [T, H, d]; rows that see nothing give zeros."""
    T, H, d = q.shape
    G = H // k.shape[1]
    out = np.zeros((T, H, d))
    for h in range(H):
        s = (q[:, h] @ k[:, h // G].T) * scale
        for t in range(T):
            j = np.flatnonzero(see[t])
            if j.size:
                p = np.exp(s[t, j] - s[t, j].max())
                out[t, h] = p @ v[j, h // G] / p.sum()
    return out
