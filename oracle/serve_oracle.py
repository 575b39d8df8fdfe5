"""CPU oracle of the serving-side operators: the 8-bit integer linear layer and
the 4-bit key/value cache with its attention.

TEST INFRASTRUCTURE, plain numpy, no code shared with the CUDA library. The
quantisers are stated twice: operation by operation in float32 (what the
library documents, code for code), and in float64 (the definition, for
error bounds). Products, softmax and sums are float64.
"""
from __future__ import annotations

import numpy as np

F32 = np.float32


# ---------------------------------------------------------------------------
# 8-bit rows
# ---------------------------------------------------------------------------
def int8_rows(x, s=None, inverse=False):
    """Codes int8 and steps float32 of x (float64 values exact in float32)
    [rows, d_in], operation by operation in float32."""
    v = np.asarray(x).astype(F32)
    with np.errstate(all="ignore"):
        if s is not None:
            v = v * ((F32(1) / s.astype(F32)) if inverse else s.astype(F32))
        bad = ~np.isfinite(v).all(axis=1)
        top = np.maximum(np.abs(np.where(np.isfinite(v), v, 0)).max(axis=1), F32(1e-8)).astype(F32)
        q = np.rint(v * (F32(127) / top)[:, None])
        step = (top / F32(127)).astype(F32)
    q[bad] = 0
    step[bad] = np.nan
    return q.astype(np.int8), step


def int8_product(xq, x_step, wq, w_step, bias=None):
    y = (xq.astype(np.float64) @ wq.astype(np.float64).T) * x_step.astype(np.float64)[:, None] * w_step.astype(np.float64)
    return y if bias is None else y + bias.astype(np.float64)


# ---------------------------------------------------------------------------
# 4-bit cache
# ---------------------------------------------------------------------------
def four_bit(x, g):
    """Codes uint8 [..., D], steps and zeros fp16 [..., D/g] of the group quantiser, in float32."""
    v = np.asarray(x).astype(F32)
    v = v.reshape(v.shape[:-1] + (v.shape[-1] // g, g))
    with np.errstate(all="ignore"):
        bad = ~np.isfinite(v).all(axis=-1)
        lo = np.minimum(v.min(axis=-1), F32(0))
        hi = np.maximum(v.max(axis=-1), F32(0))
        step = np.clip(((hi - lo) / F32(15)).astype(np.float16).astype(F32), F32(2.0 ** -24), F32(65504))
        inv = (F32(1) / step).astype(F32)
        zero = np.clip(np.rint(-lo * inv), 0, 15) + F32(0)  # +0, not -0
        code = np.clip(np.rint(v * inv[..., None]) + zero[..., None], 0, 15)
    code[bad] = 0
    zero[bad] = 0
    step[bad] = np.nan
    return code.astype(np.uint8).reshape(x.shape), step.astype(np.float16), zero.astype(np.float16)


def four_bit_values(code, step, zero):
    """float64 (code - zero) * step."""
    g = code.shape[-1] // step.shape[-1]
    rep = lambda a: np.repeat(a.astype(np.float64), g, axis=-1)  # noqa: E731
    return (code.astype(np.float64) - rep(zero)) * rep(step)


def strip_bytes(D, g):
    return 16 * D + 128 * (D // g)


def place(D, g, kind, t, c):
    """(byte, shift) in a strip of the code of channel c of the strip's token t;
    kind 0: keys, 1: values. Straight from the format's description."""
    if kind == 0:
        word, i = c // 8, c % 8
        j, q = word // 4, word % 4
        return t * (D // 2) + (q * (D // 32) + j) * 4 + i // 2, 4 * (i % 2)
    p, n, h, r = c // 32, (c // 16) % 2, (c // 8) % 2, c % 8
    q = (t % 8) // 2
    b = 2 * (t % 2) + t // 8
    return 8 * D + (((p * 8 + r) * 4 + q) * 2 + h) * 4 + b, 4 * n


def place_params(D, g, kind, t, j):
    """Byte of the (fp16 step, fp16 zero) of group j of the strip's token t."""
    return 16 * D + kind * 64 * (D // g) + (j * 16 + t) * 4


def write_token(cache, slot, head, page, D, g, kind, code, step, zero):
    """cache uint8 [pages, heads, page bytes], in place."""
    sb = strip_bytes(D, g)
    pos = slot % page
    base = (pos // 16) * sb
    blob = cache[slot // page, head]
    for c in range(D):
        byte, sh = place(D, g, kind, pos % 16, c)
        blob[base + byte] = (int(blob[base + byte]) & (0xF0 >> sh)) | (int(code[c]) << sh)
    for j in range(D // g):
        at = base + place_params(D, g, kind, pos % 16, j)
        blob[at:at + 4] = np.array([step[j], zero[j]], dtype=np.float16).view(np.uint8)


def tables(D, g):
    """byte [2, 16, D], shift [2, 16, D], parameter byte [2, 16, D/g] of a strip."""
    byte = np.zeros((2, 16, D), np.int64)
    shift = np.zeros((2, 16, D), np.int64)
    par = np.zeros((2, 16, D // g), np.int64)
    for kind in range(2):
        for t in range(16):
            for c in range(D):
                byte[kind, t, c], shift[kind, t, c] = place(D, g, kind, t, c)
            for j in range(D // g):
                par[kind, t, j] = place_params(D, g, kind, t, j)
    return byte, shift, par


def pack_pages(kc, ks, kz, vc, vs, vz, page):
    """uint8 [pages, heads, page bytes] of codes [pages, heads, page, D] and parameters [pages, heads, page, D/g]."""
    P, H, _, D = kc.shape
    ng = ks.shape[-1]
    byte, shift, par = tables(D, D // ng)
    sb = strip_bytes(D, D // ng)
    out = np.zeros((P, H, page // 16, sb), np.uint8)
    for kind, (c, s, z) in enumerate(((kc, ks, kz), (vc, vs, vz))):
        c = c.reshape(P, H, page // 16, 16, D)
        for n in (0, 4):  # low, then high nibbles (each byte has one of either)
            sel = shift[kind] == n
            out[..., byte[kind][sel]] |= (c[..., sel] << n).astype(np.uint8)
        for k, a in enumerate((s, z)):
            raw = np.ascontiguousarray(a.astype(np.float16)).view(np.uint8).reshape(P, H, page // 16, 16, ng, 2)
            for i in range(2):
                out[..., par[kind] + 2 * k + i] = raw[..., i]
    return out.reshape(P, H, page // 16 * sb)


def unpack_pages(cache, D, g):
    """Codes and parameters of a cache uint8 [pages, heads, page bytes]: per kind (code [P, H, page, D], step, zero)."""
    P, H, n = cache.shape
    byte, shift, par = tables(D, g)
    blob = cache.reshape(P, H, -1, strip_bytes(D, g))
    out = []
    for kind in range(2):
        code = (blob[..., byte[kind]] >> shift[kind].astype(np.uint8)) & 15
        at = np.stack([par[kind] + i for i in range(4)], -1)
        raw = np.ascontiguousarray(blob[..., at]).view(np.float16)  # [P, H, S, 16, ng, 2]
        flat = lambda a: a.reshape((P, H, -1) + a.shape[4:])  # noqa: E731
        out.append((flat(code), flat(raw[..., 0]), flat(raw[..., 1])))
    return out


def attention(q, k, v, share, scale, first_seen):
    """One sequence: q float64 [n, q_heads, D], k, v float64 [L, heads, D]; row j
    sees the first first_seen + j tokens. Returns out [n, q_heads, D], lse
    [n, q_heads] and the weights p [n, q_heads, L] (sum 1; rows that see nothing: 0)."""
    n, H, D = q.shape
    L = k.shape[0]
    out = np.zeros((n, H, D))
    lse = np.full((n, H), -np.inf)
    p = np.zeros((n, H, L))
    for e in range(H):
        s = scale * (q[:, e] @ k[:, e // share].T) if L else np.zeros((n, 0))
        for j in range(n):
            m = min(max(first_seen + j, 0), L)
            if m == 0:
                continue
            top = s[j, :m].max()
            w = np.exp(s[j, :m] - top)
            lse[j, e] = top + np.log(w.sum())
            p[j, e, :m] = w / w.sum()
            out[j, e] = p[j, e, :m] @ v[:m, e // share]
    return out, lse, p
