"""CPU oracle for the dense half of a batched decode block — TEST INFRASTRUCTURE
ONLY, like the rest of ``oracle``: numpy in fp64 from the formulas in
``include/spffn_block.h``, sharing no code with the CUDA side.

The 4-bit cache's values are defined by roundings to fp16 (step, zero) and to
codes; ``quantise`` takes the arithmetic's type, so that a test can ask for the
fp32 definition (bit for bit) or for the same steps in fp64.
"""
from __future__ import annotations

import numpy as np


def norm_quant(x, y, g, eps):
    """(u, q before rounding, scale): u = x + y; w = u g; w 127 / max|w|; max|w| rs / 127, in fp64."""
    u = np.asarray(x, np.float64) + (0.0 if y is None else np.asarray(y, np.float64))
    w = u * (1.0 if g is None else np.asarray(g, np.float64))
    a = np.abs(w).max(axis=1, keepdims=True)
    rs = 1.0 / np.sqrt(np.mean(u * u, axis=1) + eps)
    return u, np.divide(127.0 * w, a, out=np.zeros_like(w), where=a > 0), a[:, 0] * rs / 127.0


def mm8(A, W, sa, sw, bias=None):
    """Integer sums in int64, scales and bias in fp64."""
    acc = np.asarray(A, np.int64) @ np.asarray(W, np.int64).T
    y = acc * np.asarray(sa, np.float64)[:, None] * np.asarray(sw, np.float64)[None, :]
    return y if bias is None else y + np.asarray(bias, np.float64)[None, :]


def rotate(x, positions, freqs, interleaved, amplitude=1.0):
    """Rows x [T, heads, dh]: the first 2 len(freqs) dims turned by position freqs."""
    x = np.array(x, np.float64)
    n = len(freqs)
    if n == 0:
        return x
    ang = np.asarray(positions, np.float64)[:, None] * np.asarray(freqs, np.float64)[None, :]
    c, s = amplitude * np.cos(ang)[:, None, :], amplitude * np.sin(ang)[:, None, :]
    first = slice(0, 2 * n, 2) if interleaved else slice(0, n)
    second = slice(1, 2 * n, 2) if interleaved else slice(n, 2 * n)
    a, b = x[..., first].copy(), x[..., second].copy()
    x[..., first], x[..., second] = a * c - b * s, b * c + a * s
    return x


def quantise(x, dtype=np.float32):
    """Rows [..., dh] -> (codes uint8 [..., dh], step, zero fp16 [..., dh / 32])."""
    u = np.asarray(x, dtype).reshape(*np.shape(x)[:-1], -1, 32)
    lo, hi = u.min(axis=-1), u.max(axis=-1)
    with np.errstate(all="ignore"):
        zero = np.clip(lo, -65504, 65504).astype(np.float16)
        step = np.clip(((hi - lo) * (dtype(1) / dtype(15))).astype(dtype), -65504, 65504).astype(np.float16)
        step = np.where(np.isfinite(u).all(axis=-1), step, np.float16(np.nan))
        code = np.rint((u - zero.astype(dtype)[..., None]) / step.astype(dtype)[..., None])
    code = np.where((step > 0)[..., None], np.clip(code, 0, 15), 0)
    return code.astype(np.uint8).reshape(np.shape(x)), step, zero


def values(codes, step, zero):
    """code step + zero in fp64."""
    c = np.asarray(codes, np.float64).reshape(*codes.shape[:-1], -1, 32)
    return (c * step.astype(np.float64)[..., None] + zero.astype(np.float64)[..., None]).reshape(codes.shape)


def places(tok, dim, ng):
    """Byte of the block (16 tokens) and shift of a code, and halfword of its step, for K and V: the block format, one
    element at a time.  Returns ((k byte, k step), (v byte, v step), shift)."""
    g, e = dim // 32, dim % 32
    kb = (tok * 4 + e // 8) * 4 * ng + g * 4 + e % 8 // 2
    vb = 256 * ng + ((tok // 8 * 8 + e // 4) * 8 + tok % 8) * 2 * ng + g * 2 + e % 4 // 2
    ks = (512 * ng) // 2 + tok * ng + g
    vs = (576 * ng) // 2 + ((tok // 8 * 4 + tok % 8 // 2) * ng + g) * 2 + tok % 2
    return (kb, ks), (vb, vs), 4 * (dim % 2)


def read_pool(pool, page, kvh, dh):
    """uint8 pool [pages, kvh, page / 16, 20 dh] -> dict of codes, step, zero of K and V, [pages, page, kvh, ...]."""
    ng = dh // 32
    pool = np.ascontiguousarray(pool).reshape(-1, kvh, page // 16, 640 * ng)
    half = pool.view(np.float16)
    tok, dim = np.meshgrid(np.arange(16), np.arange(dh), indexing="ij")
    k, v, shift = places(tok, dim, ng)
    out = {}
    for name, (byte, step) in (("K", k), ("V", v)):
        code = (pool[..., byte] >> shift.astype(np.uint8)) & 15
        lay = lambda a: a.transpose(0, 2, 3, 1, 4).reshape(a.shape[0], page, kvh, a.shape[-1])  # noqa: E731
        out[name] = (lay(code), lay(half[..., step[:, ::32]]), lay(half[..., step[:, ::32] + 16 * ng]))
    return out


def write_pool(K, V, page, kvh, dh):
    """The inverse: K, V = (codes, step, zero) of [pages, page, kvh, ...] -> uint8 pool."""
    ng = dh // 32
    pages = K[0].shape[0]
    pool = np.zeros((pages, kvh, page // 16, 640 * ng), np.uint8)
    half = pool.view(np.float16)
    tok, dim = np.meshgrid(np.arange(16), np.arange(dh), indexing="ij")
    k, v, shift = places(tok, dim, ng)
    for (byte, step), (code, st, ze) in ((k, K), (v, V)):
        blocks = lambda a: a.reshape(pages, page // 16, 16, kvh, -1).transpose(0, 3, 1, 2, 4)  # noqa: E731
        c = blocks(code)
        for e in (0, 1):      # low and high four bits of a byte
            pool[..., byte[:, e::2]] |= (c[..., e::2] << np.uint8(4 * e)).astype(np.uint8)
        half[..., step[:, ::32]] = blocks(st)
        half[..., step[:, ::32] + 16 * ng] = blocks(ze)
    return pool


def attend(q, K, V, visible, scale):
    """One kv head: q [rows, dh], K, V [keys, dh], visible [rows, keys]; rows that see nothing give 0.
    Returns (o, probabilities)."""
    s = np.asarray(q, np.float64) @ np.asarray(K, np.float64).T * scale
    s = np.where(visible, s, -np.inf)
    m = s.max(axis=1, keepdims=True, initial=-np.inf)
    with np.errstate(invalid="ignore"):
        p = np.where(visible, np.exp(s - np.where(np.isfinite(m), m, 0.0)), 0.0)
    l = p.sum(axis=1, keepdims=True)
    p = np.divide(p, l, out=np.zeros_like(p), where=l > 0)
    return p @ np.where(visible.any(axis=0)[:, None], V, 0.0), p
