"""Reference (numpy) of the key/value cache held in 4 bits: quantisation, the bytes of
the format, and the values held. TEST INFRASTRUCTURE, written from the definition in
``include/attn.h``; it shares no code with the CUDA package.

Every step is exact or a single stated rounding: x and the values are bf16 numbers
held in fp64, the step's range and its fifteenth are the definition's fp32 roundings,
and quotients are formed in fp64, where x / s is off by 2^-53 while a quotient that is
not exactly halfway between two whole numbers is 1/512 or more away from halfway.
"""

from __future__ import annotations

import numpy as np

GROUP = 64
BLOCK = 64
BAD_WORD = 0x7FC0


def _f64(x):
    try:
        import torch
        if isinstance(x, torch.Tensor):
            return x.detach().to("cpu", torch.float64).numpy()
    except ImportError:  # pragma: no cover
        pass
    return np.asarray(x, dtype=np.float64)


def quantise(x):
    """x [..., d] -> (codes u, steps s, zeros u0, bad): codes [..., d]; the others [..., d/64]."""
    x = _f64(x)
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    bad = ~(np.abs(g) < 2.0 ** 127).all(-1)
    g = np.where(bad[..., None], 0.0, g)
    lo = np.minimum(g.min(-1), 0.0)
    hi = np.maximum(g.max(-1), 0.0)
    r = (hi.astype(np.float32) - lo.astype(np.float32)).astype(np.float32)
    t = (r / np.float32(15)).astype(np.float64)
    frac, ex = np.frexp(t)                                # t = frac 2^ex, frac in [0.5, 1)
    ex = np.maximum(ex, -125)                             # the fp32 subnormals share one exponent
    s = np.ceil(np.ldexp(t, 4 - ex)) * np.ldexp(1.0, ex - 4)
    one = np.where(s == 0, 1.0, s)
    u0 = np.rint(-lo / one)
    u = np.clip(np.rint(g / one[..., None]) + u0[..., None], 0, 15)
    u = np.where(bad[..., None], 0, u)
    return u.reshape(x.shape).astype(np.int64), s, np.where(bad, 0, u0).astype(np.int64), bad


def held(x):
    """The values that x [..., d] is held as (NaN in a bad group)."""
    u, s, u0, bad = quantise(x)
    s = np.where(bad, np.nan, s)
    g = u.reshape(*u.shape[:-1], -1, GROUP) - u0[..., None]
    return (g * s[..., None]).reshape(u.shape)


def coded(x):
    """s u of every channel: the held value without its zero taken out (>= 0)."""
    u, s, u0, bad = quantise(x)
    return u * np.repeat(s, GROUP, -1)


def words(s, u0, bad):
    """The groups' 16-bit words."""
    bits = s.astype(np.float32).view(np.uint32) >> 16
    return np.where(bad, BAD_WORD, bits | u0.astype(np.uint32)).astype(np.uint16)


def code_byte(k, c, d, is_k):
    """(byte inside the K or V codes, is it the high nibble) of channel c of slot k."""
    ng, q, r = d // 64, c // 64, c % 64
    if is_k:
        row = k ^ ((k >> 2 & 1) * (128 // d))
        return row * (d // 2) + ((r // 16) * ng + q) * 8 + (r % 16) // 2, r % 2 == 1
    unit = r // 8
    if d == 128 and k >> 1 & 1:
        unit ^= 4
    return k * (d // 2) + (unit * ng + q) * 4 + (r % 8) // 2, r % 2 == 1


_tables = {}


def _table(d, is_k):
    """code_byte for all slots and channels: bytes [64, d], shifts [64, d]."""
    if (d, is_k) not in _tables:
        at = np.empty((BLOCK, d), np.int64)
        sh = np.empty((BLOCK, d), np.int64)
        for k in range(BLOCK):
            for c in range(d):
                at[k, c], high = code_byte(k, c, d, is_k)
                sh[k, c] = 4 if high else 0
        _tables[d, is_k] = at, sh
    return _tables[d, is_k]


def write(cache, K, V, starts=None, counts=None, m=None):
    """A copy of the cache bytes [B, H, blocks, 34 (d_k + d_v)] (uint8) with the rows
    K, V [B, H, n, d] put in."""
    cache = np.array(cache, dtype=np.uint8)
    K, V = _f64(K), _f64(V)
    B, H, n, dk = K.shape
    dv = V.shape[3]
    m = cache.shape[2] * BLOCK if m is None else m
    for b in range(B):
        first = 0 if starts is None else int(starts[b])
        for i in range(n if counts is None else min(n, int(counts[b]))):
            slot = first + i
            if not 0 <= slot < m:
                continue
            blk, k = divmod(slot, BLOCK)
            base = 0
            for x, d, is_k in ((K, dk, True), (V, dv, False)):
                u, s, u0, bad = quantise(x[b, :, i])
                at, sh = _table(d, is_k)
                for c in range(d):
                    byte = base + at[k, c]
                    keep = 0xF0 if sh[k, c] == 0 else 0x0F
                    cache[b, :, blk, byte] = (cache[b, :, blk, byte] & keep) | (u[:, c] << sh[k, c]).astype(np.uint8)
                w = words(s, u0, bad)
                for q in range(d // 64):
                    byte = base + 32 * d + 2 * (k * (d // 64) + q)
                    cache[b, :, blk, byte] = w[:, q] & 255
                    cache[b, :, blk, byte + 1] = w[:, q] >> 8
                base += 34 * d
    return cache


def read(cache, dk, m=None, key_lengths=None):
    """The values held: fp64 K [B, H, m, d_k], V [B, H, m, d_v], 0 at or past the lengths."""
    cache = np.asarray(cache)
    B, H, blocks, width = cache.shape
    dv = width // 34 - dk
    m = blocks * BLOCK if m is None else m
    out, base = [], 0
    for d, is_k in ((dk, True), (dv, False)):
        at, sh = _table(d, is_k)
        u = (cache[..., base + at] >> sh) & 15
        at = base + 32 * d + 2 * (np.arange(BLOCK)[:, None] * (d // 64) + np.arange(d // 64))
        w = cache[..., at].astype(np.uint32) | cache[..., at + 1].astype(np.uint32) << 8
        with np.errstate(invalid="ignore"):               # unwritten words may be NaN
            s = ((w & 0xFFF0) << 16).view(np.float32).astype(np.float64)
            v = (u.astype(np.float64) - np.repeat(w & 15, 64, -1)) * np.repeat(s, 64, -1)
        v = v.reshape(B, H, blocks * BLOCK, d)[:, :, :m].copy()
        if key_lengths is not None:
            for b in range(B):
                v[b, :, max(0, int(key_lengths[b])):] = 0
        out.append(v)
        base += 34 * d
    return tuple(out)
