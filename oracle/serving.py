"""The serving operators in double: causal attention over packed prompts, the
4-bit key-value row and the decode attention over a cache of such rows, and the
log-probabilities of given tokens.

TEST INFRASTRUCTURE ONLY (see the package docstring): shares no code with the
CUDA library.

The 4-bit row (80 bytes) holds one slot's 128 values in four groups of 32
consecutive dimensions; code q (0..15) stands for s * (q - 8) + z with a bf16
scale and zero per group.  Quantiser, every decision in fp32: s = bf16((max -
min) / 15), 0 below 2^-126; z = bf16(min + 8 s); q = clamp(rint((x - z) / s) +
8, 0, 15), 8 where s is 0; a group with a value that is not finite has s = z =
NaN and code 8.  64 bytes of codes, nibble n (bits 4 (n % 2) of byte n // 2):
dimension 32 g + w t + i where n = (4 t + g) w + i, with w = 8 for keys and 4
for values; then (s, z) per group.
"""
from __future__ import annotations

import numpy as np

D, GROUP, NG, ROW = 128, 32, 4, 80


def _bf16_bits(v):
    u = np.asarray(v, np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(v), np.uint16(0x7FC0), r)


def _bf16_f32(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32)


def _nibble_of_dim(keys: bool):
    w = 8 if keys else 4
    d = np.arange(D)
    g, t, i = d // GROUP, d % GROUP // w, d % w
    return (4 * t + g) * w + i


def quantize_rows(x, keys: bool):
    """fp32 [..., 128] -> cached rows uint8 [..., 80]."""
    x = np.asarray(x, np.float32)
    g = x.reshape(*x.shape[:-1], NG, GROUP)
    with np.errstate(all="ignore"):
        lo, hi = g.min(-1), g.max(-1)
        s32 = (hi - lo) / np.float32(15)
        bad = ~(s32 <= np.finfo(np.float32).max)
        s = _bf16_f32(_bf16_bits(s32))
        s = np.where(s < np.float32(2.0 ** -126), np.float32(0), s)
        z = _bf16_f32(_bf16_bits(lo + np.float32(8) * s))
        q = np.rint((g - z[..., None]) / s[..., None]) + np.float32(8)
    q = np.where((s == 0)[..., None] | bad[..., None], 8, np.clip(q, 0, 15))
    q = np.nan_to_num(q, nan=8).astype(np.uint8).reshape(x.shape)
    nib = np.zeros(x.shape, np.uint8)
    nib[..., _nibble_of_dim(keys)] = q
    codes = nib[..., 0::2] | (nib[..., 1::2] << 4)
    sb = np.where(bad, np.uint16(0x7FC0), _bf16_bits(s))
    zb = np.where(bad, np.uint16(0x7FC0), _bf16_bits(z))
    sz = np.stack([sb, zb], -1).astype("<u2")
    sz = np.ascontiguousarray(sz).view(np.uint8).reshape(*x.shape[:-1], 16)
    return np.concatenate([codes, sz], -1)


def row_values(rows, keys: bool):
    """(codes - 8, s, z) of cached rows, per dimension, as fp32."""
    rows = np.asarray(rows, np.uint8)
    nib = np.stack([rows[..., :64] & 15, rows[..., :64] >> 4], -1).reshape(*rows.shape[:-1], D)
    c = nib[..., _nibble_of_dim(keys)].astype(np.float32) - 8
    sz = np.ascontiguousarray(rows[..., 64:]).view("<u2").reshape(*rows.shape[:-1], NG, 2)
    s = np.repeat(_bf16_f32(sz[..., 0]), GROUP, -1)
    z = np.repeat(_bf16_f32(sz[..., 1]), GROUP, -1)
    return c, s, z


def dequantize_rows(rows, keys: bool):
    """The fp32 values that cached rows stand for (s (q - 8) is exact in fp32)."""
    c, s, z = row_values(rows, keys)
    with np.errstate(all="ignore"):
        return (s * c + z).astype(np.float32)


def _softmax_rows(s, v):
    """out, log-sum-exp and sum p |v| of score rows [n, m] over values [m, d]."""
    with np.errstate(all="ignore"):
        m = s.max(-1, keepdims=True)
        e = np.exp(s - m)
        l = e.sum(-1, keepdims=True)
        p = e / l
        return p @ v, (m + np.log(l))[..., 0], p @ np.abs(v)


def decode_attention_q4(q, k_new, v_new, k_cache, v_cache, pos):
    """q [B, nh * 128], new rows [B, nkv * 128] fp32, caches uint8 [B, nkv, S,
    80].  Returns out and the absolute sum of its parts (sum_j p_j (|s_j (q_j -
    8)| + |z_j|)) [B, nh * 128], the largest sum_d |q_d| (|s (code - 8)| + |z|) /
    sqrt(d) over the slots per row and head [B, nh], and the updated caches; rows with a position outside 0 .. S - 1 are left out (NaN)."""
    B, nkv, S, _ = k_cache.shape
    nh = q.shape[1] // D
    kc, vc = k_cache.copy(), v_cache.copy()
    out = np.full((B, nh * D), np.nan)
    mag = np.full((B, nh * D), np.nan)
    top = np.full((B, nh), np.nan)
    for b in range(B):
        p = int(pos[b])
        if p < 0 or p >= S:
            continue
        kc[b, :, p] = quantize_rows(k_new[b].reshape(nkv, D), True)
        vc[b, :, p] = quantize_rows(v_new[b].reshape(nkv, D), False)
        for h in range(nh):
            g = h // (nh // nkv)
            c, s, z = (x.astype(np.float64) for x in row_values(kc[b, g, :p + 1], True))
            K, Ka = s * c + z, np.abs(s * c) + np.abs(z)
            c, s, z = (x.astype(np.float64) for x in row_values(vc[b, g, :p + 1], False))
            V, Va = s * c + z, np.abs(s * c) + np.abs(z)
            qh = np.asarray(q[b, h * D:(h + 1) * D], np.float64)
            o, _, a = _softmax_rows((K @ qh)[None] / np.sqrt(D), np.concatenate([V, Va], axis=1))
            out[b, h * D:(h + 1) * D], mag[b, h * D:(h + 1) * D] = o[0, :D], a[0, D:]
            with np.errstate(all="ignore"):
                top[b, h] = (Ka @ np.abs(qh)).max() / np.sqrt(D)
    return out, mag, top, kc, vc


def prompt_attention(q, k, v, bounds):
    """q [T, nh, 128], k and v [T, nkv, 128] (double), bounds [n + 1].  Returns
    out, its absolute sum [T, nh, 128] and the log-sum-exp [T, nh]; NaN outside
    the sequences.  Only pairs that attend to one another are touched."""
    T, nh, _ = q.shape
    grp = nh // k.shape[1]
    out = np.full((T, nh, D), np.nan)
    mag = np.full((T, nh, D), np.nan)
    lse = np.full((T, nh), np.nan)
    for a, b in zip(bounds[:-1], bounds[1:]):
        for h in range(nh):
            if b <= a:
                continue
            K, V = k[a:b, h // grp], v[a:b, h // grp]
            if np.isfinite(K).all() and np.isfinite(V).all():
                s = q[a:b, h] @ K.T / np.sqrt(D)
                s[np.triu_indices(b - a, 1)] = -np.inf
                out[a:b, h], lse[a:b, h], mag[a:b, h] = _softmax_rows(s, V)
                continue
            for t in range(b - a):
                with np.errstate(all="ignore"):
                    s = (K[:t + 1] @ q[a + t, h] / np.sqrt(D))[None]
                o, e, m = _softmax_rows(s, V[:t + 1])
                out[a + t, h], lse[a + t, h], mag[a + t, h] = o[0], e[0], m[0]
    return out, mag, lse


def token_logprobs(x, k: int):
    """Rows of logits (double) -> log-probabilities [rows, V], entropy [rows],
    and the k largest logits' indices (falling, ties by the lower index; -1
    where only NaN is left)."""
    x = np.asarray(x, np.float64)
    with np.errstate(all="ignore"):
        m = x.max(-1, keepdims=True)
        lz = np.log(np.exp(x - m).sum(-1, keepdims=True))
        lp = x - m - lz
        p = np.exp(lp)
        ent = -np.where(p == 0, 0.0, p * np.where(p == 0, 0.0, lp)).sum(-1)
    ent = np.where(np.isnan(lp).any(-1), np.nan, ent)
    lp = np.where(np.isnan(ent)[:, None], np.nan, lp)
    order = np.argsort(np.where(np.isnan(x), np.inf, -x + 0.0), axis=-1, kind="stable")[:, :k]
    gone = np.isnan(np.take_along_axis(x, order, -1))
    return lp, ent, np.where(gone, -1, order).astype(np.int32)
