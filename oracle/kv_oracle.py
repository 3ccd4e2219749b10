"""Plain oracle of the FP4 key/value cache and of the attention that reads it.

TEST INFRASTRUCTURE ONLY (see the package docstring): the product path never
uses this module.

The cache holds rows of D elements (one token, one KV head) quantized like
weights (``quantize_values``).  Its layout, as the C header documents it, is
stated here element by element; attention is evaluated row by row in float64
from the dequantized rows.
"""

from __future__ import annotations

import numpy as np

from .fp4_oracle import e4m3_value, e8m0_value, e2m1_value, group_size
from .quant_oracle import quantize_values


def kv_offsets(fmt: int, D: int):
    """Byte offsets inside a 32-token tile: (key code pairs [32][D/2], value
    code pairs [32][D/2], key scales [32][D/G], value scales [32][D/G])."""
    G = group_size(fmt)
    kc = np.zeros((32, D // 2), np.int64)
    vc = np.zeros((32, D // 2), np.int64)
    ks = np.zeros((32, D // G), np.int64)
    vs = np.zeros((32, D // G), np.int64)
    for t in range(32):
        u, r, j, i = t // 16, t % 16, t % 16 // 4, t % 4
        for d in range(0, D, 2):
            if D == 64:
                kc[t, d // 2] = (d // 16 * 16 + r) * 16 + u * 8 + d % 16 // 2
                vc[t, d // 2] = (16 * j + d // 4) * 16 + u * 8 + i * 2 + d % 4 // 2
            else:
                kc[t, d // 2] = (d // 128 * 2 + u) * 1024 + (d % 128 // 32 * 16 + r) * 16 + d % 32 // 2
                vc[t, d // 2] = (d // 128 * 2 + u) * 1024 + (16 * j + d % 128 // 8) * 16 + i * 4 + d % 8 // 2
        for g in range(D // G):
            if D == 64:
                ks[t, g] = (g * 16 + r) * 2 + u
            else:
                P, C = 32 // G, D // 128
                ks[t, g] = (g % (4 * P) // P * 16 + r) * (2 * C * P) + g // (4 * P) * 2 * P + u * P + g % P
            vs[t, g] = (g * 4 + j) * 8 + u * 4 + i
    code, scale = 16 * D, 32 * D // G
    return kc, code + vc, 2 * code + ks, 2 * code + scale + vs


def _tiles(slots, H, page_size, tile_bytes):
    """Byte offset of the tile of each (slot, head), and the token in it."""
    page, off = np.divmod(np.asarray(slots, np.int64), page_size)
    base = ((page[:, None] * H + np.arange(H)) * (page_size // 32) + (off // 32)[:, None]) * tile_bytes
    return base, off % 32


def kv_write_reference(data, slots, k, v, page_size, fmt, k_alpha=1.0, v_alpha=1.0):
    """Write rows k, v (FP32 [n][H][D]) into the cache bytes `data` in place;
    slots outside the cache are skipped."""
    n, H, D = k.shape
    G = group_size(fmt)
    tile_bytes = 32 * D + 64 * D // G
    total = data.size // (H * tile_bytes) * 32
    keep = np.flatnonzero((np.asarray(slots) >= 0) & (np.asarray(slots) < total))
    base, t = _tiles(np.asarray(slots)[keep], H, page_size, tile_bytes)
    kc, vc, ks, vs = kv_offsets(fmt, D)
    for x, alpha, codes, scales in ((k, k_alpha, kc, ks), (v, v_alpha, vc, vs)):
        c, s = quantize_values(x[keep].reshape(-1, D).astype(np.float32), fmt, alpha)
        data[base[..., None] + codes[t][:, None, :]] = c.reshape(len(keep), H, D // 2)
        data[base[..., None] + scales[t][:, None, :]] = s.reshape(len(keep), H, D // G)


def kv_read_reference(data, slots, H, D, page_size, fmt, k_alpha=1.0, v_alpha=1.0):
    """Float64 rows (k, v) [n][H][D] at `slots`: alpha * code * scale."""
    G = group_size(fmt)
    base, t = _tiles(slots, H, page_size, 32 * D + 64 * D // G)
    kc, vc, ks, vs = kv_offsets(fmt, D)
    value = e4m3_value if fmt == 0 else e8m0_value
    out = []
    for codes, scales, alpha in ((kc, ks, k_alpha), (vc, vs, v_alpha)):
        b = data[base[..., None] + codes[t][:, None, :]]
        x = np.stack([e2m1_value(b & 15), e2m1_value(b >> 4)], -1).reshape(len(t), H, D)
        s = value(data[base[..., None] + scales[t][:, None, :]])
        out.append(x * np.repeat(s, G, axis=-1) * float(np.float32(alpha)))
    return out


def attention_reference(q, k, v, page_table, seq_lens, q_offsets, page_size, causal=True, window=0, scale=1.0,
                        sinks=None):
    """Float64 attention over rows k, v [slots][H][D] (all slots of the cache).
    q [rows][heads][D].  Page entries outside the cache hold no keys.  Returns
    (out, lse, weight) with weight = sum_j p_j |v_j| / l, the size that errors
    of the probabilities scale with; rows of no sequence are NaN."""
    rows, heads, D = q.shape
    pages, H = k.shape[0] // page_size, k.shape[1]
    group = heads // H
    out = np.full(q.shape, np.nan)
    lse = np.full((rows, heads), np.nan)
    weight = np.full(q.shape, np.nan)
    for b in range(len(seq_lens)):
        n = q_offsets[b + 1] - q_offsets[b]
        L = seq_lens[b]
        pos = np.arange(L)
        page = np.asarray(page_table)[b, pos // page_size] if L else np.zeros(0, np.int64)
        there = (page >= 0) & (page < pages)
        slot = np.where(there, page, 0).astype(np.int64) * page_size + pos % page_size
        for i in range(n):
            at = L - n + i
            see = there & (pos <= at) if causal else there.copy()
            if window:
                see &= pos > at - window
            for h in range(heads):
                kk, vv = k[slot[see], h // group], v[slot[see], h // group]
                s = (kk @ q[q_offsets[b] + i, h]) * scale
                top = max(list(s) + ([float(sinks[h])] if sinks is not None else []), default=-np.inf)
                if top == -np.inf:
                    out[q_offsets[b] + i, h] = weight[q_offsets[b] + i, h] = 0.0
                    lse[q_offsets[b] + i, h] = -np.inf
                    continue
                p = np.exp(s - top)
                total = p.sum() + (np.exp(float(sinks[h]) - top) if sinks is not None else 0.0)
                out[q_offsets[b] + i, h] = p @ vv / total
                weight[q_offsets[b] + i, h] = p @ np.abs(vv) / total
                lse[q_offsets[b] + i, h] = top + np.log(total)
    return out, lse, weight
