"""Paged 4-bit cache, page tables and packed prompts, stated plainly (loops over requests and
nibbles, fp64 attention). The definitions are those of include/cacheblend.h; the pages give the
setting only ("rag的kvcache问题" §独立编码: chunk caches are computed alone and kept; §阶段 2 (Decode)).
"""

from __future__ import annotations

import numpy as np

from .attention import causal_gqa_attention

GROUP = 32


def _to_bf16(x):
    """float64 -> nearest bf16 (ties to even) as float64; finite or infinite input."""
    x = np.asarray(x, dtype=np.float64)
    m, e = np.frexp(x)  # x = m 2^e, 0.5 <= |m| < 1
    step = np.ldexp(1.0, np.maximum(e - 8, -133))  # last place: 8 significant bits, subnormals of 2^-133
    with np.errstate(invalid="ignore"):
        y = np.where(np.isfinite(x) & (x != 0), np.round(x / step) * step, x)
    return np.where(np.abs(y) > 3.3895313892515355e38, np.sign(y) * np.inf, y)


def quantise(x):
    """x [..., D] -> codes int [..., D] in -7 .. 7 and scales float64 [..., D/32] (bf16 values)."""
    x = np.asarray(x, dtype=np.float64)
    codes = np.zeros(x.shape, dtype=np.int64)
    scales = np.zeros(x.shape[:-1] + (x.shape[-1] // GROUP,))
    for g in range(x.shape[-1] // GROUP):
        part = x[..., g * GROUP:(g + 1) * GROUP]
        fine = np.isfinite(part).all(-1)
        # (by way of fp32, which changes nothing: no quotient by 7 lies that near to a midpoint of two bf16s)
        scale = np.where(fine, _to_bf16((np.abs(np.where(fine[..., None], part, 0)).max(-1) / 7)
                                        .astype(np.float32).astype(np.float64)), np.nan)
        ok = fine & (scale > 0)
        step = np.where(ok, scale, 1.0)[..., None]
        codes[..., g * GROUP:(g + 1) * GROUP] = np.where(
            ok[..., None], np.clip(np.round(np.where(ok[..., None], part, 0) / step), -7, 7), 0)
        scales[..., g] = scale
    return codes, scales


def dequantise(codes, scales):
    return codes * np.repeat(scales, GROUP, axis=-1)


def page_bytes(page_size, d):
    return page_size // 16 * 18 * d


def _places(d, dim, tok):
    """Where a record holds dim `dim` of its token `tok`: (K byte, shift), (V byte, shift), and the
    scales' K byte offset (V's follows d / 32 bf16 later)."""
    ng, g, e = d // GROUP, dim // GROUP, dim % GROUP
    word = (tok * 4 + e // 8) * ng + g
    bit = 4 * (e % 8 // 2) + 16 * (e % 2)
    k = (4 * word + bit // 8, bit % 8)
    word = ((tok // 8 * 8 + e // 4) * 4 + tok % 8 // 2) * ng + g
    bit = 4 * (e % 4) + 16 * (tok % 2)
    v = (8 * d + 4 * word + bit // 8, bit % 8)
    return k, v, 16 * d + (tok * 2 * ng + g) * 2


def store(cache, page_size, slots, k, v):
    """Quantise rows k, v [n, hkv, D] into cache (uint8 [n_pages, hkv, page_bytes]) in place."""
    n, hkv, d = np.asarray(k).shape
    rec = cache.reshape(cache.shape[0], hkv, page_size // 16, 18 * d)
    (kc, ks), (vc, vs) = quantise(k), quantise(v)
    for i, slot in enumerate(np.asarray(slots).tolist()):
        if slot < 0 or slot >= cache.shape[0] * page_size:
            continue
        at = rec[slot // page_size, :, slot % page_size // 16]  # [hkv, 18 D]
        for dim in range(d):
            (kb, ksh), (vb, vsh), sc = _places(d, dim, slot % 16)
            for byte, shift, code in ((kb, ksh, kc), (vb, vsh, vc)):
                at[:, byte] = at[:, byte] & (0xF0 >> shift) | ((code[i, :, dim] + 8) << shift).astype(np.uint8)
            if dim % GROUP == 0:
                for off, scale in ((sc, ks), (sc + d // GROUP * 2, vs)):
                    s = scale[i, :, dim // GROUP].astype(np.float32).view(np.uint32) >> 16
                    at[:, off] = s & 255
                    at[:, off + 1] = s >> 8


def load(cache, page_size, slots, d):
    """K, V [n, hkv, D] (float64, unrounded scale * code) at valid slots."""
    slots = np.asarray(slots, dtype=np.int64)
    hkv = cache.shape[1]
    rec = cache.reshape(cache.shape[0], hkv, page_size // 16, 18 * d)
    at = rec[slots // page_size, :, slots % page_size // 16].astype(np.uint32)  # [n, hkv, 18 D]
    k = np.zeros((slots.size, hkv, d))
    v = np.zeros((slots.size, hkv, d))
    for tok in range(16):
        rows = np.nonzero(slots % 16 == tok)[0]
        if rows.size == 0:
            continue
        a = at[rows]
        for dim in range(d):
            (kb, ksh), (vb, vsh), sc = _places(d, dim, tok)
            for out, byte, shift, off in ((k, kb, ksh, sc), (v, vb, vsh, sc + d // GROUP * 2)):
                scale = ((a[:, :, off] | a[:, :, off + 1] << 8) << 16).astype(np.uint32).view(np.float32)
                out[rows, :, dim] = ((a[:, :, byte] >> shift & 15).astype(np.float64) - 8) * scale
    return k, v


def page_tables(ctx, new, page_size, free, table, n_rows, free_from=0):
    """One step's page tables: (table, cu, kv_lens, positions, slots, free_to), lengths valid."""
    table = np.array(table)
    width = table.shape[1]
    cu, kv, pos, slots = [0], [], np.zeros(n_rows, np.int64), np.full(n_rows, -1, np.int64)
    at = free_from
    for s, (c, w) in enumerate(zip(ctx, new)):
        for col in range(-(-c // page_size), -(-(c + w) // page_size)):
            if col < width:
                table[s, col] = free[at] if at < len(free) else -1
                at += 1
        for i in range(w):
            row = cu[-1] + i
            if row < n_rows:
                pos[row] = c + i
                page = table[s, (c + i) // page_size] if (c + i) // page_size < width else -1
                slots[row] = page * page_size + (c + i) % page_size if page >= 0 else -1
        cu.append(cu[-1] + w)
        kv.append(min(c + w, width * page_size))
    return table, np.minimum(cu, n_rows), np.array(kv), pos, slots, min(at, max(len(free), free_from))


def packed_attention(q, k, v, cu, scale=None):
    """Causal attention of each sequence's rows; (out, sum p |v|), NaN in rows of no sequence."""
    out = np.full(np.asarray(q).shape, np.nan)
    vs = out.copy()
    for a, b in zip(cu[:-1], cu[1:]):
        if b > a:
            out[a:b], vs[a:b] = causal_gqa_attention(q[a:b], np.arange(b - a), k[a:b], v[a:b], scale=scale,
                                                     return_vscale=True)
    return out, vs
