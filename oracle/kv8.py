"""Oracle of the 8-bit KV cache: codes, quantisation and tree attention over a
prefix held in 8 bits, in plain fp64 numpy.

TEST INFRASTRUCTURE ONLY, as the rest of this package: nothing here is shared
with the CUDA path.
"""
from __future__ import annotations

import numpy as np

from . import bf16_to_f64

PAGE = 16
QMAX = {"e4m3": 448.0, "int8": 127.0}


def decode(codes: np.ndarray, fmt: str) -> np.ndarray:
    """uint8 codes to the numbers they stand for."""
    c = np.asarray(codes, dtype=np.uint8).astype(np.int64)
    if fmt == "int8":
        return np.where(c >= 128, c - 256, c).astype(np.float64)
    e, m = (c >> 3) & 15, (c & 7).astype(np.float64)
    mag = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7.0))
    mag = np.where((c & 127) == 127, np.nan, mag)
    return np.where(c >= 128, -mag, mag)


def encode(y: np.ndarray, fmt: str) -> np.ndarray:
    """Numbers (already divided by their scale) to the nearest codes, ties to
    even; found by search over all codes of the format."""
    y = np.asarray(y, dtype=np.float64)
    if fmt == "int8":
        return np.rint(y).astype(np.int64).astype(np.uint8)
    vals = decode(np.arange(127), fmt)                     # 0 .. 448, ascending with the code
    mag = np.abs(y)
    hi = np.clip(np.searchsorted(vals, mag), 1, 126)
    lo = hi - 1
    dl, dh = mag - vals[lo], vals[hi] - mag
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return (code + 128 * np.signbit(y)).astype(np.uint8)


def quantize_block(x: np.ndarray, fmt: str):
    """Codes and fp32 scale of one block of bf16 values (as fp64)."""
    if not np.isfinite(x).all():
        return np.zeros(x.shape, np.uint8), np.float32(np.nan)
    amax = np.abs(x).max()
    y = x * QMAX[fmt] / (amax if amax > 0 else 1.0)
    return encode(y, fmt), np.float32(np.float32(amax) / np.float32(QMAX[fmt]))


def quantize(k_cache, page_table, page_table8, from_len, to_len, codes, scales, fmt):
    """In place on ``codes`` [pages][Hkv][16][D] and ``scales``: the full pages
    of slots [from_len, to_len) of every request."""
    x = bf16_to_f64(k_cache)
    for b, (f, t) in enumerate(zip(from_len, to_len)):
        for lp in range(int(f) // PAGE, int(t) // PAGE):
            for g in range(x.shape[2]):
                c, s = quantize_block(x[page_table[b, lp], :, g], fmt)
                codes[page_table8[b, lp], g], scales[page_table8[b, lp], g] = c, s


def tree_attention(case, fmt):
    """fp64 outputs [T][Hq][D], the average magnitude sum p |v| / sum p of each,
    each row's largest scale * sum_d |q_d k_d|, and for each output the sum of
    the 8-bit V codes' magnitudes times the largest V scale, of a case with keys
    Hq, Hkv, D, prefix_len, node_offsets, parent, page_table, k_cache, v_cache
    (bf16 bits), page_table8, k8, v8 (codes), k_scale, v_scale, q, scale."""
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    G, offs = Hq // Hkv, case["node_offsets"]
    T = int(offs[-1])
    out, mag, top = np.zeros((T, Hq, D)), np.zeros((T, Hq, D)), np.zeros((T, Hq))
    codes = np.zeros((T, Hq, D))
    q = bf16_to_f64(case["q"])
    kc, vc = bf16_to_f64(case["k_cache"]), bf16_to_f64(case["v_cache"])
    for b in range(len(offs) - 1):
        s0, n, P = int(offs[b]), int(offs[b + 1] - offs[b]), int(case["prefix_len"][b])
        full = P // PAGE
        pg8 = case["page_table8"][b, :full]
        slots = np.arange(full * PAGE, P + n)
        pg = case["page_table"][b][slots // PAGE]
        sees = np.zeros((n, P + n), dtype=bool)
        sees[:, :P] = True
        for i in range(n):
            j = i
            while j >= 0:
                sees[i, P + j] = True
                j = int(case["parent"][s0 + j])
        for g in range(Hkv):
            K, V = [np.concatenate([(decode(case[c][pg8, g], fmt) * case[s][pg8, g].astype(np.float64)[:, None, None])
                                    .reshape(-1, D), x[pg, slots % PAGE, g]])
                    for c, s, x in (("k8", "k_scale", kc), ("v8", "v_scale", vc))]
            codes[s0:s0 + n, g * G:(g + 1) * G] = np.abs(decode(case["v8"][pg8, g], fmt)).sum(axis=(0, 1)) * \
                case["v_scale"][pg8, g].max(initial=0)
            for h in range(g * G, (g + 1) * G):
                qh = q[s0:s0 + n, h]
                with np.errstate(invalid="ignore"):
                    s = np.where(sees, case["scale"] * (qh @ K.T), -np.inf)
                    p = np.exp(s - s.max(axis=1, keepdims=True))
                    p /= p.sum(axis=1, keepdims=True)
                    # a key that a node does not see has weight zero whatever its value is
                    odd = ~np.isfinite(V)
                    V0 = np.where(odd, 0, V)
                    out[s0:s0 + n, h], mag[s0:s0 + n, h] = p @ V0, p @ np.abs(V0)
                    out[s0:s0 + n, h][(sees.astype(np.int64) @ odd) > 0] = np.nan
                    top[s0:s0 + n, h] = case["scale"] * np.where(sees, np.abs(qh) @ np.abs(K).T, 0).max(axis=1)
    return out, mag, top, codes


def held_terms(case, fmt, tiles):
    """For each output, what the 8-bit keys' weights and values may be off by
    beyond roundings relative to themselves, as [T][Hq][D].  With w_j the
    weight of key j relative to the row's largest and top the largest V scale
    of the eight pages of a 128-slot tile:
      streaming form   sum_j min(w_j, 2^-25) |v_j| / sum_j w_j
      tcgen05 form     sum_j (min(w_j, 2^-31) |v_j| + w_j 2^-28 top_j) / sum_j w_j"""
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    G, offs = Hq // Hkv, case["node_offsets"]
    out = np.zeros((int(offs[-1]), Hq, D))
    q = bf16_to_f64(case["q"])
    kc = bf16_to_f64(case["k_cache"])
    for b in range(len(offs) - 1):
        s0, n, P = int(offs[b]), int(offs[b + 1] - offs[b]), int(case["prefix_len"][b])
        full = P // PAGE
        pg8 = case["page_table8"][b, :full]
        slots = np.arange(full * PAGE, P + n)
        pg = case["page_table"][b][slots // PAGE]
        sees = np.zeros((n, P + n), dtype=bool)
        sees[:, :P] = True
        for i in range(n):
            j = i
            while j >= 0:
                sees[i, P + j] = True
                j = int(case["parent"][s0 + j])
        for g in range(Hkv):
            ks, vs = (case[x][pg8, g].astype(np.float64) for x in ("k_scale", "v_scale"))
            K = np.concatenate([(decode(case["k8"][pg8, g], fmt) * ks[:, None, None]).reshape(-1, D), kc[pg, slots % PAGE, g]])
            V = np.abs(decode(case["v8"][pg8, g], fmt) * vs[:, None, None]).reshape(-1, D)
            top = np.repeat([vs[i // 8 * 8:i // 8 * 8 + 8].max() for i in range(full)], PAGE)
            for h in range(g * G, (g + 1) * G):
                s = np.where(sees, case["scale"] * (q[s0:s0 + n, h] @ K.T), -np.inf)
                w = np.exp(s - s.max(axis=1, keepdims=True))
                total, w = w.sum(axis=1, keepdims=True), w[:, :full * PAGE]
                off = np.minimum(w, 2.0 ** (-31 if tiles else -25)) @ V
                if tiles and full:
                    off = off + 2.0 ** -28 * (w @ top)[:, None]
                out[s0:s0 + n, h] = off / total
    return out
