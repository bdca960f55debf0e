"""CPU oracle of the 4-bit key/value cache, its attention and its eviction, and
of the token log probabilities (test infrastructure only).

Only the tests may import this module; the CUDA path shares nothing with it.

What is computed is stated in include/skinny.h (kv4_append, kv4_attention,
kv4_evict, token_logprobs).  The cache's codes follow the rounding rule of
oracle.quant (each step an IEEE binary32 operation, then nearest-even onto the
format's table); everything else runs in float64, one sequence, head and row at
a time.

Parity status: pinned (tests/test_oracle_kv4.py).
"""
from __future__ import annotations

import numpy as np

from .oracle import e2m1_to_f64, e4m3_to_f64
from .quant import e2m1_round, e4m3_round

_F32 = np.float32


def encode(w, G):
    """FP16 [..., D] -> (E2M1 codes 0..15 [..., D], E4M3 scale codes [..., D/16]) under the scale G."""
    w = np.asarray(w, np.float16).astype(_F32)
    blocks = w.reshape(w.shape[:-1] + (w.shape[-1] // 16, 16))
    b = np.abs(blocks).max(-1).astype(_F32)
    sc = e4m3_round(((b / _F32(6.0)).astype(_F32) / _F32(G)).astype(_F32))
    S = e4m3_to_f64(np.arange(256)).astype(_F32)[sc]
    unit = (S * _F32(G)).astype(_F32)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        q = (blocks / unit).astype(_F32)
    nib = np.where(unit == 0, np.where(np.signbit(blocks), 8, 0), e2m1_round(np.where(unit == 0, _F32(0), q)))
    return nib.astype(np.uint8).reshape(w.shape), sc.astype(np.uint8)


def values(nib, sc, G):
    """What codes and scale codes stand for, float64 [..., D]."""
    nib, sc = np.asarray(nib), np.asarray(sc)
    v = e2m1_to_f64(nib).reshape(sc.shape + (16,)) * e4m3_to_f64(sc).reshape(sc.shape + (1,)) * float(_F32(G))
    return v.reshape(nib.shape)


def _where(D, i):
    """Byte offsets inside a record of position i: (key codes [D/2], key scales [D/16], value codes [D/2],
    value scales [D/16])."""
    nb = D // 16
    b, byte = np.repeat(np.arange(nb), 8), np.tile(np.arange(8), nb)
    return (i * (D // 2) + np.arange(D // 2), 8 * D + i * nb + np.arange(nb),
            9 * D + (i // 8) * 4 * D + b * 64 + (i % 8) * 8 + byte, 17 * D + np.arange(nb) * 16 + i)


def write(cache, slot, head, k, v, kG, vG):
    """Write the FP16 key and value [D] of one head to a slot of `cache` (u8 array, changed in place)."""
    page = cache.shape[2] * 16
    D = cache.shape[3] // 18
    rec = cache[slot // page, head, slot % page // 16]
    at = _where(D, slot % 16)
    for part, (x, G) in enumerate(((k, kG), (v, vG))):
        nib, sc = encode(x, G)
        rec[at[2 * part]] = nib[0::2] | (nib[1::2] << 4)
        rec[at[2 * part + 1]] = sc


def read(cache, slot, head, kG, vG):
    """(key, value) float64 [D] that a slot stands for."""
    page = cache.shape[2] * 16
    D = cache.shape[3] // 18
    rec = cache[slot // page, head, slot % page // 16]
    at = _where(D, slot % 16)
    got = []
    for part, G in ((0, kG), (1, vG)):
        c = rec[at[2 * part]]
        got.append(values(np.stack((c & 15, c >> 4), -1).reshape(-1), rec[at[2 * part + 1]], G))
    return got


def sequence(cache, table, n, head, kG, vG):
    """(keys, values) float64 [n][D] of a sequence's first n positions."""
    page = cache.shape[2] * 16
    D = cache.shape[3] // 18
    k, v = np.zeros((n, D)), np.zeros((n, D))
    for j in range(n):
        k[j], v[j] = read(cache, int(table[j // page]) * page + j % page, head, kG, vG)
    return k, v


def attention(q, cache, table, lens, kG, vG, scale, rows):
    """q f16 [B * rows][Hq][D] -> dict with float64 out, lse, weights [B][H][longest] (the sum of p per position),
    and for tolerances: absum = sum_j p_j |v_j| [like out], zmax = the largest scale * sum_d |q_d k_jd| seen [like lse]."""
    B, H = len(lens), cache.shape[1]
    Hq, D = q.shape[1], q.shape[2]
    G = Hq // H
    out, absum = np.zeros((B * rows, Hq, D)), np.zeros((B * rows, Hq, D))
    lse, zmax = np.full((B * rows, Hq), -np.inf), np.zeros((B * rows, Hq))
    weights = np.zeros((B, H, max(1, int(max(lens)))))
    q = np.asarray(q, np.float16).astype(np.float64)
    for b in range(B):
        n = int(lens[b])
        for h in range(H):
            k, v = sequence(cache, table[b], n, h, kG, vG)
            for m in range(rows):
                sees = n - (rows - 1 - m)
                if sees <= 0:
                    continue
                for x in range(h * G, (h + 1) * G):
                    r = b * rows + m
                    z = float(_F32(scale)) * (k[:sees] @ q[r, x])
                    p = np.exp(z - z.max())
                    lse[r, x] = z.max() + np.log(p.sum())
                    p /= p.sum()
                    out[r, x] = p @ v[:sees]
                    absum[r, x] = p @ np.abs(v[:sees])
                    zmax[r, x] = float(scale) * (np.abs(k[:sees]) @ np.abs(q[r, x])).max()
                    weights[b, h, :sees] += p
    return {"out": out, "lse": lse, "weights": weights, "absum": absum, "zmax": zmax}


def keep(acc, n, budget, recent):
    """The positions kept of n by their weights acc [>= n]: ascending."""
    if n <= budget:
        return np.arange(n)
    old = n - recent
    order = np.argsort(-np.asarray(acc[:old], np.float64), kind="stable")[:budget - recent]
    return np.concatenate((np.sort(order), np.arange(old, n)))


def evict(cache, table, lens, acc, dst_table, budget, recent):
    """(cache after, kept [B][H][budget], new_lens [B], acc after [B][H][dst positions])."""
    cache = cache.copy()
    before = cache.copy()
    B, H, recs, rec = cache.shape[0] and len(lens), cache.shape[1], cache.shape[2], cache.shape[3]
    page, D = recs * 16, rec // 18
    kept = np.full((B, H, budget), -1, np.int32)
    out = np.zeros((B, H, dst_table.shape[1] * page), np.float32)
    new = np.minimum(np.maximum(lens, 0), budget).astype(np.int32)
    for b in range(B):
        for h in range(H):
            idx = keep(acc[b, h], int(lens[b]), budget, recent)
            kept[b, h, :len(idx)] = idx
            out[b, h, :len(idx)] = acc[b, h, idx]
            for j, s in enumerate(idx):
                src = before[int(table[b, s // page]), h, s % page // 16]
                dst = cache[int(dst_table[b, j // page]), h, j % page // 16]
                for x, y in zip(_where(D, j % 16), _where(D, s % 16)):
                    dst[x] = src[y]
    return cache, kept, new, out


def logprobs(z, token, temperature, top_n):
    """(logprob, rank, entropy, top ids, top logprobs) of one row of logits, float64."""
    z = np.asarray(z).astype(np.float64)
    t = z / float(_F32(temperature))
    N = z.size
    order = np.lexsort((np.arange(N), -z))[:top_n]
    if np.isnan(z).any() or np.isposinf(z).any():
        lp, ent = np.full(N, np.nan), np.nan
    elif np.isneginf(z).all():
        lp, ent = np.full(N, -np.inf), 0.0
    else:
        d = t - t.max()
        lp = d - np.log(np.exp(d).sum())
        p = np.exp(lp)
        ent = float(-(p[p > 0] * lp[p > 0]).sum())
    ids = np.concatenate((order, np.full(top_n - len(order), -1))).astype(np.int64)
    top = np.concatenate((lp[order], np.full(top_n - len(order), -np.inf)))
    if not 0 <= token < N:
        return 0.0, 0, ent, ids, top
    rank = 1 + int((z > z[token]).sum() + (z[:token] == z[token]).sum())
    return lp[token], rank, ent, ids, top
