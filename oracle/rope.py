"""CPU oracle of the rotary positions, the norms of query and key heads and the
rotated append (test infrastructure only; include/skinny.h: rope_frequencies,
qk_norm_rope, kv4_append_rope).

Everything runs in float64 on the inputs' exact values; angles come from whole
numbers modulo 2^64.

Parity status: pinned (tests/test_oracle_rope.py).
"""
from __future__ import annotations

import math

import numpy as np

from .oracle import e4m3_to_f64
from .quant import _E2M1_POS, _E4M3_POS, _round_to_table
from . import kv4


def frequencies(rot, base, scaling="plain", factor=1.0, original=0.0, low=1.0, high=32.0):
    """Radians per position of the rot / 2 pairs, float64."""
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2))
    out = []
    at = lambda turns: rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))      # noqa: E731
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        keep = 1.0
        if scaling == "linear":
            keep = 0.0
        elif scaling == "turns":
            keep = (original * f / (2 * math.pi) - low) / (high - low)
        elif scaling == "index":
            first, last = max(0, math.floor(at(high))), min(rot - 1, math.ceil(at(low)))
            keep = 1 - (i - first) / max(1e-3, last - first)
        keep = min(1.0, max(0.0, keep))
        out.append(f if scaling in ("plain", "base") else f * (keep + (1 - keep) / factor))
    return np.array(out)


def turned(x, positions, freqs, weight, eps, amplitude, interleaved):
    """x f16 [T][H][D], freqs int64 [R/2] (units of 2^-64 turns) -> (y float64 [T][H][D], size): size bounds what a
    component is made of, the sum of its two terms' magnitudes without cosine and sine."""
    y = np.asarray(x, np.float16).astype(np.float64)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float32).astype(np.float64)
    R = 2 * len(freqs)
    size = np.abs(y)
    if R == 0:
        return y, size
    with np.errstate(over="ignore"):
        low = np.asarray(positions, np.int64).astype(np.uint64)[:, None] * np.asarray(freqs, np.int64).astype(np.uint64)
    angle = low.view(np.int64).astype(np.float64) * 2.0 ** -64 * (2 * math.pi)
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    a_at = np.arange(0, R, 2) if interleaved else np.arange(R // 2)
    b_at = a_at + 1 if interleaved else a_at + R // 2
    a, b = y[..., a_at], y[..., b_at]
    out = y.copy()
    out[..., a_at] = (a * c - b * s) * amplitude
    out[..., b_at] = (b * c + a * s) * amplitude
    both = (np.abs(a) + np.abs(b)) * max(1.0, abs(amplitude))
    size[..., a_at] = both
    size[..., b_at] = both
    return out, size


def encode(y, G):
    """float64 [..., D] -> (E2M1 codes 0..15, E4M3 scale codes [..., D/16]) from the exact quotients."""
    G = float(np.float32(G))
    blocks = y.reshape(y.shape[:-1] + (y.shape[-1] // 16, 16))
    top = np.abs(blocks).max(-1)
    sc = _round_to_table(top / (6.0 * G), _E4M3_POS, 0).reshape(top.shape)
    unit = (e4m3_to_f64(sc).reshape(sc.shape) * G)[..., None]
    q = np.where(unit == 0, np.copysign(0.0, blocks), blocks / np.where(unit == 0, 1.0, unit))
    return _round_to_table(q, _E2M1_POS, 8).astype(np.uint8).reshape(y.shape), sc.astype(np.uint8)


def write(cache, slot, head, key, v, kG, vG):
    """Write a turned key (float64 [D]) and an FP16 value [D] of one head to a slot of `cache` (changed in place)."""
    page, D = cache.shape[2] * 16, cache.shape[3] // 18
    rec = cache[slot // page, head, slot % page // 16]
    at = kv4._where(D, slot % 16)
    for part, (nib, sc) in enumerate((encode(key, kG), kv4.encode(v, vG))):
        rec[at[2 * part]] = nib[0::2] | (nib[1::2] << 4)
        rec[at[2 * part + 1]] = sc


def chunks(q, cache, table, lens, starts, kG, vG, scale, window=0, sinks=0):
    """Attention of each sequence's last rows (q f16 [rows][Hq][D], starts [B + 1]): dict as kv4.attention's, rows of
    no sequence NaN."""
    rows, Hq, D = q.shape
    H = cache.shape[1]
    G = Hq // H
    got = {"out": np.full((rows, Hq, D), np.nan), "absum": np.zeros((rows, Hq, D)), "lse": np.full((rows, Hq), np.nan),
           "zmax": np.zeros((rows, Hq))}
    q = np.asarray(q, np.float16).astype(np.float64)
    for b in range(len(lens)):
        n, lo, hi = int(lens[b]), int(starts[b]), int(starts[b + 1])
        for h in range(H):
            k, v = kv4.sequence(cache, table[b], n, h, kG, vG)
            j = np.arange(n)
            for r in range(lo, hi):
                at = n - (hi - lo) + (r - lo)
                seen = j <= at
                if window:
                    seen &= (j > at - window) | (j < sinks)
                x = slice(h * G, (h + 1) * G)
                if not seen.any():
                    got["out"][r, x], got["lse"][r, x] = 0.0, -np.inf
                    continue
                z = float(np.float32(scale)) * (q[r, x] @ k[seen].T)
                top = z.max(-1, keepdims=True)
                p = np.exp(z - top)
                got["lse"][r, x] = top[:, 0] + np.log(p.sum(-1))
                p /= p.sum(-1, keepdims=True)
                got["out"][r, x] = p @ v[seen]
                got["absum"][r, x] = p @ np.abs(v[seen])
                got["zmax"][r, x] = float(scale) * (np.abs(q[r, x]) @ np.abs(k[seen]).T).max(-1)
    return got
