"""GPU tests of kv4_chunk_attention and kv4_window_attention where the scores are far larger than a model's, as
test_kv4_scores_gpu.py has them for kv4_attention: neither the output nor the log sum's error depends on what all scores
have in common. FP32 holds every score exactly, so the tolerances are that file's, derived there: a weight's rounding to
FP16 (2^-11), the exponential and the sums (2^-15), half a step of the output; the exponent of a weight is rounded at the
size of a difference of scores, at most 2^-19 for weights that count."""
import numpy as np
import pytest

from gpu_util import Guarded, dev
from oracle import kv4
from test_kv4_scores_gpu import VG, _cache, _tied_keys, sk          # noqa: F401

pytestmark = pytest.mark.gpu

# rows per sequence; the last ones of each head size fill tiles of more than 128 rows
FORMS = [(64, 6, 2, 1), (64, 8, 1, 30), (128, 12, 1, 1), (128, 12, 1, 8), (128, 13, 1, 21), (256, 6, 2, 2), (256, 24, 1, 12)]


def _run(sk, call, cache, tables, lens, q, rows, Hq, D, width, copies=1):       # noqa: F811
    import torch

    table = np.zeros((len(lens), width), np.int32)
    for b, t in enumerate(tables):
        table[b, :len(t)] = t
    B = len(lens) * copies
    out, lse = Guarded((B * rows, Hq, D), torch.float16), Guarded((B * rows, Hq), torch.float32)
    args = (dev(np.tile(q, (copies, 1, 1))), dev(cache), dev(np.tile(table, (copies, 1))), dev(np.tile(np.array(lens, np.int32), copies)))
    if call == "chunk":
        sk.kv4_chunk_attention(*args, dev((np.arange(B + 1) * rows).astype(np.int32)), 1.0, VG, 0.7, out=out.t, lse=lse.t)
    else:
        sk.kv4_window_attention(*args, 1.0, VG, 0.7, 1 << 20, rows=rows, out=out.t, lse=lse.t)
    ref = kv4.attention(q, cache, table, lens, 1.0, VG, 0.7, rows)
    tol = (2.0 ** -11 + 2.0 ** -15) * ref["absum"] + 2.0 ** -11 * np.abs(ref["out"]) + 2.0 ** -25
    empty = np.isneginf(ref["lse"])
    y, z, n = out.host("out"), lse.host("lse"), len(lens) * rows
    for c in range(copies):
        part = slice(c * n, (c + 1) * n)
        assert np.all(np.isfinite(y[part])) and np.all(np.abs(y[part] - ref["out"]) <= tol), c
        assert np.array_equal(np.isneginf(z[part]), empty)
        off = np.abs(z[part][~empty] - ref["lse"][~empty])
        assert np.all(off <= 2.0 ** -16 + 2.0 ** -22 * np.abs(ref["lse"][~empty])), c


def _tied_queries(rows, Hq, D):
    q = np.full((rows, Hq, D), 32768.0, np.float16)
    q[..., 1::3] = 16384.0
    q[..., 2::3] = -32768.0
    return q


@pytest.mark.parametrize("D,Hq,H,rows", FORMS)
@pytest.mark.parametrize("wide", [False, True])
def test_equal_scores_of_any_size_share_the_weight(sk, D, Hq, H, rows, wide):       # noqa: F811
    r = np.random.default_rng(D + Hq)
    lens, page = [200, 0, 37, 1], 32
    keys = [_tied_keys(r, n, D) if n else np.zeros((0, D), np.float16) for n in lens]
    cache, tables = _cache(r, keys, H, D, page)
    _run(sk, "chunk", cache, tables, lens, _tied_queries(len(lens) * rows, Hq, D), rows, Hq, D, 300 if wide else 7)


@pytest.mark.parametrize("D,Hq,H,rows", [(64, 13, 1, 8), (128, 12, 1, 8), (256, 12, 1, 8)])
@pytest.mark.parametrize("call", ["chunk", "window"])
def test_references_that_rise_to_such_scores(sk, D, Hq, H, rows, call):       # noqa: F811
    """The largest scores stand late in a sequence, in copies enough that a CTA takes several (and that rows of windows
    go to the kernel of chunks)."""
    r = np.random.default_rng(D + Hq)
    keys = [_tied_keys(r, 700, D, hot_from=500)]
    cache, tables = _cache(r, keys, H, D, 64)
    q = np.full((rows, Hq, D), 32768.0, np.float16)
    q[..., 1::3] = 16384.0
    _run(sk, call, cache, tables, [700], q, rows, Hq, D, 32, copies=160)


def _near_keys(r, lens, D):
    """Scores of millions, at q0 = size / 64 and the others 16384 size / D, that differ by 0 to 12 times `size`."""
    keys = []
    for n in lens:
        k = np.full((n, D), 768.0)
        k[:, 0] = 64.0 * r.choice([0, 1, 2, 3, 4, 6, 8, 12], n)
        keys.append(k.astype(np.float16))
    return keys


@pytest.mark.parametrize("D,Hq,H,rows", FORMS)
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("size", [0.25, 1, 4, 16])
def test_small_differences_of_large_scores(sk, D, Hq, H, rows, wide, size):       # noqa: F811
    """On both sides of where a row's base is one float (exponents of 2^24)."""
    r = np.random.default_rng(D * Hq)
    lens, page = [150, 0, 41, 2], 32
    cache, tables = _cache(r, _near_keys(r, lens, D), H, D, page)
    q = np.full((len(lens) * rows, Hq, D), 16384.0 * size / D, np.float16)
    q[..., 0] = size / 64
    _run(sk, "chunk", cache, tables, lens, q, rows, Hq, D, 300 if wide else 5)


@pytest.mark.parametrize("D,Hq", [(64, 13), (128, 12), (256, 12)])
@pytest.mark.parametrize("size", [1, 16])
def test_small_differences_in_windows_of_many_rows(sk, D, Hq, size):       # noqa: F811
    r = np.random.default_rng(D * Hq)
    lens, page = [150, 0, 41, 2], 32
    cache, tables = _cache(r, _near_keys(r, lens, D), 1, D, page)
    q = np.full((len(lens) * 8, Hq, D), 16384.0 * size / D, np.float16)
    q[..., 0] = size / 64
    _run(sk, "window", cache, tables, lens, q, 8, Hq, D, 1600, copies=2)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("wide", [False, True])
def test_bases_that_cross_that_border(sk, D, wide):       # noqa: F811
    """Maxima that rise from block to block, from one-float bases to those of two, and rows of a warp that differ."""
    r = np.random.default_rng(D)
    n, Hq, rows = 330, 8, 5
    k = np.zeros((n, D))
    k[:, 0] = 2.0 ** -6 * r.choice([0, 1, 2, 3], n)
    k[:, 1] = np.repeat([0.0, 96.0, 192.0, 384.0, 768.0, 1536.0], 55)[:n]
    cache, tables = _cache(r, [k.astype(np.float16)], 1, D, 32)
    q = np.zeros((rows, Hq, D), np.float16)
    q[..., 0] = 64.0
    q[..., 1] = np.array([0.0, 1.0, 64.0, 2048.0, 8192.0, 16384.0, 24576.0, 32768.0])[:, None].T
    _run(sk, "chunk", cache, tables, [n], q, rows, Hq, D, 300 if wide else 11)
