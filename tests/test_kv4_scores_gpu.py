"""GPU tests of kv4_attention where the scores are far larger than a model's: the softmax of scores is unchanged by what
all of them have in common, however large, so neither the output nor the weights may depend on it.

The cases' scores are whole numbers below 2^24 times a power of two, sums of such products, so FP32 holds them exactly and
the error of the scores (e of test_kv4_gpu.py) is zero.  What is left, derived before the first run: a weight's rounding to
FP16 (2^-11) and the exponential and sums (2^-15) times sum_j p_j |v_j|, and half a ulp of the FP16 output (2^-11 |out|,
2^-25 at least); the log sum is within 2^-16 + 2^-22 |lse|; a position's weight w added to a is within
2^-15 w + 2^-22 (a + w) + 2^-24."""
import numpy as np
import pytest

from gpu_util import Guarded, dev
from oracle import kv4

pytestmark = pytest.mark.gpu

FORMS = [(64, 6, 2, 1), (64, 8, 1, 4), (128, 12, 1, 1), (128, 12, 1, 8), (128, 28, 1, 1), (128, 13, 1, 8), (256, 6, 2, 2),
         (256, 24, 1, 1)]
VG = 0.015


@pytest.fixture(scope="module")
def sk():
    import torch

    torch.cuda.set_device(0)
    import fp8_weight_only_skinny_gb300 as skm

    skm.init()
    yield skm
    assert skm.last_device_error() == skm.SK_OK


def _cache(r, keys, H, D, page):
    """A cache whose sequence j's positions hold keys[j] (FP16 [n][D]) in every head, under a key scale of one."""
    need = [(len(k) + page - 1) // page for k in keys]
    cache = np.full((sum(need) + 1, H, page // 16, 18 * D), 0xFF, np.uint8)
    order, at = r.permutation(len(cache)).astype(np.int32), 0
    tables = []
    for k, pages in zip(keys, need):
        tables.append(order[at:at + pages])
        at += pages
        for j in range(len(k)):
            for h in range(H):
                kv4.write(cache, int(tables[-1][j // page]) * page + j % page, h, k[j], r.standard_normal(D).astype(np.float16),
                          1.0, VG)
    return cache, tables


def _run(sk, cache, tables, lens, q, rows, Hq, D, scale, width, copies=1, weights=False):
    """Compare a call (the sequences `copies` times over) with the oracle."""
    import torch

    page, H, B = cache.shape[2] * 16, cache.shape[1], len(lens) * copies
    table = np.zeros((len(lens), width), np.int32)
    for b, t in enumerate(tables):
        table[b, :len(t)] = t
    n = B * rows
    out, lse = Guarded((n, Hq, D), torch.float16), Guarded((n, Hq), torch.float32)
    acc = np.random.default_rng(1).random((len(lens), H, width * page)).astype(np.float32)
    ao = Guarded((B, H, width * page), torch.float32, fill=7.0) if weights else None
    sk.kv4_attention(dev(np.tile(q, (copies, 1, 1))), dev(cache), dev(np.tile(table, (copies, 1))),
                     dev(np.tile(np.array(lens, np.int32), copies)), 1.0, VG, scale, rows=rows, out=out.t, lse=lse.t,
                     **({"acc": dev(np.tile(acc, (copies, 1, 1))), "acc_out": ao.t} if weights else {}))
    ref = kv4.attention(q, cache, table, lens, 1.0, VG, scale, rows)
    tol = (2.0 ** -11 + 2.0 ** -15) * ref["absum"] + 2.0 ** -11 * np.abs(ref["out"]) + 2.0 ** -25
    empty = np.isneginf(ref["lse"])
    y, z, got = out.host("out"), lse.host("lse"), ao.host("acc") if weights else None
    for c in range(copies):
        part = slice(c * len(lens) * rows, (c + 1) * len(lens) * rows)
        assert np.all(np.isfinite(y[part])) and np.all(np.abs(y[part] - ref["out"]) <= tol), c
        assert np.array_equal(np.isneginf(z[part]), empty)
        off = np.abs(z[part][~empty] - ref["lse"][~empty])
        assert np.all(off <= 2.0 ** -16 + 2.0 ** -22 * np.abs(ref["lse"][~empty])), c
        for b, m in enumerate(lens if weights else []):
            w, old = ref["weights"][b, :, :m], acc[b, :, :m].astype(np.float64)
            a = got[c * len(lens) + b]
            assert np.all(np.abs(a[:, :m] - (old + w)) <= 2.0 ** -15 * w + 2.0 ** -22 * (old + w) + 2.0 ** -24), (c, b)
            assert np.all(a[:, m:] == 7.0)


def _tied_keys(r, n, D, hot_from=0):
    """Keys of +-1536 in all components: a tenth of the positions from hot_from on give the largest score, 2^32 and more,
    the others zero or its opposite."""
    k = np.where(np.arange(D) % 2, -1536.0, 1536.0) * np.ones((n, 1))
    k[r.random(n) < 0.3] = -1536.0
    hot = np.arange(n) >= hot_from
    hot &= r.random(n) < 0.1
    hot[-1] = True
    k[hot] = 1536.0
    return k.astype(np.float16)


@pytest.mark.parametrize("D,Hq,H,rows", FORMS)
@pytest.mark.parametrize("wide", [False, True])
def test_equal_scores_of_any_size_share_the_weight(sk, D, Hq, H, rows, wide):
    r = np.random.default_rng(D + Hq)
    lens, page = [200, 0, 37, 1], 32
    keys = [_tied_keys(r, n, D) if n else np.zeros((0, D), np.float16) for n in lens]
    cache, tables = _cache(r, keys, H, D, page)
    q = np.full((len(lens) * rows, Hq, D), 32768.0, np.float16)
    q[..., 1::3] = 16384.0
    q[..., 2::3] = -32768.0
    _run(sk, cache, tables, lens, q, rows, Hq, D, 0.7, 300 if wide else 7)


@pytest.mark.parametrize("D,Hq,H,rows", [(64, 6, 2, 1), (128, 12, 1, 1), (128, 12, 1, 8), (256, 12, 1, 1)])
def test_references_that_rise_to_such_scores(sk, D, Hq, H, rows):
    """The largest scores stand late in a sequence; enough copies of it that a CTA takes several tiles in turn."""
    r = np.random.default_rng(D + Hq)
    keys = [_tied_keys(r, 700, D, hot_from=500)]
    cache, tables = _cache(r, keys, H, D, 64)
    q = np.full((rows, Hq, D), 32768.0, np.float16)
    q[..., 1::3] = 16384.0
    _run(sk, cache, tables, [700], q, rows, Hq, D, 0.7, 32, copies=160)


@pytest.mark.parametrize("D,Hq,H,rows", FORMS)
@pytest.mark.parametrize("wide", [False, True])
def test_small_differences_of_large_scores(sk, D, Hq, H, rows, wide):
    """Scores of millions that differ by 0 to 12: the output and the weights are those of the differences."""
    r = np.random.default_rng(D * Hq)
    lens, page = [150, 0, 41, 2], 32
    keys = []
    for n in lens:
        k = np.full((n, D), 768.0)
        k[:, 0] = 64.0 * r.choice([0, 1, 2, 3, 4, 6, 8, 12], n)
        keys.append(k.astype(np.float16))
    cache, tables = _cache(r, keys, H, D, page)
    q = np.full((len(lens) * rows, Hq, D), 16384.0 / D, np.float16)
    q[..., 0] = 1 / 64
    _run(sk, cache, tables, lens, q, rows, Hq, D, 0.7, 300 if wide else 5)


@pytest.mark.parametrize("D,Hq,H,rows", FORMS)
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("tied", [False, True])
def test_weights_of_large_scores(sk, D, Hq, H, rows, wide, tied):
    """What positions get is what the outputs were made of, whatever the scores' size."""
    r = np.random.default_rng(D * Hq + 1)
    lens, page = [150, 0, 41, 1], 32
    keys = []
    for n in lens:
        k = np.full((n, D), 768.0)
        k[:, 0] = 64.0 * r.choice([0, 1, 2, 3, 4, 6, 8, 12], n)
        keys.append(_tied_keys(r, n, D) if tied and n else k.astype(np.float16))
    cache, tables = _cache(r, keys, H, D, page)
    q = np.full((len(lens) * rows, Hq, D), 32768.0 if tied else 16384.0 / D, np.float16)
    if tied:
        q[..., 1::3] = 16384.0
    else:
        q[..., 0] = 1 / 64
    _run(sk, cache, tables, lens, q, rows, Hq, D, 0.7, 300 if wide else 5, weights=True)
