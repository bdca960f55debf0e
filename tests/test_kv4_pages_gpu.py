"""Where the cache's pages lie, and which are looked at: pages that no row sees any more may hold anything, and offsets
may pass 32 bits. The same positions are read in the same order, so results are compared bit for bit."""
import numpy as np
import pytest

from gpu_util import dev
from test_kv4_chunk_gpu import _rows_of, sk          # noqa: F401
from test_kv4_gpu import KG, VG, _case

pytestmark = pytest.mark.gpu

HEADS = [(64, 6, 2), (128, 12, 1), (256, 12, 1)]


def _bits(x):
    return [t.cpu().numpy().tobytes() for t in x]


@pytest.mark.parametrize("D,Hq,H", HEADS)
@pytest.mark.parametrize("n,window,sinks", [(1, 40, 4), (8, 33, 0), (70, 50, 20), (130, 1, 17)])
@pytest.mark.parametrize("width", [None, 300])
def test_pages_behind_a_window_may_be_given_away(sk, D, Hq, H, n, window, sinks, width):       # noqa: F811
    page, length = 16, 500
    cache, table, lens, _ = _case(D, [length], 1, Hq, H, D, page, width=width)
    q, starts = _rows_of(4, [n], Hq, D)
    held = cache.copy(), table.copy()
    for pg in range(length // page):
        if pg * page >= sinks and (pg + 1) * page <= length - n - window + 1:
            cache[table[0, pg]] = 0xFF                # scales that are no numbers
            table[0, pg] = -3 if pg % 2 else 1 << 30
    assert not np.array_equal(table, held[1])
    qd, ln, st = dev(q).unflatten(1, (Hq, D)), dev(lens), dev(starts)
    calls = [lambda c, t: sk.kv4_chunk_attention(qd, dev(c), dev(t), ln, st, KG, VG, 0.1, window=window, sinks=sinks)]
    if n <= 8:
        calls.append(lambda c, t: sk.kv4_window_attention(qd, dev(c), dev(t), ln, KG, VG, 0.1, window, sinks=sinks, rows=n))
    for call in calls:
        got = _bits(call(cache, table))
        assert got == _bits(call(*held))
        assert np.all(np.isfinite(np.frombuffer(got[0], np.float16)))


def test_offsets_beyond_32_bits(sk):                  # noqa: F811
    import torch

    D, Hq, H, page = 256, 12, 1, 64
    cache, table, lens, _ = _case(3, [300, 129], 1, Hq, H, D, page)
    q, starts = _rows_of(6, [40, 3], Hq, D)
    first = (1 << 32) // cache[0].size + 7
    big = sk.kv4_cache(first + len(cache), H, D, page)
    assert first * cache[0].size > 1 << 32
    small = dev(cache)
    big[first:] = small
    used = np.clip(table, 0, len(cache) - 1)
    qd, ln, st = dev(q).unflatten(1, (Hq, D)), dev(lens), dev(starts)
    low, high = dev(used), dev((used + first).astype(np.int32))
    for call in (lambda c, t: sk.kv4_chunk_attention(qd, c, t, ln, st, KG, VG, 0.1),
                 lambda c, t: sk.kv4_chunk_attention(qd, c, t, ln, st, KG, VG, 0.1, window=50, sinks=4),
                 lambda c, t: sk.kv4_window_attention(qd[:16], c, t, ln, KG, VG, 0.1, 50, sinks=4, rows=8)):
        assert _bits(call(big, high)) == _bits(call(small, low))
    r = np.random.default_rng(8)
    k, v = (dev(r.standard_normal((9, H, D)).astype(np.float16)) for _ in range(2))
    slots = np.arange(9, dtype=np.int32) * 5
    f, pos = sk.rope_frequencies(64), dev(np.arange(9, dtype=np.int32))
    a = sk.kv4_append_rope(qd[:9], k, v, dev(slots), pos, f, small, KG, VG)
    b = sk.kv4_append_rope(qd[:9], k, v, dev((slots + first * page).astype(np.int32)), pos, f, big, KG, VG)
    assert torch.equal(a, b) and torch.equal(big[first:], small)
