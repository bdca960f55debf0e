"""Bounded waits of the chunk kernel that run out where a CTA has more pieces of work than its list has places, and where
tiles cut between CTAs are joined after it: the call ends within the same seconds, reports SK_ERR_TIMEOUT and leaves
nothing behind (the failure-injection hook of test_kv4_timeout_gpu.py: blocks are decoded, and nobody is told)."""
import numpy as np
import pytest

from gpu_util import dev
from test_kv4_chunk_gpu import _rows_of, sk          # noqa: F401
from test_kv4_gpu import KG, VG
from test_kv4_timeout_gpu import _timed

pytestmark = pytest.mark.gpu


def _shared_pages(seed, lens, H, D, page, width):
    """A small pool of pages that hold tokens everywhere, shared by all sequences over and over."""
    r = np.random.default_rng(seed)
    cache = r.integers(0, 256, (7, H, page // 16, 18 * D), dtype=np.uint8)
    cache[..., 8 * D:9 * D] = r.integers(0x20, 0x38, cache[..., 8 * D:9 * D].shape)       # scales: numbers around one
    cache[..., 17 * D:] = r.integers(0x20, 0x38, cache[..., 17 * D:].shape)
    return cache, r.integers(0, 7, (len(lens), width)).astype(np.int32), np.array(lens, np.int32)


def _ends(sk, D, Hq, H, lens, rows, width, page):       # noqa: F811
    import torch

    cache, table, lens = _shared_pages(D, lens, H, D, page, width)
    q, starts = _rows_of(1, rows, Hq, D)
    a = (dev(q).unflatten(1, (Hq, D)), dev(cache), dev(table), dev(lens), dev(starts), KG, VG, 0.1)
    want = [x.clone() for x in sk.kv4_chunk_attention(*a)]
    assert bool(torch.isfinite(want[0]).all())              # (log sums of rows before the first position are -inf)
    _timed(sk, lambda: sk.kv4_chunk_attention(*a), 1)
    got = sk.kv4_chunk_attention(*a)
    assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_more_pieces_than_the_list_holds(sk, D):       # noqa: F811
    """(at 152 SMs six pieces a CTA, eleven a pair of CTAs)"""
    _ends(sk, D, 12, 2, [300, 5, 1, 129] * 100, [3] * 400, 21, 16)


@pytest.mark.parametrize("D,small", [(64, 140), (128, 140), (256, 70)])
def test_few_tiles_of_which_one_is_joined(sk, D, small):       # noqa: F811
    """One sequence of a million positions, cut between most CTAs, and short ones, twelve or more a CTA, fewer in all than
    CTAs: the join looks at every tile's entry."""
    _ends(sk, D, 12, 1, [1000003] + [5] * small, [1] * (small + 1), 977, 1024)
