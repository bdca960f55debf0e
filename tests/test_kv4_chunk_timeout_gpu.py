"""Bounded waits of the chunk and window kernels that run out (the failure-injection hook of test_kv4_timeout_gpu.py): a
call ends by itself, reports SK_ERR_TIMEOUT and leaves nothing behind."""
import numpy as np
import pytest

from gpu_util import dev
from test_kv4_chunk_gpu import _rows_of, sk          # noqa: F401
from test_kv4_gpu import KG, VG, _case
from test_kv4_timeout_gpu import _timed

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,Hq,H", [(64, 14, 2), (128, 12, 1), (256, 12, 1)])
@pytest.mark.parametrize("width", [None, 300])
def test_chunks_whose_blocks_never_come(sk, D, Hq, H, width):       # noqa: F811
    import torch

    cache, table, lens, _ = _case(D, [300, 0, 129], 1, Hq, H, D, 32, width=width)
    q, starts = _rows_of(1, [40, 0, 3], Hq, D)
    a = (dev(q).unflatten(1, (Hq, D)), dev(cache), dev(np.clip(table, 0, len(cache) - 1)), dev(lens), dev(starts), KG, VG, 0.1)
    want = [x.clone() for x in sk.kv4_chunk_attention(*a)]
    _timed(sk, lambda: sk.kv4_chunk_attention(*a), 1)
    got = sk.kv4_chunk_attention(*a)
    assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("D,Hq,H,rows", [(64, 6, 2, 1), (128, 12, 1, 8), (256, 24, 1, 1)])
def test_windows_whose_copies_never_come(sk, D, Hq, H, rows):       # noqa: F811
    import torch

    cache, table, lens, q = _case(D, [300, 0, 129], rows, Hq, H, D, 32)
    a = (dev(q).unflatten(1, (Hq, D)), dev(cache), dev(np.clip(table, 0, len(cache) - 1)), dev(lens), KG, VG, 0.1, 200, 4, rows)
    want = [x.clone() for x in sk.kv4_window_attention(*a)]
    _timed(sk, lambda: sk.kv4_window_attention(*a), 1)
    got = sk.kv4_window_attention(*a)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
