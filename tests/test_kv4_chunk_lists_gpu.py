"""Sequences without positions that have rows all the same (the unused places of a padded batch), many in a row and after
ones that hold something: a CTA of the chunk kernel takes several such pieces of work after one with blocks, and rows of
sequences without positions are zeros with a log sum of minus infinity. Tolerances as in test_kv4_chunk_gpu.py."""
import numpy as np
import pytest

from test_kv4_chunk_gpu import _check, _check_window, _rows_of, sk          # noqa: F401
from test_kv4_gpu import _case

pytestmark = pytest.mark.gpu

# (at 152 SMs up to eight pieces a CTA, on 12 to 32 CTAs one with blocks before three and more without)
LENS = [130] + [0] * 25 + [70] + [0] * 6


@pytest.mark.parametrize("D,Hq,H", [(64, 32, 32), (128, 32, 32), (256, 16, 16)])
@pytest.mark.parametrize("width,window,sinks", [(None, 0, 0), (300, 0, 0), (None, 40, 4)])
def test_runs_of_empty_sequences_with_rows(sk, D, Hq, H, width, window, sinks):       # noqa: F811
    cache, table, lens, _ = _case(D, LENS, 1, Hq, H, D, 16, width=width)
    q, starts = _rows_of(D, [1] * len(LENS), Hq, D)
    y = _check(sk, cache, table, lens, q, starts, Hq, D, window, sinks)
    assert np.all(y[np.array(LENS) == 0] == 0) and np.all(np.any(y[np.array(LENS) > 0] != 0, -1))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows", [3, 40])
def test_rows_before_the_first_position_in_every_sequence(sk, D, rows):       # noqa: F811
    """More rows than positions: tiles that see nothing beside ones that see a little."""
    lens = [1, 2, 0, 0, 0, 65, 0, 0, 0, 0, 1, 0, 0, 0] * 3
    cache, table, lens, _ = _case(D, lens, 1, 64, 8, D, 16)
    q, starts = _rows_of(D, [rows] * len(lens), 64, D)
    _check(sk, cache, table, lens, q, starts, 64, D)


@pytest.mark.parametrize("D,Hq,H", [(64, 104, 8), (128, 96, 8), (256, 96, 8)])
def test_windows_over_padded_batches(sk, D, Hq, H):       # noqa: F811
    """Rows enough for the kernel of chunks; most sequences of the batch are empty."""
    lens = ([70] + [0] * 11) * 6
    cache, table, lens, q = _case(D, lens, 8, Hq, H, D, 16, width=30)
    _check_window(sk, cache, table, lens, q, 8, Hq, D, 400, 4)
