"""The decode-round example's bookkeeping: the weight that decides what stays in the cache comes from the rows that were
accepted, and from no others."""
import importlib.util
import os

import numpy as np
import pytest

from gpu_util import host

pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_round.py")
    spec = importlib.util.spec_from_file_location("decode_round", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    return example


@pytest.mark.parametrize("rows", [1, 4, 8])
def test_rejected_rows_leave_no_weight(rows):
    """Without an eviction every accepted row's weights stay, and sum to one for each of its query heads."""
    example = _example()
    got = example.decode(rounds=25, rows=rows, page=32, high_water=256)
    assert got["evictions"] == 0 and got["length"] == len(got["report"])
    acc = host(got["acc"])[0]
    per_head = got["length"] * example.Q_HEADS // example.KV_HEADS
    # each row's weights are within 2^-13 of their sum (test_kv4_gpu.py's bound on a position's weight)
    assert np.all(np.abs(acc.sum(-1) - per_head) <= 2.0 ** -13 * per_head)
    assert np.all(acc[:, got["length"]:] == 0) and np.all(acc[:, :got["length"]] > 0)
