"""Bounded waits of the cache kernels that run out: with the failure-injection hook a call's kernels issue no copies, so
that every wait for one lasts its second and that for copies in flight another.  The call ends by itself, reports
SK_ERR_TIMEOUT and leaves nothing behind: the next call gives what it gives alone."""
import time

import numpy as np
import pytest

from gpu_util import dev
from oracle import kv4

pytestmark = pytest.mark.gpu

KG, VG = 0.02, 0.015
SK_ERR_TIMEOUT = 6


@pytest.fixture(scope="module")
def sk():
    import torch

    torch.cuda.set_device(0)
    import fp8_weight_only_skinny_gb300 as skm

    skm.init()
    yield skm
    assert skm.last_device_error() == skm.SK_OK


def _timed(sk, call, kernels):
    """Run `call` with the hook set; it has to end within three seconds a kernel that waits, and report the timeout."""
    import torch

    torch.cuda.synchronize()
    sk.lib.sk_inject_wait_timeout(1)
    t = time.time()
    call()
    torch.cuda.synchronize()
    t = time.time() - t
    assert 0.9 < t < 3.0 * kernels + 1.0, t
    assert sk.last_device_error() == SK_ERR_TIMEOUT
    assert sk.last_device_error() == sk.SK_OK                     # read once


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("D,Hq,H,rows", [(64, 6, 2, 1), (128, 12, 1, 2), (128, 12, 1, 8), (256, 24, 1, 1)])
def test_attention_whose_copies_never_come(sk, D, Hq, H, rows, wide, weights):
    import torch

    r = np.random.default_rng(D)
    page, lens = 32, [300, 0, 129]
    cache = np.zeros((14, H, 2, 18 * D), np.uint8)
    for j in range(14 * page):
        for h in range(H):
            kv4.write(cache, j, h, r.standard_normal(D).astype(np.float16), r.standard_normal(D).astype(np.float16), KG, VG)
    table = np.zeros((3, 300 if wide else 10), np.int32)
    table[:, :10] = np.arange(10)
    table[2, :5] = [13, 12, 11, 10, 9]
    q = dev(r.standard_normal((3 * rows, Hq, D)).astype(np.float16))
    c, t, n = dev(cache), dev(table), dev(np.array(lens, np.int32))
    acc = torch.zeros(3, H, table.shape[1] * page, device="cuda:0") if weights else None

    def call():
        if weights:
            acc.zero_()
        return [x.clone() for x in sk.kv4_attention(q, c, t, n, KG, VG, D ** -0.5, rows=rows, acc_out=acc)]

    want = call()
    sums = acc.clone() if weights else None
    _timed(sk, call, 2 if weights else 1)
    got = call()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert not weights or torch.equal(sums, acc)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("longest", [900, 9000])
def test_evict_whose_copies_never_come(sk, D, longest):
    import torch

    r = np.random.default_rng(D)
    page, H, budget = 16, 2, 200
    need, per = (longest + page - 1) // page, (budget + page - 1) // page
    c = dev(r.integers(0, 256, (need + per, H, 1, 18 * D), dtype=np.uint8))
    before = c.clone()
    table, dst = dev(np.arange(need, dtype=np.int32)[None]), dev(np.arange(need, need + per, dtype=np.int32)[None])
    n, acc = dev(np.array([longest], np.int32)), dev(r.random((1, H, need * page)).astype(np.float32))
    want = [x.clone() for x in sk.kv4_evict(c, table, n, acc, dst, budget, 20)]
    after = c.clone()
    c.copy_(before)
    _timed(sk, lambda: sk.kv4_evict(c, table, n, acc, dst, budget, 20), 1)
    assert torch.equal(c[:need], before[:need])                   # the source pages are only read
    got = sk.kv4_evict(c, table, n, acc, dst, budget, 20)
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and torch.equal(c, after)
