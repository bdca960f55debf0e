"""GPU parity of token_logprobs against the float64 oracle (oracle/kv4.py).

Tolerances, fixed before the first run: a term 2^d of the sum is within
2^-21 + |d| 2^-23 relative, terms below 2^-30 of the largest not mattering, and
a thread adds at most a few hundred terms before the tree: ln S is within
2^-14.  So a log probability is within 2^-14 + 2^-21 |lp|, and the entropy,
whose second sum weighs the terms by |d|, within 2^-13 (1 + H).  Ranks and
indices are exact."""
import numpy as np
import pytest

from gpu_util import Guarded, dev, host
from oracle import kv4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sk():
    import torch

    torch.cuda.set_device(0)
    import fp8_weight_only_skinny_gb300 as skm

    skm.init()
    return skm


def _check(sk, z, tokens, T, n, stride_pad=0, offset=0):
    import torch

    M, N = z.shape
    wide = np.full((M, N + stride_pad + offset), 1e4, z.dtype)     # what lies between the rows must not count
    wide[:, offset:offset + N] = z
    zd = dev(wide)[:, offset:offset + N]
    outs = [Guarded((M,), torch.float32), Guarded((M,), torch.int32, fill=-9), Guarded((M,), torch.float32),
            Guarded((M, n), torch.int32, fill=-9), Guarded((M, n), torch.float32)]
    sk.token_logprobs(zd, dev(np.asarray(tokens, np.int32)), top_n=n, temperature=T, logprob=outs[0].t, rank=outs[1].t,
                      entropy=outs[2].t, top_ids=outs[3].t, top_logprobs=outs[4].t)
    lp, rank, ent, ids, top = (o.host("logprobs") for o in outs)
    for r in range(M):
        wl, wr, we, wi, wt = kv4.logprobs(z[r], int(tokens[r]), T, n)
        assert rank[r] == wr, (r, rank[r], wr)
        assert np.array_equal(ids[r], wi), (r, ids[r], wi)
        for got, want, tol in ((lp[r], wl, 2.0 ** -14 + 2.0 ** -21 * abs(wl)), (ent[r], we, 2.0 ** -13 * (1 + abs(we)))):
            assert (np.isnan(want) and np.isnan(got)) or got == want or abs(got - want) <= tol, (r, got, want)
        fin = np.isfinite(wt)
        assert np.array_equal(np.isnan(top[r]), np.isnan(wt)) and np.array_equal(np.isneginf(top[r]), np.isneginf(wt))
        assert np.all(np.abs(top[r] - wt)[fin] <= (2.0 ** -14 + 2.0 ** -21 * np.abs(wt))[fin])


@pytest.mark.parametrize("dtype", [np.float32, np.float16])
@pytest.mark.parametrize("M,N,n", [(1, 1, 1), (3, 2, 5), (2, 7, 7), (5, 255, 20), (4, 4095, 64), (2, 4097, 1), (3, 8193, 20),
                                   (1, 65537, 5), (2, 151936, 20), (9, 10007, 0), (400, 1234, 8), (700, 5003, 5)])
@pytest.mark.parametrize("T", [1.0, 0.6])
def test_rows_of_all_lengths(sk, dtype, M, N, n, T):
    r = np.random.default_rng(M * N)
    z = (r.standard_normal((M, N)) * 3).astype(dtype)
    _check(sk, z, r.integers(0, N, M), T, n)


@pytest.mark.parametrize("dtype", [np.float32, np.float16])
@pytest.mark.parametrize("pad,offset", [(1, 0), (3, 1), (0, 5), (13, 2)])
def test_rows_at_odd_addresses(sk, dtype, pad, offset):
    r = np.random.default_rng(pad)
    z = (r.standard_normal((6, 5003)) * 2).astype(dtype)
    _check(sk, z, r.integers(0, 5003, 6), 1.3, 9, pad, offset)


@pytest.mark.parametrize("dtype", [np.float32, np.float16])
def test_ties_go_to_the_lower_index(sk, dtype):
    r = np.random.default_rng(4)
    z = r.integers(-2, 3, (5, 9001)).astype(dtype)
    z[0] = 0
    z[1, ::2] = -0.0
    z[1, 1::2] = 0.0
    _check(sk, z, [0, 9000, 4500, 8999, 17], 1.0, 33)


@pytest.mark.parametrize("order", [1, -1])
@pytest.mark.parametrize("N", [9001, 70001])
def test_sorted_rows(sk, order, N):
    """Rising logits put every round's entries above all before them."""
    z = np.tile(np.linspace(-20, 20, N, dtype=np.float32)[::order], (2, 1))
    _check(sk, z, [3, N - 2], 1.0, 20)


def test_masked_rows(sk):
    r = np.random.default_rng(6)
    z = r.standard_normal((8, 6000)).astype(np.float32)
    z[0, ::3] = -np.inf
    z[1, :5990] = -np.inf
    z[2] = -np.inf
    z[3, :] = -np.inf
    z[3, 4321] = -2.0
    z[4, ::2] = np.finfo(np.float32).min
    z[5, 17] = np.nan
    z[6, 17] = np.inf
    z[7, :] = -1e30
    with np.errstate(invalid="ignore"):
        _check(sk, z[[0, 1, 2, 3, 4, 6, 7]], [0, 5995, 7, 4321, 2, 17, 5], 1.0, 12)
    lp, _, ent, _, top = sk.token_logprobs(dev(z[5:6]), dev(np.array([3], np.int32)), top_n=2)
    assert np.isnan(host(lp)).all() and np.isnan(host(ent)).all() and np.isnan(host(top)).all()
    h = r.standard_normal((2, 5000)).astype(np.float16)
    h[0, ::2] = np.finfo(np.float16).min
    h[1, ::5] = -np.inf
    _check(sk, h, [1, 0], 0.8, 6)


@pytest.mark.parametrize("dtype", [np.float32, np.float16])
@pytest.mark.parametrize("M,N,n", [(700, 300, 20), (3, 1023, 20), (5, 1024, 64), (5, 1025, 64), (700, 1025, 20),
                                   (650, 2048, 33), (650, 2049, 5), (620, 19, 40), (640, 1, 2)])
def test_short_rows(sk, dtype, M, N, n):
    """One round of a narrow CTA, two of them, and the lengths on either side."""
    r = np.random.default_rng(M + N)
    z = (r.standard_normal((M, N)) * 3).astype(dtype)
    z[M // 2] = np.sort(z[M // 2])
    z[M // 3] = 1.0
    z[M - 1, : N // 2] = -np.inf
    _check(sk, z, r.integers(N // 2, N, M), 1.0, n)
    if N > 2:
        _check(sk, z[:, 1:], r.integers(N // 2, N - 1, M), 0.7, n, 3, 1)


@pytest.mark.parametrize("order", [1, -1])
def test_sorted_short_rows(sk, order):
    z = np.tile(np.linspace(-20, 20, 2000, dtype=np.float32)[::order], (640, 1))
    _check(sk, z, np.full(640, 1999), 1.0, 64)


def test_outputs_belong_to_the_given_stream(sk):
    """Outputs made by a call on a stream come from that stream's memory: freed, they go to it and to no other."""
    import torch

    s = torch.cuda.Stream()
    z = torch.randn((3, 70000), device="cuda")
    torch.cuda.synchronize()
    got = sk.token_logprobs(z, top_n=4, stream=s)
    s.synchronize()
    at = {t.data_ptr() for t in got if t is not None}
    want = sk.token_logprobs(z, top_n=4)
    torch.cuda.synchronize()
    assert torch.equal(got[3], want[3])
    del got
    other = [torch.empty(3, 4, device="cuda") for _ in range(8)]
    assert at.isdisjoint({t.data_ptr() for t in other})


def test_tokens_outside_the_row_and_calls_without_tokens(sk):
    z = np.random.default_rng(9).standard_normal((3, 1000)).astype(np.float32)
    _check(sk, z, [-1, 1000, -100], 1.0, 4)
    lp, rank, ent, ids, top = sk.token_logprobs(dev(z), top_n=3)
    assert lp is None and rank is None
    for r in range(3):
        assert np.array_equal(host(ids)[r], kv4.logprobs(z[r], 0, 1.0, 3)[3])


def test_repeated_calls_are_identical_and_flat_rows_have_full_entropy(sk):
    import torch

    z = torch.randn(5, 151936, device="cuda:0")
    z[4] = 1.5
    t = torch.tensor([1, 2, 3, 4, 5], dtype=torch.int32, device="cuda:0")
    a = [x.clone() for x in sk.token_logprobs(z, t, top_n=20)]
    for _ in range(3):
        for x, y in zip(a, sk.token_logprobs(z, t, top_n=20)):
            assert torch.equal(x, y)
    assert abs(float(a[2][4]) - np.log(151936)) < 1e-3 and list(host(a[3])[4]) == list(range(20))


def test_binding_refusals(sk):
    import torch

    z = torch.zeros(2, 10, device="cuda:0")
    t = torch.zeros(2, dtype=torch.int32, device="cuda:0")
    with pytest.raises(TypeError):
        sk.token_logprobs(z.double(), t)
    with pytest.raises(ValueError):
        sk.token_logprobs(z.t(), t)
    with pytest.raises(ValueError):
        sk.token_logprobs(z, t.long())
    with pytest.raises(sk.SkinnyError):
        sk.token_logprobs(z, t, top_n=65)
    with pytest.raises(sk.SkinnyError):
        sk.token_logprobs(z, t, temperature=0.0)
