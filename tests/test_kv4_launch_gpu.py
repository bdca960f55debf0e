"""The cache and log-probability calls launched in other ways: without programmatic dependent launch, back to back with
calls that depend on one another, and captured.  Results are bitwise those of separate calls."""
import contextlib

import numpy as np
import pytest

from gpu_util import dev
from test_kv4_gpu import KG, VG, _case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sk():
    import torch

    torch.cuda.set_device(0)
    import fp8_weight_only_skinny_gb300 as skm

    skm.init()
    yield skm
    assert skm.last_device_error() == skm.SK_OK


@contextlib.contextmanager
def _pdl(sk, on):
    was = sk.set_pdl(on)
    try:
        yield
    finally:
        sk.set_pdl(was)


def _round(sk, D, Hq, H, rows, width, gap):
    """Append, attend with weights, evict, attend again over what is kept; `gap` runs between the calls."""
    import torch

    page, lens = 32, [700, 0, 33]
    cache, table, n, q = _case(31, lens, rows, Hq, H, D, page, width=width)
    B, pages = len(lens), cache.shape[0]
    r = np.random.default_rng(2)
    c = torch.full((pages + 3 * B,) + cache.shape[1:], 0xFF, dtype=torch.uint8, device="cuda:0")
    c[:pages] = dev(cache)
    dst = dev(np.arange(pages, pages + 3 * B, dtype=np.int32).reshape(B, 3))
    x = dev(r.standard_normal((2, H, D)).astype(np.float16))
    slots = dev(np.array([int(table[0, 3]) * page + 5, int(table[2, 0]) * page + 31], np.int32))
    q, t, ln = dev(q).unflatten(1, (Hq, D)), dev(np.clip(table, 0, pages - 1)), dev(n)
    acc = torch.zeros(B, H, table.shape[1] * page, device="cuda:0")
    torch.cuda.synchronize()
    sk.kv4_append(x, x, slots, c, KG, VG)
    gap()
    out, lse = sk.kv4_attention(q, c, t, ln, KG, VG, 0.1, rows=rows, acc_out=acc)
    gap()
    new, kept, acc2 = sk.kv4_evict(c, t, ln, acc, dst, 90, 8)
    gap()
    out2, lse2 = sk.kv4_attention(q, c, dst, new, KG, VG, 0.1, rows=rows, acc=acc2, acc_out=acc2)
    torch.cuda.synchronize()
    return [out, lse, acc, new, kept, out2, lse2, acc2, c]


@pytest.mark.parametrize("D,Hq,H,rows", [(64, 6, 2, 1), (128, 12, 1, 2), (128, 12, 1, 8), (256, 24, 2, 2)])
@pytest.mark.parametrize("width", [None, 300])
def test_a_round_without_dependent_launch_and_without_gaps(sk, D, Hq, H, rows, width):
    import torch

    with _pdl(sk, False):
        want = _round(sk, D, Hq, H, rows, width, torch.cuda.synchronize)
    for on in (True, False):
        with _pdl(sk, on):
            for _ in range(5):
                assert all(torch.equal(a, b) for a, b in zip(want, _round(sk, D, Hq, H, rows, width, lambda: None)))


@pytest.mark.parametrize("M,N", [(700, 5003), (3, 151936), (1300, 20001)])
def test_log_probabilities_in_one_launch_or_two(sk, M, N):
    """More rows than CTAs take two launches, the second of which starts early; what follows them, and what they follow,
    keeps its place."""
    import torch

    r = torch.Generator(device="cuda").manual_seed(M)
    rows = [torch.randn(M, N, generator=r, device="cuda:0") for _ in range(2)]
    tok = torch.randint(0, N, (M,), generator=r, device="cuda:0", dtype=torch.int32)
    with _pdl(sk, False):
        want = [[x.clone() for x in sk.token_logprobs(z, tok, top_n=20)] for z in rows]
    torch.cuda.synchronize()
    z = rows[0].clone()
    for on in (True, False):
        with _pdl(sk, on):
            for _ in range(10):                       # the logits change under the calls, in stream order
                z.copy_(rows[0])
                a = sk.token_logprobs(z, tok, top_n=20)
                z.copy_(rows[1])
                b = sk.token_logprobs(z, tok, top_n=20)
                a_then = [x.clone() for x in a]
                z.fill_(float("nan"))
                torch.cuda.synchronize()
                for got, ref in ((a, want[0]), (a_then, want[0]), (b, want[1])):
                    assert all(torch.equal(x, y) for x, y in zip(got, ref))


def test_captured_log_probabilities(sk):
    import torch

    M, N = 900, 4001
    r = torch.Generator(device="cuda").manual_seed(1)
    rows = [torch.randn(M, N, generator=r, device="cuda:0").half() for _ in range(3)]
    tok = torch.randint(0, N, (M,), generator=r, device="cuda:0", dtype=torch.int32)
    want = [[x.clone() for x in sk.token_logprobs(z, tok, top_n=9, temperature=0.7)] for z in rows]
    z, out = rows[0].clone(), [torch.empty_like(x) for x in want[0]]

    def call():
        sk.token_logprobs(z, tok, top_n=9, temperature=0.7, logprob=out[0], rank=out[1], entropy=out[2], top_ids=out[3],
                          top_logprobs=out[4])

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
        after = [x.clone() for x in out]
    for i in (1, 2, 0, 1):
        z.copy_(rows[i])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) and torch.equal(w, y) for x, w, y in zip(out, after, want[i]))
