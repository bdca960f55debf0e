"""More pieces of work than the list of a CTA of the chunk kernel has places, several times over; log sums of pieces of a
prompt and of replayed graphs; windows as long as the sequences with more rows than one pass takes. Tolerances as in
test_kv4_chunk_gpu.py."""
import numpy as np
import pytest

from gpu_util import Guarded, dev, host
from oracle import rope
from test_kv4_chunk_gpu import _check, _compare, _rows_of, sk          # noqa: F401
from test_kv4_gpu import KG, VG, _case

pytestmark = pytest.mark.gpu


def _short(seed, count):
    """Lengths and rows of short sequences: one position to three blocks, empty ones and ones of several tiles among them."""
    r = np.random.default_rng(seed)
    lens = [int(x) for x in np.where(r.random(count) < 0.15, r.integers(60, 180, count), r.integers(0, 20, count))]
    rows = [int(x) for x in np.where(r.random(count) < 0.05, r.integers(20, 60, count), r.integers(0, 5, count))]
    return lens, rows


@pytest.mark.parametrize("D,Hq,H", [(64, 16, 4), (128, 16, 4), (256, 12, 4)])
@pytest.mark.parametrize("width,window", [(None, 0), (300, 30)])
def test_several_laps_of_the_list(sk, D, Hq, H, width, window):       # noqa: F811
    """(at 152 SMs five to twelve pieces a CTA)"""
    lens, rows = _short(D, 260)
    cache, table, lens, _ = _case(D, lens, 1, Hq, H, D, 16, width=width)
    q, starts = _rows_of(D, rows, Hq, D)
    _check(sk, cache, table, lens, q, starts, Hq, D, window, 3)


@pytest.mark.parametrize("D,Hq,H", [(64, 14, 2), (128, 12, 1), (256, 24, 2)])
def test_log_sums_of_replays_whose_work_is_shared_out_anew(sk, D, Hq, H):       # noqa: F811
    """One captured call, lengths and starts changed on the device between replays: other tiles, cut elsewhere."""
    import torch

    lens0 = [190, 77, 300]
    cache, table, lens, _ = _case(9, lens0, 1, Hq, H, D, 16, width=300)
    q, starts = _rows_of(3, [150, 40, 3], Hq, D)
    qd, c, t, ln, st = dev(q).unflatten(1, (Hq, D)), dev(cache), dev(table), dev(lens), dev(starts)
    out, lse = Guarded((len(q), Hq, D), torch.float16), Guarded((len(q), Hq), torch.float32)
    call = lambda: sk.kv4_chunk_attention(qd, c, t, ln, st, KG, VG, D ** -0.5, out=out.t, lse=lse.t)      # noqa: E731
    call()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call()
    for n, s in (([190, 77, 300], [0, 150, 190, 193]), ([5, 77, 299], [0, 1, 2, 3]), ([0, 0, 300], [0, 0, 0, 150]),
                 ([190, 0, 1], [3, 193, 193, 193]), ([100, 50, 200], [0, 64, 65, 190])):
        ln.copy_(dev(np.array(n, np.int32)))
        st.copy_(dev(np.array(s, np.int32)))
        out.t.fill_(7.0)
        lse.t.fill_(7.0)
        graph.replay()
        y, z = out.host("out"), lse.host("lse")
        ref = rope.chunks(q.reshape(len(q), Hq, D), cache, table, n, s, KG, VG, D ** -0.5)
        there = np.zeros(len(q), bool)
        there[s[0]:s[-1]] = True
        _compare(y, z, ref, D, there)
        assert np.all(y[~there] == 7.0) and np.all(z[~there] == 7.0)


@pytest.mark.parametrize("D,Hq,H", [(64, 14, 2), (128, 12, 1), (256, 24, 2)])
def test_log_sums_of_a_prompt_in_pieces(sk, D, Hq, H):       # noqa: F811
    n = 190
    cache, table, lens, _ = _case(9, [n], 1, Hq, H, D, 16, width=300)
    q, _ = _rows_of(3, [n], Hq, D)
    qd, c, t = dev(q).unflatten(1, (Hq, D)), dev(cache), dev(table)
    y, z, at = [], [], 0
    for step in (100, 1, 60, 29):
        out, lse = sk.kv4_chunk_attention(qd[at:at + step], c, t, dev(np.array([at + step], np.int32)),
                                          dev(np.array([0, step], np.int32)), KG, VG, D ** -0.5)
        y.append(host(out))
        z.append(host(lse))
        at += step
    ref = rope.chunks(q.reshape(n, Hq, D), cache, table, lens, [0, n], KG, VG, D ** -0.5)
    _compare(np.concatenate(y), np.concatenate(z), ref, D, np.ones(n, bool))


@pytest.mark.parametrize("D,Hq,H,rows", [(256, 24, 2, 8), (256, 12, 1, 3), (64, 16, 1, 4), (64, 6, 2, 8)])
def test_windows_of_several_passes_as_long_as_the_sequences(sk, D, Hq, H, rows):       # noqa: F811
    """More than 24 rows a kv head: the same kernel and the same steps as without a window, so the same bits."""
    import torch

    assert rows * Hq // H >= 24
    cache, table, lens, q = _case(D, [300, 0, 65], rows, Hq, H, D, 16)
    a = (dev(q).unflatten(1, (Hq, D)), dev(cache), dev(table), dev(lens), KG, VG, 0.1)
    want = sk.kv4_attention(*a, rows=rows)
    got = sk.kv4_window_attention(*a, 1000, rows=rows)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
