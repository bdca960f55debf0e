"""GPU parity of kv4_chunk_attention and kv4_window_attention against the float64 oracle (oracle/rope.py `chunks`).

Tolerances as in test_kv4_gpu.py, fixed before the first run: with u = 2^-24 a score is within e = (D/16 + 16) 2 u zmax
(D exact products in D/16 steps, and the exponent's roundings, which are of the score's size), plus 4 u |lse|; a weight
within 2 e + 2^-20, and 2^-11 more in FP16; the sums add 2^-16 at most at these lengths:
|dout| <= (2^-11 + 4 e + 2^-15) sum_j p_j |v_j| + 2^-11 |out| + 2^-25,  |dlse| <= e + 2^-16 + 2^-22 |lse|.
"""
import numpy as np
import pytest

from gpu_util import Guarded, dev
from oracle import rope
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


def _rows_of(seed, counts, Hq, D, gap=0, spread=1.5, behind=0):
    r = np.random.default_rng(seed)
    q = (r.standard_normal((sum(counts) + behind, Hq * D + gap)) * spread).astype(np.float16)
    return q, np.concatenate(([0], np.cumsum(counts))).astype(np.int32)


def _compare(y, z, ref, D, there):
    u = 2.0 ** -24
    out, lse, absum, zmax = (ref[k][there] for k in ("out", "lse", "absum", "zmax"))
    e = (D / 16 + 16) * 2 * u * zmax + 4 * u * np.abs(np.where(np.isfinite(lse), lse, 0))
    tol = (2.0 ** -11 + 4 * e[..., None] + 2.0 ** -15) * absum + 2.0 ** -11 * np.abs(out) + 2.0 ** -25
    assert np.all(np.abs(y[there] - out) <= tol), np.max(np.abs(y[there] - out) / tol)
    empty = np.isneginf(lse)
    assert np.array_equal(np.isneginf(z[there]), empty)
    assert np.all(np.abs(z[there] - lse)[~empty] <= (e + 2.0 ** -16 + 2.0 ** -22 * np.abs(lse))[~empty])


def _check(sk, cache, table, lens, q, starts, Hq, D, window=0, sinks=0, scale=None):
    import torch

    rows = len(q)
    out, lse = Guarded((rows, Hq, D), torch.float16, fill=7.0), Guarded((rows, Hq), torch.float32, fill=7.0)
    scale = scale or D ** -0.5
    sk.kv4_chunk_attention(dev(q)[:, :Hq * D].unflatten(1, (Hq, D)), dev(cache), dev(table), dev(lens), dev(starts), KG, VG,
                           scale, window=window, sinks=sinks, out=out.t, lse=lse.t)
    y, z = out.host("out"), lse.host("lse")
    cap = table.shape[1] * cache.shape[2] * 16
    ref = rope.chunks(q[:, :Hq * D].reshape(rows, Hq, D), cache, table, np.clip(lens, 0, cap), starts, KG, VG, scale, window,
                      sinks)
    there = np.zeros(rows, bool)
    there[starts[0]:starts[-1]] = True
    _compare(y, z, ref, D, there)
    assert np.all(y[~there] == 7.0) and np.all(z[~there] == 7.0)          # rows of no sequence stay as they were
    return y


LENS = [0, 1, 17, 64, 65, 200, 3, 128]
ROWS = [0, 1, 5, 64, 3, 130, 5, 1]           # of the seventh, two rows come before its first position


@pytest.mark.parametrize("Hq,H,D,page", [(6, 2, 64, 16), (7, 1, 128, 48), (3, 3, 256, 16), (12, 1, 256, 64), (24, 2, 64, 32),
                                         (2, 2, 128, 16)])
@pytest.mark.parametrize("width", [None, 300])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (16, 4), (100, 20), (33, 64)])
def test_ragged_chunks(sk, Hq, H, D, page, width, window, sinks):
    """A table as narrow as the longest sequence takes one launch, a wide one parts that are joined."""
    cache, table, lens, _ = _case(D + Hq, LENS, 1, Hq, H, D, page, width=width)
    q, starts = _rows_of(D, ROWS, Hq, D, gap=8, behind=3)
    _check(sk, cache, table, lens, q, starts, Hq, D, window, sinks)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,rows,G", [(63, 1, 1), (64, 1, 12), (65, 11, 12), (127, 10, 13), (128, 21, 12), (129, 22, 12), (700, 1, 1),
                                      (700, 43, 6), (1500, 2, 12), (1500, 90, 3)])
def test_one_sequence_in_parts(sk, D, n, rows, G):
    """Tiles of one row to several, of which most CTAs have a part."""
    cache, table, lens, _ = _case(n + rows, [n], 1, G, 1, D, 16, width=200)
    q, starts = _rows_of(n, [rows], G, D)
    _check(sk, cache, table, lens, q, starts, G, D)


@pytest.mark.parametrize("D,Hq,H", [(64, 24, 2), (128, 12, 1), (256, 24, 2)])
@pytest.mark.parametrize("window", [0, 20])
def test_many_sequences_and_several_tiles_a_cta(sk, D, Hq, H, window):
    """More sequences than a warp has lanes, more tiles than CTAs, empty and single rows among them."""
    r = np.random.default_rng(D)
    lens = [int(x) for x in r.integers(0, 90, 45)]
    rows = [int(min(x, n + 2)) for x, n in zip(r.integers(0, 60, 45), lens)]
    cache, table, lens, _ = _case(D, lens, 1, Hq, H, D, 16)
    q, starts = _rows_of(D, rows, Hq, D)
    _check(sk, cache, table, lens, q, starts, Hq, D, window, 3)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("spread", [0.01, 8.0, 60.0])
def test_bases_that_move_and_scores_far_apart(sk, D, spread):
    """Keys whose size grows and falls along the sequence, so that rows' maxima rise from block to block."""
    from oracle import kv4

    r = np.random.default_rng(D)
    n, Hq, page = 400, 6, 16
    cache = np.zeros((n // page, 1, 1, 18 * D), np.uint8)
    table = r.permutation(n // page).astype(np.int32)[None]
    for j in range(n):
        grow = 0.05 + (j % 150) / 40
        kv4.write(cache, int(table[0, j // page]) * page + j % page, 0, (r.standard_normal(D) * grow).astype(np.float16),
                  r.standard_normal(D).astype(np.float16), KG, VG)
    q, starts = _rows_of(1, [50], Hq, D, spread=spread)
    _check(sk, cache, table, np.array([n], np.int32), q, starts, Hq, D)
    wide = np.zeros((1, 400), np.int32)
    wide[:, :n // page] = table
    _check(sk, cache, wide, np.array([n], np.int32), q, starts, Hq, D)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_lengths_outside_the_table_and_starts_that_leave_rows_out(sk, D):
    cache, table, lens, _ = _case(D, [40, 30, 0], 1, 4, 2, D, 16)
    q, _ = _rows_of(2, [12], 4, D)
    lens = np.array([40, -5, 0], np.int32)
    table[1] = table[0]
    _check(sk, cache, table, lens, q, np.array([2, 7, 9, 9], np.int32), 4, D)
    lens = np.array([40, 30, 1 << 30], np.int32)
    table = np.tile(table[:1], (3, 1))
    full = table.shape[1] * 16
    cache[table[0, -1]] = cache[table[0, 0]]                      # the table's end holds tokens, too
    _check(sk, cache, table, np.array([40, 30, full], np.int32), q, np.array([0, 3, 7, 12], np.int32), 4, D)
    _check(sk, cache, table, lens, q, np.array([0, 3, 7, 12], np.int32), 4, D)


@pytest.mark.parametrize("D,Hq,H", [(64, 14, 2), (128, 12, 1), (256, 24, 2)])
def test_repeated_calls_pieces_and_captures_agree(sk, D, Hq, H):
    """The same call gives the same bits; a prompt in one piece and in three agree within the tolerance; a captured call
    follows lengths and starts that change on the device."""
    import torch

    n = 190
    cache, table, lens, _ = _case(9, [n, 77], 1, Hq, H, D, 16, width=300)
    q, starts = _rows_of(3, [n, 77], Hq, D)
    want = _check(sk, cache, table, lens, q, starts, Hq, D)
    qd, c, t = dev(q).unflatten(1, (Hq, D)), dev(cache), dev(table)
    ln, st = dev(lens), dev(starts)
    out = torch.zeros(len(q), Hq, D, dtype=torch.float16, device="cuda:0")
    call = lambda: sk.kv4_chunk_attention(qd, c, t, ln, st, KG, VG, D ** -0.5, out=out)      # noqa: E731
    for _ in range(3):
        call()
        torch.cuda.synchronize()
        assert np.array_equal(out.cpu().numpy().astype(np.float64), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    at = [0, 0]
    pieces = torch.zeros_like(out)
    for step in ((100, 7), (60, 0), (30, 70)):
        # these rows alone, at the front of q's sequences: rows [at, at + step) of each
        first = [at[0], n + at[1]]
        rows = torch.cat([qd[f:f + s] for f, s in zip(first, step)])
        got, _ = sk.kv4_chunk_attention(rows, c, t, dev(np.array([at[0] + step[0], at[1] + step[1]], np.int32)),
                                        dev(np.array([0, step[0], sum(step)], np.int32)), KG, VG, D ** -0.5)
        pieces[first[0]:first[0] + step[0]] = got[:step[0]]
        pieces[first[1]:first[1] + step[1]] = got[step[0]:]
        at = [a + s for a, s in zip(at, step)]
    ref = rope.chunks(q.reshape(len(q), Hq, D), cache, table, lens, starts, KG, VG, D ** -0.5)
    _compare(pieces.cpu().numpy().astype(np.float64), ref["lse"], ref, D, np.ones(len(q), bool))
    ln.copy_(dev(np.array([120, 5], np.int32)))
    st.copy_(dev(np.array([0, 13, 18], np.int32)))
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    ref = rope.chunks(q.reshape(len(q), Hq, D), cache, table, [120, 5], [0, 13, 18], KG, VG, D ** -0.5)
    there = np.arange(len(q)) < 18
    y = out.cpu().numpy().astype(np.float64)
    _compare(y, np.where(there[:, None], ref["lse"], 0), ref, D, there)
    assert np.all(y[18:] == 0)


def test_streams_with_workspaces_of_their_own(sk):
    import torch

    D, Hq, H = 128, 12, 1
    cache, table, lens, _ = _case(5, [600], 1, Hq, H, D, 16, width=300)
    c, t, ln = dev(cache), dev(table), dev(lens)
    calls = [_rows_of(s, [40 + s], Hq, D) for s in range(3)]
    args = [(dev(q).unflatten(1, (Hq, D)), dev(st)) for q, st in calls]
    want = [sk.kv4_chunk_attention(q, c, t, ln, st, KG, VG, 0.1) for q, st in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    for s in streams:
        sk.stream_workspace(s, 1 << 20)
    try:
        for _ in range(5):
            got = [sk.kv4_chunk_attention(q, c, t, ln, st, KG, VG, 0.1, stream=s) for (q, st), s in zip(args, streams)]
            torch.cuda.synchronize()
            for a, b in zip(got, want):
                assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    finally:
        for s in streams:
            sk.stream_workspace(s, 0)


# ------------------------------------------------------------------ window ---

def _check_window(sk, cache, table, lens, q, rows, Hq, D, window, sinks):
    import torch

    B = len(lens)
    out, lse = Guarded((B * rows, Hq, D), torch.float16), Guarded((B * rows, Hq), torch.float32)
    sk.kv4_window_attention(dev(q)[:, :Hq * D].unflatten(1, (Hq, D)), dev(cache), dev(table), dev(lens), KG, VG, D ** -0.5,
                            window, sinks=sinks, rows=rows, out=out.t, lse=lse.t)
    y, z = out.host("out"), lse.host("lse")
    cap = table.shape[1] * cache.shape[2] * 16
    ref = rope.chunks(q[:, :Hq * D].reshape(B * rows, Hq, D), cache, table, np.clip(lens, 0, cap), np.arange(B + 1) * rows, KG, VG,
                      D ** -0.5, window, sinks)
    _compare(y, z, ref, D, np.ones(B * rows, bool))


@pytest.mark.parametrize("Hq,H,D,page,rows", [(6, 2, 64, 16, 1), (12, 1, 128, 48, 8), (12, 1, 256, 16, 3), (24, 2, 128, 64, 1),
                                              (32, 1, 64, 32, 2), (3, 3, 256, 16, 8)])
@pytest.mark.parametrize("width", [None, 500])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 0), (16, 16), (33, 4), (100, 20), (129, 64), (5000, 3), (64, 5000)])
def test_windows(sk, Hq, H, D, page, rows, width, window, sinks):
    cache, table, lens, q = _case(D + rows, [0, 1, 3, 16, 130, 300, 47], rows, Hq, H, D, page, width=width, q_gap=8)
    _check_window(sk, cache, table, lens, q, rows, Hq, D, window, sinks)


@pytest.mark.parametrize("D,Hq,H,rows,page", [(256, 12, 1, 8, 16), (256, 24, 2, 6, 48), (128, 12, 1, 8, 32), (64, 16, 1, 8, 16)])
@pytest.mark.parametrize("window,sinks", [(40, 4), (7000, 0), (130, 6000)])
def test_windows_of_many_rows(sk, D, Hq, H, rows, page, window, sinks):
    """Rows that take several passes, and tables wide enough for the kernel of chunks; with a narrow window they keep to
    the passes."""
    cache, table, lens, q = _case(D + rows, [0, 1, 5, 16, 130, 260, 47], rows, Hq, H, D, page, width=7500 // page)
    _check_window(sk, cache, table, lens, q, rows, Hq, D, window, sinks)


@pytest.mark.parametrize("D,Hq,H,rows", [(64, 8, 1, 1), (128, 12, 2, 2), (256, 24, 2, 1)])
@pytest.mark.parametrize("window,sinks", [(900, 4), (1300, 700)])
def test_long_windows_in_parts(sk, D, Hq, H, rows, window, sinks):
    cache, table, lens, q = _case(D, [2000, 31, 1100], rows, Hq, H, D, 16, width=200)
    _check_window(sk, cache, table, lens, q, rows, Hq, D, window, sinks)


@pytest.mark.parametrize("D,Hq,H,rows", [(64, 8, 1, 1), (128, 12, 2, 2), (256, 24, 2, 8)])
def test_a_window_as_long_as_the_sequences_is_plain_attention(sk, D, Hq, H, rows):
    """The same kernel's steps over the same positions, so the same bits."""
    import torch

    cache, table, lens, q = _case(D, [300, 0, 65], rows, Hq, H, D, 16)
    a = (dev(q).unflatten(1, (Hq, D)), dev(cache), dev(table), dev(lens), KG, VG, 0.1)
    if rows * Hq // H <= 24:                      # (more rows of head size 128 take another kernel there)
        want = sk.kv4_attention(*a, rows=rows)
        got = sk.kv4_window_attention(*a, 1000, rows=rows)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_window_refusals(sk):
    import torch

    cache, table, lens, q = _case(1, [20], 1, 4, 2, 64, 16)
    a = (dev(q).unflatten(1, (4, 64)), dev(cache), dev(table), dev(lens), KG, VG, 0.1)
    with pytest.raises(sk.SkinnyError):
        sk.kv4_window_attention(*a, 0)
    with pytest.raises(ValueError):
        sk.kv4_window_attention(*a, 5, rows=2)
    with pytest.raises(ValueError):
        sk.kv4_chunk_attention(a[0], a[1], a[2], a[3], torch.zeros(3, dtype=torch.int32, device="cuda:0"), KG, VG, 0.1)
