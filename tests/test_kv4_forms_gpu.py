"""The attention's long-table forms (shares of all tiles joined in a second launch; the tensor cores for many rows) on the
inputs where they can go wrong.  A table with room for far more positions than the sequences hold keeps the one-launch form
for short tables out; tolerances are those of test_kv4_gpu.py."""
import numpy as np
import pytest

from gpu_util import dev, host
from oracle import kv4
from test_kv4_gpu import KG, VG, _case, _check_attention

pytestmark = pytest.mark.gpu

WIDE = 300                             # pages of 32 and 64: more than a cluster's 16 x 4 x 128 positions


@pytest.fixture(scope="module")
def sk():
    import torch

    torch.cuda.set_device(0)
    import fp8_weight_only_skinny_gb300 as skm

    skm.init()
    yield skm
    assert skm.last_device_error() == skm.SK_OK


# (rows, query heads of one kv head): 28, 36, 60, 77, 96 rows in tensor-core tiles of 32, 48, 64, 80, 96, and 104 and 200
# rows in two and three tiles
MANY = [(1, 28), (3, 12), (6, 10), (7, 11), (8, 12), (8, 13), (8, 25)]


@pytest.mark.parametrize("rows,G", MANY)
@pytest.mark.parametrize("lens", [[0, 1, 7, 128], [129, 300, 64, 5]])
def test_many_rows_per_kv_head(sk, rows, G, lens):
    cache, table, lens, q = _case(G * rows + lens[0], lens, rows, 2 * G, 2, 128, 32, width=WIDE, q_gap=128)
    _check_attention(sk, cache, table, lens, q, rows, 2 * G, 128, acc=False)


@pytest.mark.parametrize("order", ["rising", "falling"])
@pytest.mark.parametrize("rows,G", MANY)
def test_bases_move_across_the_tiles_of_a_cta(sk, order, rows, G):
    """Scores that rise by far more than the slack from tile to tile, or fall as far, in enough copies of a sequence that
    every CTA takes several tiles in turn: its ring wraps, sums and outputs are rescaled, segments end inside its share."""
    D, n, page, H = 128, 1100, 64, 2
    r = np.random.default_rng(rows)
    pages = (n + page - 1) // page
    cache = np.full((pages, H, page // 16, 18 * D), 0xFF, np.uint8)
    for j in range(n):
        for h in range(H):
            k = np.full(D, (j if order == "rising" else n - j) / n * 6, np.float16)
            kv4.write(cache, j, h, k, r.standard_normal(D).astype(np.float16), KG, VG)
    B = 70
    table = np.tile(np.arange(pages, dtype=np.int32), (B, 1))
    q = (r.random((rows, G * H * D)) + 0.5).astype(np.float16)
    lens = np.full(B, n, np.int32)
    ref = kv4.attention(q.reshape(rows, G * H, D), cache, table[:1], lens[:1], KG, VG, 0.1, rows)
    out, lse = sk.kv4_attention(dev(np.tile(q, (B, 1))).unflatten(1, (G * H, D)), dev(cache), dev(table), dev(lens), KG, VG,
                                0.1, rows=rows)
    out, lse = host(out).reshape(B, rows, G * H, D), host(lse).reshape(B, rows, G * H)
    e = (D / 16 + 16) * 2.0 ** -23 * ref["zmax"] + 2.0 ** -22 * np.abs(ref["lse"])
    tol = (2.0 ** -11 + 4 * e[..., None] + 2.0 ** -15) * ref["absum"] + 2.0 ** -11 * np.abs(ref["out"]) + 2.0 ** -25
    for b in range(B):
        assert np.all(np.abs(out[b] - ref["out"]) <= tol), b
        assert np.all(np.abs(lse[b] - ref["lse"]) <= e + 2.0 ** -16 + 2.0 ** -22 * np.abs(ref["lse"])), b


FORMS = [(64, 6, 2, 1), (64, 8, 1, 8), (128, 12, 1, 1), (128, 12, 1, 2), (128, 12, 1, 8), (128, 13, 1, 8), (256, 12, 1, 1),
         (256, 12, 1, 2)]


@pytest.mark.parametrize("spread", [0.0, 1e-3, 40.0])
@pytest.mark.parametrize("D,Hq,H,rows", FORMS)
def test_flat_and_peaked_scores(sk, spread, D, Hq, H, rows):
    cache, table, lens, q = _case(11, [777, 20], rows, Hq, H, D, 64, width=WIDE, spread=spread)
    _check_attention(sk, cache, table, lens, q, rows, Hq, D, acc=False)


@pytest.mark.parametrize("D,Hq,H,rows", FORMS)
def test_lengths_past_the_table_or_negative(sk, D, Hq, H, rows):
    """Copies of a sequence that fills its table and of an empty one, more than the short tables' form takes."""
    n = 1120
    cache, table, lens, q = _case(5, [n], rows, Hq, H, D, 32)
    B = 200
    table, q = np.tile(table, (B, 1)), np.tile(q, (B, 1))
    given = np.where(np.arange(B) % 2, 5000, -3).astype(np.int32)
    out, lse = sk.kv4_attention(dev(q).unflatten(1, (Hq, D)), dev(cache), dev(table), dev(given), KG, VG, 0.1, rows=rows)
    ref = kv4.attention(q[:rows].reshape(rows, Hq, D), cache, table[:1], [n], KG, VG, 0.1, rows)
    out, lse = host(out).reshape(B, rows, Hq, D), host(lse).reshape(B, rows, Hq)
    assert np.all(out[0::2] == 0) and np.all(np.isneginf(lse[0::2]))
    e = (D / 16 + 16) * 2.0 ** -23 * ref["zmax"] + 2.0 ** -22 * np.abs(ref["lse"])
    tol = (2.0 ** -11 + 4 * e[..., None] + 2.0 ** -15) * ref["absum"] + 2.0 ** -11 * np.abs(ref["out"]) + 2.0 ** -25
    assert np.all(np.abs(out[1::2] - ref["out"]) <= tol)
    assert np.all(np.abs(lse[1::2] - ref["lse"]) <= e + 2.0 ** -16 + 2.0 ** -22 * np.abs(ref["lse"]))


@pytest.mark.parametrize("D,Hq,H,rows", FORMS)
def test_nan_scales_count_as_zero_and_infinite_queries_stay_in_their_row(sk, D, Hq, H, rows):
    import torch

    cache, table, lens, q = _case(9, [150], rows, Hq, H, D, 32, width=WIDE)
    at = kv4._where(D, 149 % 16)
    rec = int(table[0, 149 // 32]), 0, 149 % 32 // 16
    cache[rec][at[3]] = 0x7F                              # the last position's value scales are NaN
    a = dev(q).unflatten(1, (Hq, D)), dev(table), dev(lens)
    out, lse = sk.kv4_attention(a[0], dev(cache), a[1], a[2], KG, VG, 0.125, rows=rows)
    zero = cache.copy()
    zero[rec][at[3]] = 0
    out2, lse2 = sk.kv4_attention(a[0], dev(zero), a[1], a[2], KG, VG, 0.125, rows=rows)
    assert torch.isfinite(out).all() and torch.equal(out, out2) and torch.equal(lse, lse2)
    a[0][rows - 1, Hq - 1, 5] = float("inf")
    out, lse = sk.kv4_attention(a[0], dev(zero), a[1], a[2], KG, VG, 0.125, rows=rows)
    assert torch.isnan(lse[rows - 1, Hq - 1]) and torch.isnan(out[rows - 1, Hq - 1]).all()
    keep = torch.ones(rows, Hq, dtype=torch.bool, device="cuda:0")
    keep[rows - 1, Hq - 1] = False
    # the other rows' bases may move with it: both within the bound of a call, so twice that from each other
    absum = dev(kv4.attention(q.reshape(rows, Hq, D), zero, table, lens, KG, VG, 0.125, rows)["absum"])
    assert torch.all((out.double() - out2.double()).abs()[keep] <= 2.0 ** -8 * absum[keep] + 2.0 ** -24)
    assert torch.all((lse - lse2).abs()[keep] <= 2.0 ** -11)


@pytest.mark.parametrize("D,Hq,H,rows", [(64, 8, 4, 1), (128, 48, 4, 1), (128, 48, 4, 8), (256, 24, 2, 2)])
def test_records_past_four_gigabytes(sk, D, Hq, H, rows):
    """A pool of 5 GB whose last pages hold the sequence: byte offsets pass 32 bits, in the second pass for the weights too."""
    import torch

    page = 64
    cache, table, lens, q = _case(21, [200], rows, Hq, H, D, page, width=WIDE)
    pages = (5 << 30) // (H * (page // 16) * 18 * D)
    big = torch.empty((pages, H, page // 16, 18 * D), dtype=torch.uint8, device="cuda:0")
    big[pages - cache.shape[0]:] = dev(cache)
    moved = np.where(table < cache.shape[0], table + pages - cache.shape[0], 0).astype(np.int32)
    acc = [torch.zeros(1, H, WIDE * page, device="cuda:0") for _ in range(2)]
    a = dev(q).unflatten(1, (Hq, D))
    out, lse = sk.kv4_attention(a, big, dev(moved), dev(lens), KG, VG, 0.1, rows=rows, acc_out=acc[0])
    small, lse2 = sk.kv4_attention(a, dev(cache), dev(table), dev(lens), KG, VG, 0.1, rows=rows, acc_out=acc[1])
    assert torch.equal(out, small) and torch.equal(lse, lse2) and torch.equal(*acc)
    assert abs(float(acc[0].sum()) - rows * Hq) <= 2.0 ** -13 * rows * Hq


@pytest.mark.parametrize("D,Hq,H,rows", FORMS)
def test_reproducible_on_any_stream_and_workspace(sk, D, Hq, H, rows):
    """Bitwise the same on the device's workspace, on a stream's own, and after other calls have used the scratch memory."""
    import torch

    cache, table, lens, q = _case(13, [1500, 3, 0, 700], rows, Hq, H, D, 32, width=WIDE)
    a = (dev(q).unflatten(1, (Hq, D)), dev(cache), dev(table), dev(lens), KG, VG, 0.09)
    other = _case(14, [300, 900], 1, 12, 2, 64, 32, width=WIDE)
    o = (dev(other[3]).unflatten(1, (12, 64)), dev(other[0]), dev(other[1]), dev(other[2]), KG, VG, 0.1)
    acc = torch.zeros(4, H, WIDE * 32, device="cuda:0")
    first = [t.clone() for t in sk.kv4_attention(*a, rows=rows, acc_out=acc)] + [acc.clone()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    sk.stream_workspace(s, 1 << 20)
    try:
        for stream in (None, s, s, None):
            for _ in range(3):
                acc2 = torch.zeros_like(acc)
                torch.cuda.synchronize()
                sk.kv4_attention(*o, acc_out=torch.zeros(2, 2, WIDE * 32, device="cuda:0"), stream=stream)
                got = [*sk.kv4_attention(*a, rows=rows, acc_out=acc2, stream=stream), acc2]
                torch.cuda.synchronize()
                for x, y in zip(first, got):
                    assert torch.equal(x, y)
        assert sk.last_device_error(s) == sk.SK_OK
    finally:
        sk.stream_workspace(s, 0)


def test_streams_with_workspaces_of_their_own_overlap(sk):
    """Long forms on two streams at the same time, with no synchronisation between their calls."""
    import torch

    cases = []
    for seed, (D, Hq, H, rows) in enumerate([(128, 12, 1, 8), (256, 12, 1, 1)]):
        cache, table, lens, q = _case(seed, [1500, 9, 700], rows, Hq, H, D, 32, width=WIDE)
        cases.append(((dev(q).unflatten(1, (Hq, D)), dev(cache), dev(table), dev(lens), KG, VG, 0.09), rows, H))
    want = [[x.clone() for x in sk.kv4_attention(*a, rows=rows)] for a, rows, _ in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for s in streams:
        sk.stream_workspace(s, 1 << 20)
    try:
        outs = [[(torch.empty_like(w[0]), torch.empty_like(w[1])) for _ in range(20)] for w in want]
        torch.cuda.synchronize()
        for i in range(20):
            for (a, rows, _), s, o in zip(cases, streams, outs):
                sk.kv4_attention(*a, rows=rows, out=o[i][0], lse=o[i][1], stream=s)
        torch.cuda.synchronize()
        for w, o in zip(want, outs):
            assert all(torch.equal(w[0], x) and torch.equal(w[1], y) for x, y in o)
        assert all(sk.last_device_error(s) == sk.SK_OK for s in streams)
    finally:
        for s in streams:
            sk.stream_workspace(s, 0)


@pytest.mark.parametrize("D,Hq,H,rows", FORMS)
def test_a_captured_call_of_several_kernels_follows_changing_lengths(sk, D, Hq, H, rows):
    """Append, attention, join and weights in one graph, replayed for lengths that move the shares and their joins."""
    import torch

    page, most = 32, 900
    cache, table, _, q = _case(19, [most, 0], rows, Hq, H, D, page, width=WIDE)
    table[1] = table[0]                                   # two sequences over the same pages
    r = np.random.default_rng(1)
    kv = r.standard_normal((1, H, D)).astype(np.float16)
    c, t, ln = dev(cache), dev(table), torch.zeros(2, dtype=torch.int32, device="cuda:0")
    a, slot = dev(q).unflatten(1, (Hq, D)), torch.full((1,), -1, dtype=torch.int32, device="cuda:0")
    x = dev(kv)
    acc = torch.zeros(2, H, WIDE * page, device="cuda:0")
    out, lse = torch.empty_like(a), torch.empty(2 * rows, Hq, device="cuda:0")

    def step():
        sk.kv4_append(x, x, slot, c, KG, VG)
        sk.kv4_attention(a, c, t, ln, KG, VG, 0.1, rows=rows, out=out, lse=lse, acc_out=acc)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n0, n1 in ((0, 0), (most, 0), (1, most), (rows, 129), (640, 641), (0, 5)):
        ln.copy_(torch.tensor([n0, n1], dtype=torch.int32))
        slot.fill_(int(table[0, 0]) * page + 3)
        acc.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        for h in range(H):
            kv4.write(cache, int(table[0, 0]) * page + 3, h, kv[0, h], kv[0, h], KG, VG)
        ref = kv4.attention(q.reshape(2 * rows, Hq, D), cache, table, [n0, n1], KG, VG, 0.1, rows)
        assert np.all(np.abs(host(out) - ref["out"]) <= 2.0 ** -9 * ref["absum"] + 2.0 ** -20)
        assert np.array_equal(np.isneginf(host(lse)), np.isneginf(ref["lse"]))
        got = host(acc)
        for b, n in enumerate((n0, n1)):
            assert np.all(np.abs(got[b, :, :n] - ref["weights"][b, :, :n]) <= 2.0 ** -10 * ref["weights"][b, :, :n] + 2.0 ** -20)
            assert np.all(got[b, :, n:] == 7.0)


@pytest.mark.parametrize("D,Hq,H", [(64, 32, 4), (128, 48, 4), (256, 24, 2)])
@pytest.mark.parametrize("lens", [[900], [130, 2100]])
def test_verify_rounds_whose_rows_are_joined_one_a_cta(sk, D, Hq, H, lens):
    """Eight rows of grouped heads over few sequences: more rows than SMs, each of many parts."""
    cache, table, lens, q = _case(D + lens[0], lens, 8, Hq, H, D, 32, width=WIDE)
    acc = np.random.default_rng(1).random((len(lens), H, WIDE * 32)).astype(np.float32)
    _check_attention(sk, cache, table, lens, q, 8, Hq, D, acc=acc)


# -------------------------------------------------------------- evict forms ---

def _evict(sk, lens, budget, recent, H, D, page, kind):
    """One call against the oracle: every byte of the cache, every kept position and copied weight."""
    import torch

    r = np.random.default_rng(sum(lens) + budget + D)
    B = len(lens)
    need = [(n + page - 1) // page for n in lens]
    width, per = max(1, max(need)), (budget + page - 1) // page
    pages = sum(need) + B * per + 1
    order = r.permutation(pages).astype(np.int32)
    table = np.full((B, width), -7, np.int32)
    at = 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    dst = order[at:at + B * per].reshape(B, per)
    cache = r.integers(0, 256, (pages, H, page // 16, 18 * D), dtype=np.uint8)
    acc = r.random((B, H, width * page), dtype=np.float32)
    if kind == "ties":
        acc = np.floor(acc * 3).astype(np.float32)
    elif kind == "zeros":
        acc[:] = 0
    elif kind == "signed":
        acc -= np.float32(0.5)
        acc[..., ::5] = -0.0
        acc[..., 1::5] = 0.0
        acc[..., 7::11] = np.inf
        acc[..., 8::11] = -np.inf
    want, kept, new, acc_out = kv4.evict(cache, table, np.array(lens), acc, dst, budget, recent)
    c = dev(cache)
    got = sk.kv4_evict(c, dev(table), dev(np.array(lens, np.int32)), dev(acc), dev(dst), budget, recent)
    torch.cuda.synchronize()
    assert np.array_equal(got[0].cpu().numpy(), new) and np.array_equal(got[1].cpu().numpy(), kept)
    assert np.array_equal(got[2].cpu().numpy(), acc_out) and np.array_equal(c.cpu().numpy(), want)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens,budget,recent", [([9000, 300], 700, 30), ([8193, 20000, 0], 1500, 0), ([33000], 900, 900)])
@pytest.mark.parametrize("kind", ["random", "ties", "zeros", "signed"])
def test_evict_in_clusters_at_every_head_size(sk, D, lens, budget, recent, kind):
    _evict(sk, lens, budget, recent, 1, D, 32, kind)


@pytest.mark.parametrize("seqs,H", [(160, 1), (50, 2), (39, 2)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", ["random", "ties", "zeros"])
def test_evict_of_more_positions_a_cta_than_it_keeps_keys_and_records_for(sk, seqs, H, D, kind):
    """One CTA a head, two, and two again for fewer heads: parts of 16,000 positions and more, past the 8192 keys in shared
    memory and the 1024 records numbered at a time."""
    r = np.random.default_rng(seqs)
    lens = [int(x) for x in r.integers(0, 60, seqs)]
    lens[seqs // 2] = 34000
    _evict(sk, lens, 1300 if D == 64 else 40, 17, H, D, 16, kind)


@pytest.mark.parametrize("kind", ["random", "ties", "signed"])
def test_evict_that_keeps_nearly_all_of_a_long_part(sk, kind):
    lens = [3] * 159 + [20000]
    _evict(sk, lens, 19000, 100, 1, 64, 16, kind)
