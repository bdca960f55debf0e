"""GPU parity of the 4-bit cache (kv4_append, kv4_attention, kv4_evict) against
the float64 oracle (oracle/kv4.py).

Tolerances, fixed before the first run.  Codes, scales, kept positions and
copied weights are exact.  For attention, with u = 2^-24:
  * a score is a sum of D exact products in FP32, in D/16 tensor-core steps of
    16: |dz| <= e = (D/16 + 16) 2 u * max_j scale sum_d |q_d k_jd|, plus the
    rounding of the exponent's argument, 4 u max |z| (in e's last term);
  * a weight p is within (2 e + 2^-20) relative, and 2^-11 more when rounded to
    FP16 for the second product; the sums over positions add 2^-16 at most at
    these lengths:  |dout| <= (2^-11 + 4 e + 2^-15) sum_j p_j |v_j|, plus half a
    ulp of the FP16 output (2^-11 |out|, 2^-25 at least);
  * |dlse| <= e + 2^-16 + 2^-22 |lse|;
  * a position's weight, a sum of such p:  (4 e + 2^-15) w + 2^-22 acc + 2^-24.
"""
import numpy as np
import pytest

from gpu_util import Guarded, dev, host
from oracle import kv4

pytestmark = pytest.mark.gpu

KG, VG = 0.02, 0.015


@pytest.fixture(scope="module")
def sk():
    import torch

    torch.cuda.set_device(0)
    import fp8_weight_only_skinny_gb300 as skm

    skm.init()
    yield skm
    assert skm.last_device_error() == skm.SK_OK


# ------------------------------------------------------------------ append ---

@pytest.mark.parametrize("T,H,D,page,gap", [(1, 4, 128, 64, 0), (5, 1, 64, 16, 8), (37, 2, 256, 48, 4096), (16, 8, 64, 32, 64),
                                             (9, 3, 128, 16, 0), (130, 1, 128, 16, 1024)])
@pytest.mark.parametrize("held", [False, True])
def test_append_writes_the_oracles_bytes_and_no_others(sk, T, H, D, page, gap, held):
    import torch

    r = np.random.default_rng(T * 31 + D)
    pages = (T + page - 1) // page + 2
    cache = r.integers(0, 256, (pages, H, page // 16, 18 * D), dtype=np.uint8)
    kv = [r.standard_normal((T, H * D + gap)).astype(np.float16) for _ in range(2)]
    for x in kv:
        x[0, :16] = 0
        x[-1, 16:32] = [0.0, -0.0] * 8
        x[0, 32:48] = 1e-5                      # the scale underflows
        x[T // 2, 48:64] = 60000.0              # and saturates
    slots = r.permutation(pages * page)[:T].astype(np.int32)
    if T > 4:
        slots[2], slots[3] = -1, pages * page + 7          # padding
    g = Guarded(cache.shape, torch.uint8, fill=None)
    g.t.copy_(torch.from_numpy(cache))
    x = [dev(a)[:, :H * D].view(T, H, D) if gap == 0 else dev(a)[:, :H * D].unflatten(1, (H, D)) for a in kv]
    hk = [Guarded((T, H, D), torch.float16) for _ in range(2)] if held else None
    sk.kv4_append(x[0], x[1], dev(slots), g.t, KG, VG, **({"k_held": hk[0].t, "v_held": hk[1].t} if held else {}))
    got = g.host("cache")
    want = cache.copy()
    for t in range(T):
        if 0 <= slots[t] < pages * page:
            for h in range(H):
                kv4.write(want, int(slots[t]), h, kv[0][t, h * D:(h + 1) * D], kv[1][t, h * D:(h + 1) * D], KG, VG)
    assert np.array_equal(got, want)
    if held:
        for a, y, G in zip(kv, hk, (KG, VG)):
            nib, sc = kv4.encode(a[:, :H * D].reshape(T, H, D), G)
            v = kv4.values(nib, sc, 1.0).astype(np.float32) * np.float32(G)       # exact times G, rounded to FP32
            with np.errstate(over="ignore"):
                assert np.array_equal(y.t.cpu().numpy(), v.astype(np.float16))    # and once more to FP16
            y.check("held")


# --------------------------------------------------------------- attention ---

def _case(seed, lens, rows, Hq, H, D, page, width=None, q_gap=0, poison=True, spread=1.5):
    """Random cache of sequences in shuffled pages; bytes of positions that hold nothing are NaN scales (0xFF)."""
    r = np.random.default_rng(seed)
    B = len(lens)
    need = [(n + page - 1) // page for n in lens]
    width = width or max(1, max(need))
    pages = sum(need) + 1
    order = r.permutation(pages)
    table = np.full((B, width), 1 << 30 if not poison else pages + 5, np.int32)      # never read past the length
    cache = np.full((pages, H, page // 16, 18 * D), 0xFF, np.uint8)
    at = 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        for j in range(n):
            for h in range(H):
                kv4.write(cache, int(table[b, j // page]) * page + j % page, h, r.standard_normal(D).astype(np.float16),
                          r.standard_normal(D).astype(np.float16), KG, VG)
    q = (r.standard_normal((B * rows, Hq * D + q_gap)) * spread).astype(np.float16)
    return cache, table, np.array(lens, np.int32), q


def _check_attention(sk, cache, table, lens, q, rows, Hq, D, acc=None, scale=None):
    import torch

    B, H = len(lens), cache.shape[1]
    scale = scale or D ** -0.5
    n = B * rows
    out, lse = Guarded((n, Hq, D), torch.float16), Guarded((n, Hq), torch.float32)
    cap = table.shape[1] * cache.shape[2] * 16
    ao = None
    if acc is not None:
        ao = Guarded((B, H, cap), torch.float32, fill=7.0)
    qd = dev(q)[:, :Hq * D].unflatten(1, (Hq, D))
    c = dev(cache)
    sk.kv4_attention(qd, c, dev(table), dev(lens), KG, VG, scale, rows=rows, out=out.t, lse=lse.t,
                     acc=None if acc is None or acc is False else dev(acc), acc_out=None if ao is None else ao.t)
    real = np.clip(lens, 0, cap)
    ref = kv4.attention(q[:, :Hq * D].reshape(n, Hq, D), cache, table, real, KG, VG, scale, rows)
    u = 2.0 ** -24
    e = ((D / 16 + 16) * 2 * u * ref["zmax"] + 4 * u * np.abs(np.where(np.isfinite(ref["lse"]), ref["lse"], 0)))
    y = out.host("out")
    tol = (2.0 ** -11 + 4 * e[..., None] + 2.0 ** -15) * ref["absum"] + 2.0 ** -11 * np.abs(ref["out"]) + 2.0 ** -25
    assert np.all(np.abs(y - ref["out"]) <= tol), np.max(np.abs(y - ref["out"]) / tol)
    z = lse.host("lse")
    empty = np.isneginf(ref["lse"])
    assert np.array_equal(np.isneginf(z), empty)
    assert np.all(np.abs(z - ref["lse"])[~empty] <= (e + 2.0 ** -16 + 2.0 ** -22 * np.abs(ref["lse"]))[~empty])
    if ao is not None:
        got = ao.host("acc")
        emax = float(e.max()) if e.size else 0.0
        for b in range(B):
            w = ref["weights"][b, :, :real[b]]
            old = 0.0 if acc is False else acc[b, :, :real[b]].astype(np.float64)
            assert np.all(np.abs(got[b, :, :real[b]] - (old + w)) <= (4 * emax + 2.0 ** -15) * w + 2.0 ** -22 * np.abs(old + w)
                          + 2.0 ** -24)
            assert np.all(got[b, :, real[b]:] == 7.0)          # not written past the length
    return y


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [0, 1, 2, 15, 16, 17, 31, 33, 127, 128, 129, 300])
def test_attention_lengths_from_nothing(sk, D, n):
    cache, table, lens, q = _case(n + D, [n], 1, 6, 2, D, 16)
    _check_attention(sk, cache, table, lens, q, 1, 6, D)


@pytest.mark.parametrize("rows", range(1, 9))
@pytest.mark.parametrize("D,Hq,H", [(128, 12, 1), (64, 6, 2), (256, 5, 1)])
def test_attention_rounds_are_causal_and_short_sequences_leave_rows_empty(sk, rows, D, Hq, H):
    lens = [0, 1, 3, rows, 40, 131]
    cache, table, lens, q = _case(rows + D, lens, rows, Hq, H, D, 32, q_gap=64)
    acc = np.random.default_rng(1).random((len(lens), H, table.shape[1] * 32)).astype(np.float32)
    _check_attention(sk, cache, table, lens, q, rows, Hq, D, acc=acc)


@pytest.mark.parametrize("Hq,H,rows", [(1, 1, 1), (8, 8, 1), (16, 1, 1), (17, 1, 1), (24, 1, 2), (20, 1, 8), (40, 2, 8), (33, 1, 5)])
def test_attention_head_groups(sk, Hq, H, rows):
    D = 64
    cache, table, lens, q = _case(Hq * rows, [70, 9], rows, Hq, H, D, 48)
    _check_attention(sk, cache, table, lens, q, rows, Hq, D, acc=False)


@pytest.mark.parametrize("Hq,H,rows", [(33, 1, 1), (17, 1, 2), (12, 1, 4), (48, 1, 1), (10, 1, 5), (16, 1, 4), (16, 1, 5), (12, 1, 7),
                                        (12, 1, 8), (13, 1, 8), (25, 1, 8), (32, 2, 6)])
@pytest.mark.parametrize("lens", [[0, 1, 7, 128], [129, 300, 64, 5]])
def test_attention_of_many_rows_per_kv_head(sk, Hq, H, rows, lens):
    """Head size 128: row counts on both sides of the tensor-core kernel's tiles (48, 64, 80, 96 rows, and two tiles)."""
    cache, table, lens, q = _case(Hq * rows + lens[0], lens, rows, Hq, H, 128, 32, q_gap=128)
    _check_attention(sk, cache, table, lens, q, rows, Hq, 128, acc=False)


@pytest.mark.parametrize("order", ["rising", "falling"])
@pytest.mark.parametrize("Hq,rows", [(12, 1), (12, 3), (12, 8)])
def test_attention_references_move_across_tiles(sk, order, Hq, rows):
    """Head size 128, scores that rise by far more than the slack from tile to tile of one CTA (a batch that gives each
    CTA several tiles of a sequence), or fall as far."""
    import torch

    D, n, page, H = 128, 1100, 64, 2
    r = np.random.default_rng(rows)
    pages = (n + page - 1) // page
    cache = np.full((pages, H, page // 16, 18 * D), 0xFF, np.uint8)
    for j in range(n):
        for h in range(H):
            k = np.full(D, (j if order == "rising" else n - j) / n * 6, np.float16)
            kv4.write(cache, j, h, k, r.standard_normal(D).astype(np.float16), KG, VG)
    B = 70                                         # the same sequence many times: over 1200 tiles
    table = np.tile(np.arange(pages, dtype=np.int32), (B, 1))
    q = (r.random((rows, Hq * H * D)) + 0.5).astype(np.float16)
    lens = np.full(B, n, np.int32)
    ref = kv4.attention(q.reshape(rows, Hq * H, D), cache, table[:1], lens[:1], KG, VG, 0.1, rows)
    out, lse = sk.kv4_attention(dev(np.tile(q, (B, 1))).unflatten(1, (Hq * H, D)), dev(cache), dev(table), dev(lens), KG, VG,
                                0.1, rows=rows)
    out, lse = host(out).reshape(B, rows, Hq * H, D), host(lse).reshape(B, rows, Hq * H)
    e = (D / 16 + 16) * 2.0 ** -23 * ref["zmax"] + 2.0 ** -22 * np.abs(ref["lse"])
    tol = (2.0 ** -11 + 4 * e[..., None] + 2.0 ** -15) * ref["absum"] + 2.0 ** -11 * np.abs(ref["out"]) + 2.0 ** -25
    for b in range(B):
        assert np.all(np.abs(out[b] - ref["out"]) <= tol), b
        assert np.all(np.abs(lse[b] - ref["lse"]) <= e + 2.0 ** -16 + 2.0 ** -22 * np.abs(ref["lse"])), b


@pytest.mark.parametrize("D,Hq,H,rows", [(64, 6, 2, 1), (64, 12, 1, 1), (64, 10, 1, 2), (64, 8, 1, 4), (64, 7, 1, 7),
                                         (128, 4, 2, 2), (128, 12, 1, 1), (128, 12, 1, 2), (128, 5, 1, 5), (128, 12, 1, 3),
                                         (128, 8, 1, 6), (128, 16, 1, 4), (128, 10, 1, 8), (128, 12, 1, 8), (128, 13, 1, 8),
                                         (256, 3, 1, 2), (256, 12, 1, 1), (256, 5, 1, 5)])
@pytest.mark.parametrize("wide", [False, True])
def test_attention_does_not_depend_on_the_tables_width(sk, D, Hq, H, rows, wide):
    """A table of few positions (a cluster per segment, one launch) and one with room for more (shares of all tiles, joined
    in a second launch; many rows of 128 on the tensor cores), over the same sequences."""
    lens = [0, 1, 3, rows, 131, 300, 40, 64]
    cache, table, lens, q = _case(rows + D + Hq, lens, rows, Hq, H, D, 32, width=300 if wide else None, q_gap=64)
    acc = np.random.default_rng(1).random((len(lens), H, table.shape[1] * 32)).astype(np.float32)
    _check_attention(sk, cache, table, lens, q, rows, Hq, D, acc=acc)


@pytest.mark.parametrize("D,Hq,H,rows,lens", [(64, 4, 2, 1, [2000]), (128, 12, 1, 2, [1999, 17]), (256, 8, 1, 1, [1030, 0]),
                                              (128, 12, 1, 8, [700, 1025]), (64, 8, 1, 4, [513, 1, 64, 385]),
                                              (128, 2, 1, 1, [129, 4000]), (64, 4, 1, 1, [7300])])
def test_attention_clusters(sk, D, Hq, H, rows, lens):
    """Segments over clusters of every size, whole and partial tiles, CTAs without positions."""
    cache, table, lens, q = _case(sum(lens), lens, rows, Hq, H, D, 64)
    _check_attention(sk, cache, table, lens, q, rows, Hq, D, acc=False)


@pytest.mark.parametrize("B", [75, 150, 200, 320])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_many_short_sequences(sk, D, B):
    r = np.random.default_rng(B)
    lens = [int(x) for x in r.integers(0, 20, B)]
    lens[5] = 200
    cache, table, lens, q = _case(B, lens, 1, 4, 2, D, 16)
    _check_attention(sk, cache, table, lens, q, 1, 4, D)


@pytest.mark.parametrize("page", [16, 48, 64, 80, 256])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_page_sizes(sk, page, D):
    cache, table, lens, q = _case(page, [page - 1, page, page + 1, 2 * page + 17], 2, 4, 2, D, page)
    _check_attention(sk, cache, table, lens, q, 2, 4, D, acc=False)


@pytest.mark.parametrize("D,Hq,H,rows", [(128, 12, 1, 1), (128, 12, 1, 8), (256, 4, 1, 3), (64, 8, 2, 2)])
def test_attention_many_sequences_over_split_work(sk, D, Hq, H, rows):
    """Lengths that give every CTA parts of several sequences and split the long ones."""
    r = np.random.default_rng(D)
    lens = [int(x) for x in r.integers(0, 90, 61)] + [2000, 0, 515]
    cache, table, lens, q = _case(3, lens, rows, Hq, H, D, 16)
    _check_attention(sk, cache, table, lens, q, rows, Hq, D, acc=False)


@pytest.mark.parametrize("spread", [0.0, 1e-3, 40.0])
@pytest.mark.parametrize("rows", [1, 8])
def test_attention_flat_and_peaked_scores(sk, spread, rows):
    cache, table, lens, q = _case(11, [777], rows, 12, 1, 128, 64, spread=spread)
    _check_attention(sk, cache, table, lens, q, rows, 12, 128, acc=False)


@pytest.mark.parametrize("order", ["rising", "falling"])
@pytest.mark.parametrize("rows", [1, 8])
def test_attention_scores_that_rise_or_fall_with_the_position(sk, order, rows):
    """The running maximum changes at every step, or never after the first."""
    D, n = 64, 400
    r = np.random.default_rng(2)
    cache = np.full((7, 1, 4, 18 * D), 0xFF, np.uint8)
    for j in range(n):
        k = np.full(D, (j if order == "rising" else n - j) / n, np.float16)
        kv4.write(cache, j, 0, k, r.standard_normal(D).astype(np.float16), KG, VG)
    q = np.full((rows, 12 * D), 4.0, np.float16)
    _check_attention(sk, cache, np.arange(7, dtype=np.int32)[None], np.array([n], np.int32), q, rows, 12, D, acc=False,
                     scale=0.5)


def test_attention_lengths_past_the_table_or_negative_are_brought_into_it(sk):
    cache, table, lens, q = _case(5, [64, 64, 20], 1, 4, 1, 64, 32)
    _check_attention(sk, cache, table, np.array([1000, -3, 20], np.int32), q, 1, 4, 64)


def test_attention_nan_scales_count_as_zero_and_infinite_queries_stay_in_their_row(sk):
    import torch

    D, rows = 64, 2
    cache, table, lens, q = _case(9, [50], rows, 4, 1, D, 16)
    at = kv4._where(D, 49 % 16)
    cache[int(table[0, 49 // 16]), 0, 0, at[3]] = 0x7F         # the last position's value scales are NaN
    qd = dev(q).unflatten(1, (4, D))
    out, lse = sk.kv4_attention(qd, dev(cache), dev(table), dev(lens), KG, VG, 0.125, rows=rows)
    zero = cache.copy()
    zero[int(table[0, 49 // 16]), 0, 0, at[3]] = 0
    out2, lse2 = sk.kv4_attention(qd, dev(zero), dev(table), dev(lens), KG, VG, 0.125, rows=rows)
    assert torch.isfinite(out).all() and torch.equal(out, out2) and torch.equal(lse, lse2)
    qd[1, 2, 5] = float("inf")
    out, lse = sk.kv4_attention(qd, dev(cache), dev(table), dev(lens), KG, VG, 0.125, rows=rows)
    assert torch.isfinite(out[0]).all() and torch.isnan(lse[1, 2])


@pytest.mark.parametrize("rows", [1, 8])
def test_attention_records_past_four_gigabytes(sk, rows):
    """A pool of 5 GB whose last pages hold the sequence: byte offsets pass 32 bits."""
    import torch

    D, H, page = 128, 4, 64
    cache, table, lens, q = _case(21, [200], rows, 48, H, D, page)
    pages = (5 << 30) // (H * (page // 16) * 18 * D)
    big = torch.empty((pages, H, page // 16, 18 * D), dtype=torch.uint8, device="cuda:0")
    big[pages - cache.shape[0]:] = dev(cache)
    moved = table + pages - cache.shape[0]
    out, lse = sk.kv4_attention(dev(q).unflatten(1, (48, D)), big, dev(moved.astype(np.int32)), dev(lens), KG, VG, 0.1, rows=rows)
    small, lse2 = sk.kv4_attention(dev(q).unflatten(1, (48, D)), dev(cache), dev(table), dev(lens), KG, VG, 0.1, rows=rows)
    assert torch.equal(out, small) and torch.equal(lse, lse2)
    x = dev(np.random.default_rng(0).standard_normal((1, H, D)).astype(np.float16))
    sk.kv4_append(x, x, torch.tensor([pages * page - 1], dtype=torch.int32, device="cuda:0"), big, KG, VG)
    k, _ = kv4.read(big[-1:].cpu().numpy(), page - 1, 2, KG, VG)
    assert np.abs(k - host(x)[0, 2]).max() < 1.0


@pytest.mark.parametrize("rows,D,Hq,H", [(1, 128, 12, 1), (8, 128, 12, 1), (2, 256, 12, 1)])
def test_attention_is_reproducible_and_independent_of_the_stream(sk, rows, D, Hq, H):
    import torch

    cache, table, lens, q = _case(13, [1500, 3, 700], rows, Hq, H, D, 32)
    a = (dev(q).unflatten(1, (Hq, D)), dev(cache), dev(table), dev(lens), KG, VG, 0.09)
    acc = torch.zeros(3, H, table.shape[1] * 32, device="cuda:0")
    first = [t.clone() for t in sk.kv4_attention(*a, rows=rows, acc_out=acc)] + [acc.clone()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    sk.stream_workspace(s)
    for stream in (None, s, s, None):
        acc2 = torch.zeros_like(acc)
        torch.cuda.synchronize()
        got = [*sk.kv4_attention(*a, rows=rows, acc_out=acc2, stream=stream), acc2]
        torch.cuda.synchronize()
        for x, y in zip(first, got):
            assert torch.equal(x, y)
    assert sk.last_device_error(s) == sk.SK_OK
    sk.stream_workspace(s, 0)


def test_a_captured_decode_step_follows_changing_lengths(sk):
    """append + attention in one graph, replayed as the sequence grows; the weights are accumulated in place."""
    import torch

    D, Hq, H, page = 128, 12, 1, 16
    r = np.random.default_rng(3)
    steps, start = 40, 30
    cache, table, lens, _ = _case(17, [start], 1, Hq, H, D, page, width=6)
    cache = np.concatenate((cache, np.full((4,) + cache.shape[1:], 0xFF, np.uint8)))
    used = (start + page - 1) // page
    table[0, used:] = np.arange(cache.shape[0] - 4, cache.shape[0])[:6 - used]
    c, t, ln = dev(cache), dev(table), dev(lens)
    qkv = torch.zeros(1, (Hq + 2 * H) * D, dtype=torch.float16, device="cuda:0")
    slot = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    acc = torch.zeros(1, H, 6 * page, device="cuda:0")
    out = torch.empty(1, Hq, D, dtype=torch.float16, device="cuda:0")
    lse = torch.empty(1, Hq, device="cuda:0")
    q, k, v = (qkv[:, :Hq * D].view(1, Hq, D), qkv[:, Hq * D:(Hq + H) * D].view(1, H, D), qkv[:, (Hq + H) * D:].view(1, H, D))

    def step():
        sk.kv4_append(k, v, slot, c, KG, VG)
        sk.kv4_attention(q, c, t, ln, KG, VG, 0.1, out=out, lse=lse, acc=acc, acc_out=acc)

    sk.kv4_attention(q, c, t, ln, KG, VG, 0.1, out=out, lse=lse)     # the kernels' attributes are set before the capture
    sk.kv4_append(k, v, torch.full_like(slot, -1), c, KG, VG)
    sk.kv4_attention(q, c, t, ln, KG, VG, 0.1, out=out, lse=lse, acc_out=torch.zeros_like(acc))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    total = np.zeros((1, H, 6 * page))
    for i in range(steps):
        n = start + i
        x = r.standard_normal(qkv.shape).astype(np.float16)
        qkv.copy_(torch.from_numpy(x))
        slot.fill_(int(table[0, n // page]) * page + n % page)
        ln.fill_(n + 1)
        graph.replay()
        torch.cuda.synchronize()
        kv4.write(cache, int(slot[0]), 0, x[0, Hq * D:(Hq + H) * D], x[0, (Hq + H) * D:], KG, VG)
        if i % 13 == 0 or i == steps - 1:
            ref = kv4.attention(x[:, :Hq * D].reshape(1, Hq, D), cache, table, [n + 1], KG, VG, 0.1, 1)
            assert np.abs(host(out) - ref["out"]).max() <= 2.0 ** -9 * np.abs(ref["absum"]).max()
        total += 1.0
    assert np.isclose(host(acc).sum(), steps * Hq, rtol=1e-4)      # every row's weights sum to one


# ------------------------------------------------------------------- evict ---

@pytest.mark.parametrize("lens,budget,recent,H,D,page", [
    ([0, 1, 5, 40], 16, 4, 2, 64, 16), ([100, 33, 64, 65], 33, 0, 1, 128, 32), ([300, 17], 17, 17, 3, 64, 16),
    ([257, 256, 255], 100, 31, 1, 256, 64), ([50], 200, 3, 2, 128, 48), ([5000, 4097, 1], 1000, 10, 1, 64, 16),
    ([3000], 1, 0, 1, 64, 16), ([9000], 2049, 1, 2, 64, 16), ([8193, 8192, 20000], 3000, 100, 1, 64, 16), ([40000], 20000, 0, 1, 64, 32)])
@pytest.mark.parametrize("kind", ["random", "ties", "zeros"])
def test_evict_moves_the_oracles_positions(sk, lens, budget, recent, H, D, page, kind):
    import torch

    r = np.random.default_rng(sum(lens) + budget)
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
    acc = r.random((B, H, width * page)).astype(np.float32)
    if kind == "ties":
        acc = np.floor(acc * 3).astype(np.float32)
    elif kind == "zeros":
        acc[:] = 0
    want, kept, new, acc_out = kv4.evict(cache, table, np.array(lens), acc, dst, budget, recent)
    g = Guarded(cache.shape, torch.uint8, fill=None)
    g.t.copy_(torch.from_numpy(cache))
    ko, no = Guarded(kept.shape, torch.int32, fill=-99), Guarded(new.shape, torch.int32, fill=-99)
    ao = Guarded(acc_out.shape, torch.float32)
    sk.kv4_evict(g.t, dev(table), dev(np.array(lens, np.int32)), dev(acc), dev(dst), budget, recent, kept=ko.t,
                 new_lens=no.t, acc_out=ao.t)
    assert np.array_equal(no.host("new_lens"), new)
    assert np.array_equal(ko.host("kept"), kept)
    assert np.array_equal(ao.host("acc_out"), acc_out)
    assert np.array_equal(g.host("cache"), want)


def test_evicted_cache_serves_attention_over_the_kept_positions(sk):
    """Eviction that drops positions no row attends to leaves the output as it was."""
    import torch

    D, Hq, H, page, n = 64, 4, 1, 16, 120
    r = np.random.default_rng(8)
    cache = np.zeros((16, H, 1, 18 * D), np.uint8)
    hot = np.sort(r.permutation(n)[:25])
    for j in range(n):
        k = np.full(D, 2.0 if j in hot else -2.0, np.float16)
        kv4.write(cache, j, 0, k, r.standard_normal(D).astype(np.float16), KG, VG)
    q = dev(np.full((1, Hq * D), 3.0, np.float16)).unflatten(1, (Hq, D))
    c, table, lens = dev(cache), dev(np.arange(8, dtype=np.int32)[None]), dev(np.array([n], np.int32))
    acc = torch.zeros(1, H, 128, device="cuda:0")
    out, _ = sk.kv4_attention(q, c, table, lens, KG, VG, 0.125, acc=acc, acc_out=acc)
    dst = dev(np.array([[8, 9]], np.int32))
    new, kept, acc2 = sk.kv4_evict(c, table, lens, acc, dst, 25, 0)
    assert np.array_equal(host(kept)[0, 0], hot) and int(new[0]) == 25
    out2, _ = sk.kv4_attention(q, c, dst, new, KG, VG, 0.125, acc=acc2, acc_out=acc2)
    assert np.abs(host(out) - host(out2)).max() <= 2.0 ** -9


def test_example_of_a_decode_round(sk):
    """The example's rounds: its picks are greedy (rank 1, the first alternative), its cache stays within bounds
    through several evictions, and every position holds keys of the sequence's own pages."""
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_round.py")
    spec = importlib.util.spec_from_file_location("decode_round", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    got = example.decode(rounds=120, rows=4, page=16, high_water=64, budget=32, recent=8)
    assert got["evictions"] >= 3 and 0 < got["length"] <= 64
    for token, lp, rank, entropy, ids, top in got["report"]:
        assert rank == 1 and ids[0] == token and abs(top[0] - lp) < 1e-6 and lp < 0 < entropy
    acc = host(got["acc"])[0, :, :got["length"]]
    assert np.all(acc >= 0) and acc.sum() > 0
    k, _ = kv4.read(got["cache"].cpu().numpy(), int(got["table"][0, 0]) * 16, 0, 0.002, 0.002)
    assert np.abs(k).max() > 0


def test_binding_refuses_what_the_library_cannot_see(sk):
    import torch

    c = sk.kv4_cache(4, 2, 128, 32)
    k = torch.zeros(3, 2, 128, dtype=torch.float16, device="cuda:0")
    s = torch.zeros(3, dtype=torch.int32, device="cuda:0")
    with pytest.raises(ValueError):
        sk.kv4_append(k.float(), k, s, c, KG, VG)
    with pytest.raises(ValueError):
        sk.kv4_append(k.transpose(0, 1).contiguous().transpose(0, 1), k, s, c, KG, VG)
    with pytest.raises(ValueError):
        sk.kv4_append(k, k, s.long(), c, KG, VG)
    with pytest.raises(ValueError):
        sk.kv4_append(k, k[:2], s, c, KG, VG)
    with pytest.raises(TypeError):
        sk.kv4_append(k, k, s, c[:, :1], KG, VG)
    with pytest.raises(ValueError):
        sk.kv4_attention(k, c, torch.zeros(2, 2, dtype=torch.int32, device="cuda:0"), s[:2], KG, VG, 0.1)
    with pytest.raises(sk.SkinnyError):
        sk.kv4_attention(k, c, torch.zeros(3, 2, dtype=torch.int32, device="cuda:0"), s, KG, VG, -0.1)
    with pytest.raises(sk.SkinnyError):
        sk.kv4_evict(c, torch.zeros(1, 2, dtype=torch.int32, device="cuda:0"), s[:1], torch.zeros(1, 2, 64, device="cuda:0"),
                     torch.zeros(1, 1, dtype=torch.int32, device="cuda:0"), 33, 0)
    with pytest.raises(ValueError):
        sk.kv4_evict(c, torch.zeros(1, 2, dtype=torch.int32, device="cuda:0"), s[:1], torch.zeros(1, 2, 32, device="cuda:0"),
                     torch.zeros(1, 1, dtype=torch.int32, device="cuda:0"), 16, 0)
