"""Refusals of the cache and log-probability entry points (no GPU needed): each
returns its status before anything could be launched, on fake pointers that are
never dereferenced."""
import pytest

import fp8_weight_only_skinny_gb300 as sk

OK, INVALID, UNSUPPORTED, MISALIGNED = 0, 1, 2, 3
A = 0x10000


def _append(k=A, ks=512, v=A, vs=512, slots=A, cache=A, kg=0.02, vg=0.02, hk=None, hv=None, T=0, pages=4, H=4, D=128,
            page=64):
    return sk.lib.kv4_append(k, ks, v, vs, slots, cache, kg, vg, hk, hv, T, pages, H, D, page, None)


def _attn(q=A, qs=6144, cache=A, table=A, lens=A, kg=0.02, vg=0.02, scale=0.1, out=A, lse=A, ai=None, ao=None, B=1, M=1,
          Hq=48, H=4, D=128, pages=4, page=64, width=2):
    return sk.lib.kv4_attention(q, qs, cache, table, lens, kg, vg, scale, out, lse, ai, ao, B, M, Hq, H, D, pages, page,
                                width, None)


def _evict(cache=A, table=A, lens=A, acc=A, dst=A, kept=A, new=A + 64, ao=None, B=1, budget=64, recent=8, H=4, D=128, pages=9,
           page=64, width=4, dwidth=1):
    return sk.lib.kv4_evict(cache, table, lens, acc, dst, kept, new, ao, B, budget, recent, H, D, pages, page, width,
                            dwidth, None)


def _lp(z=A, f16=0, stride=100, tok=A, T=1.0, n=0, lp=A, rank=A, ent=A, ids=None, top=None, rows=1, N=100):
    return sk.lib.token_logprobs(z, f16, stride, tok, T, n, lp, rank, ent, ids, top, rows, N, None)


@pytest.mark.parametrize("D", [0, 16, 96, 512])
def test_head_sizes_outside_the_three(D):
    assert _append(D=D, T=1) == UNSUPPORTED
    assert _attn(D=D) == UNSUPPORTED
    assert _evict(D=D) == UNSUPPORTED


@pytest.mark.parametrize("page", [8, 24, 100])
def test_pages_hold_whole_records(page):
    assert _append(page=page, T=1) == UNSUPPORTED
    assert _attn(page=page) == UNSUPPORTED
    assert _evict(page=page, budget=4, recent=0) == UNSUPPORTED


def test_sizes_out_of_range():
    assert _append(T=-1) == INVALID and _append(H=0) == INVALID and _append(pages=0) == INVALID
    assert _append(pages=1 << 30, page=16) == UNSUPPORTED
    assert _attn(M=0) == INVALID and _attn(M=9) == INVALID and _attn(B=-1) == INVALID and _attn(width=0) == INVALID
    assert _attn(Hq=50) == INVALID
    assert _attn(B=40000) == UNSUPPORTED                      # more than 131072 row tiles
    assert _evict(budget=0, recent=0) == INVALID and _evict(recent=65) == INVALID and _evict(recent=-1) == INVALID
    assert _evict(budget=65) == INVALID                       # past the destination pages
    assert _lp(N=0) == INVALID and _lp(rows=-1) == INVALID and _lp(stride=99) == INVALID and _lp(f16=2) == INVALID
    assert _lp(n=-1) == INVALID and _lp(n=65, ids=A, top=A) == UNSUPPORTED


@pytest.mark.parametrize("g", [0.0, -1.0, 1e-30, float("inf"), float("nan")])
def test_scales_outside_their_range(g):
    assert _append(kg=g, T=1) == INVALID and _append(vg=g, T=1) == INVALID
    assert _attn(kg=g) == INVALID and _attn(vg=g) == INVALID
    assert _attn(scale=-abs(g) if g == 1e-30 else g) == INVALID
    assert _lp(T=-1.0 if g == 1e-30 else g) == INVALID


def test_null_pointers():
    assert _append(T=1, k=None) == INVALID and _append(T=1, slots=None) == INVALID and _append(T=1, cache=None) == INVALID
    assert _append(T=1, hk=A) == INVALID                      # both held outputs or neither
    for name in ("q", "cache", "table", "lens", "out"):
        assert _attn(**{name: None}) == INVALID
    assert _attn(ao=A, lse=None) == INVALID                   # the weights need the log sums
    assert _attn(ai=A) == INVALID
    for name in ("cache", "table", "lens", "acc", "dst", "kept", "new"):
        assert _evict(**{name: None}) == INVALID
    assert _evict(ao=A) == INVALID                            # acc_out is acc
    assert _evict(new=A) == INVALID                           # new_lens is lens
    assert _lp(z=None) == INVALID and _lp(tok=None) == INVALID and _lp(n=3) == INVALID


def test_strides_and_alignment():
    assert _append(T=1, ks=504) == INVALID and _append(T=1, ks=516) == MISALIGNED and _append(T=1, v=A + 8) == MISALIGNED
    assert _append(T=1, slots=A + 2) == MISALIGNED and _append(T=1, cache=A + 4) == MISALIGNED
    assert _attn(qs=6136) == INVALID and _attn(qs=6148) == MISALIGNED and _attn(q=A + 2) == MISALIGNED
    assert _attn(lse=A + 1) == MISALIGNED and _attn(out=A + 8) == MISALIGNED and _attn(table=A + 1) == MISALIGNED
    assert _evict(acc=A + 2) == MISALIGNED and _evict(kept=A + 1) == MISALIGNED
    assert _lp(z=A + 2) == MISALIGNED and _lp(z=A + 1, f16=1) == MISALIGNED and _lp(ent=A + 2) == MISALIGNED


def test_nothing_to_do():
    assert _append(T=0) == OK
    assert _attn(B=0) == OK
    assert _evict(B=0) == OK
    assert _lp(rows=0) == OK


def test_cache_allocation_checks_its_sizes():
    with pytest.raises(ValueError):
        sk.kv4_cache(4, 2, 128, 40, device="cpu")
    with pytest.raises(ValueError):
        sk.kv4_cache(4, 2, 96, 64, device="cpu")
    assert tuple(sk.kv4_cache(3, 2, 128, 64, device="cpu").shape) == (3, 2, 4, 18 * 128)
