"""Refusals of the rotating, chunk and window entry points (no GPU needed): each returns its status before anything
could be launched, on fake pointers that are never dereferenced."""
import ctypes

import pytest

import fp8_weight_only_skinny_gb300 as sk

OK, INVALID, UNSUPPORTED, MISALIGNED = 0, 1, 2, 3
A = 0x10000


def _freqs(rot=64, kind=0, base=1e4, factor=1.0, original=0.0, low=1.0, high=32.0, out=True):
    room = (ctypes.c_uint64 * 256)()
    return sk.lib.rope_frequencies(ctypes.addressof(room) if out else None, rot, kind, base, factor, original, low, high)


def _rope(q=A, qs=6144, k=A, ks=512, pos=A, f=A, qw=None, kw=None, eps=1e-6, amp=1.0, qo=A, qos=6144, ko=A, kos=512, T=1,
          Hq=48, H=4, D=128, R=128, inter=0):
    return sk.lib.qk_norm_rope(q, qs, k, ks, pos, f, qw, kw, eps, amp, qo, qos, ko, kos, T, Hq, H, D, R, inter, None)


def _append(q=A, qs=6144, k=A, ks=512, v=A, vs=512, slots=A, pos=A, f=A, qw=None, kw=None, eps=1e-6, amp=1.0, qo=A,
            qos=6144, cache=A, kg=0.02, vg=0.02, T=1, pages=4, Hq=48, H=4, D=128, page=64, R=128, inter=0):
    return sk.lib.kv4_append_rope(q, qs, k, ks, v, vs, slots, pos, f, qw, kw, eps, amp, qo, qos, cache, kg, vg, T, pages, Hq,
                                  H, D, page, R, inter, None)


def _chunk(q=A, qs=6144, cache=A, table=A, lens=A, starts=A, kg=0.02, vg=0.02, scale=0.1, window=0, sinks=0, out=A, lse=A,
           rows=3, B=1, Hq=48, H=4, D=128, pages=4, page=64, width=2):
    return sk.lib.kv4_chunk_attention(q, qs, cache, table, lens, starts, kg, vg, scale, window, sinks, out, lse, rows, B, Hq,
                                      H, D, pages, page, width, None)


def _window(q=A, qs=6144, cache=A, table=A, lens=A, kg=0.02, vg=0.02, scale=0.1, window=5, sinks=0, out=A, lse=A, B=1, M=1,
            Hq=48, H=4, D=128, pages=4, page=64, width=2):
    return sk.lib.kv4_window_attention(q, qs, cache, table, lens, kg, vg, scale, window, sinks, out, lse, B, M, Hq, H, D,
                                       pages, page, width, None)


def test_frequencies():
    assert _freqs() == OK and _freqs(rot=0) == OK and _freqs(kind=2, factor=2.0) == OK
    assert _freqs(out=False) == INVALID and _freqs(rot=-2) == INVALID and _freqs(rot=63) == INVALID
    assert _freqs(kind=5) == INVALID and _freqs(kind=-1) == INVALID
    for bad in (1.0, 0.0, -5.0, 1e13, float("nan"), float("inf")):
        assert _freqs(base=bad) == INVALID
    for bad in (0.5, 0.0, -1.0, 1e7, float("nan")):
        assert _freqs(kind=1, factor=bad) == INVALID
        assert _freqs(factor=bad) == OK                       # not read
    assert _freqs(kind=2, rot=2, factor=2.0) == INVALID
    for kind in (3, 4):
        assert _freqs(kind=kind, factor=8.0, original=4096.0) == OK
        assert _freqs(kind=kind, factor=8.0) == INVALID
        assert _freqs(kind=kind, factor=8.0, original=4096.0, low=4.0, high=4.0) == INVALID
        assert _freqs(kind=kind, factor=8.0, original=4096.0, low=0.0) == INVALID


@pytest.mark.parametrize("D,R", [(96, 64), (512, 64), (0, 0), (128, 144), (64, 128), (128, 8), (128, 40)])
def test_head_and_rotated_sizes(D, R):
    assert _rope(D=D, R=R) == UNSUPPORTED and _append(D=D, R=R) == UNSUPPORTED


def test_rotating_sizes_and_numbers():
    for call in (_rope, _append):
        assert call(T=-1) == INVALID and call(Hq=0) == INVALID and call(H=0) == INVALID and call(R=-16) == INVALID
        assert call(inter=2) == INVALID and call(inter=-1) == INVALID
        assert call(Hq=5000, qs=640000, qos=640000) == UNSUPPORTED
        for eps in (-1e-9, 1.5, float("nan")):
            assert call(eps=eps) == INVALID
        for amp in (0.0, 1e-4, 2e3, float("nan"), float("inf")):
            assert call(amp=amp) == INVALID
        assert call(qw=A) == INVALID and call(kw=A) == INVALID            # both weights or neither
        assert call(T=0) == OK
    for g in (0.0, -1.0, 1e-30, float("inf"), float("nan")):
        assert _append(kg=g) == INVALID and _append(vg=g) == INVALID
    assert _append(pages=0) == INVALID and _append(page=40) == UNSUPPORTED and _append(pages=1 << 30, page=16) == UNSUPPORTED


def test_rotating_pointers():
    for name in ("q", "k", "qo", "ko", "pos", "f"):
        assert _rope(**{name: None}) == INVALID
    for name in ("q", "k", "v", "qo", "slots", "cache", "pos", "f"):
        assert _append(**{name: None}) == INVALID
    for call in (_rope, _append):
        assert call(qs=6136) == INVALID and call(qs=6148) == MISALIGNED and call(ks=504) == INVALID and call(ks=516) == MISALIGNED
        assert call(qos=6136) == INVALID and call(qos=6148) == MISALIGNED
        assert call(q=A + 8) == MISALIGNED and call(qo=A + 4) == MISALIGNED and call(f=A + 4) == MISALIGNED
        assert call(pos=A + 2) == MISALIGNED and call(qw=A + 2, kw=A) == MISALIGNED
    assert _rope(kos=504) == INVALID and _rope(ko=A + 8) == MISALIGNED
    assert _append(vs=516) == MISALIGNED and _append(v=A + 8) == MISALIGNED and _append(cache=A + 8) == MISALIGNED
    assert _append(slots=A + 1) == MISALIGNED


@pytest.mark.parametrize("call", [_chunk, _window])
def test_attention_sizes_and_pointers(call):
    assert call(B=-1) == INVALID and call(width=0) == INVALID and call(Hq=50) == INVALID and call(pages=0) == INVALID
    assert call(D=96) == UNSUPPORTED and call(page=40) == UNSUPPORTED
    assert call(sinks=-1) == INVALID and call(window=-1) == INVALID
    for g in (0.0, -1.0, 1e-30, float("inf"), float("nan")):
        assert call(kg=g) == INVALID and call(vg=g) == INVALID
    assert call(scale=0.0) == INVALID and call(scale=1e19, kg=1e10) == INVALID and call(scale=1e-37, kg=1.0) == INVALID
    for name in ("q", "cache", "table", "lens", "out"):
        assert call(**{name: None}) == INVALID
    assert call(qs=6136) == INVALID and call(qs=6148) == MISALIGNED and call(q=A + 2) == MISALIGNED
    assert call(out=A + 8) == MISALIGNED and call(lse=A + 1) == MISALIGNED and call(table=A + 2) == MISALIGNED
    assert call(lens=A + 1) == MISALIGNED and call(cache=A + 4) == MISALIGNED
    assert call(B=0) == OK


def test_chunks_alone():
    assert _chunk(rows=-1) == INVALID and _chunk(starts=None) == INVALID and _chunk(starts=A + 2) == MISALIGNED
    assert _chunk(rows=0) == OK
    assert _chunk(B=16384) == UNSUPPORTED
    assert _chunk(rows=1 << 29) == UNSUPPORTED                # rows of a kv head's list
    assert _chunk(width=1 << 26) == UNSUPPORTED               # positions
    assert _window(window=0) == INVALID and _window(M=0) == INVALID and _window(M=9) == INVALID


def test_binding_checks():
    with pytest.raises(ValueError):
        sk.rope_frequencies(64, scaling="none", device="cpu")
    with pytest.raises(sk.SkinnyError):
        sk.rope_frequencies(64, base=0.5, device="cpu")
    assert sk.rope_frequencies(0, device="cpu").numel() == 0
