"""Pins of the rotation oracle (no GPU): closed forms of the rotation, the norm and the frequencies, its codes against
the binary32 steps of kv4_append away from ties, and the library's frequency tables against it."""
import math

import numpy as np
import pytest

import fp8_weight_only_skinny_gb300 as sk
from oracle import kv4, rope

SCALINGS = [("plain", {}), ("linear", dict(factor=4.0)), ("base", dict(factor=2.5)),
            ("turns", dict(factor=8.0, original=8192, low=1.0, high=4.0)), ("index", dict(factor=16.0, original=4096)),
            ("index", dict(factor=4.0, original=32768, low=0.5, high=50.0))]


@pytest.mark.parametrize("scaling,kw", SCALINGS)
@pytest.mark.parametrize("rot,base", [(16, 10000.0), (64, 1e6), (128, 500000.0), (256, 10000.0)])
def test_frequency_tables(scaling, kw, rot, base):
    got = sk.rope_frequencies(rot, base, scaling, device="cpu", **kw).numpy()
    want = rope.frequencies(rot, base, scaling, **kw) / (2 * math.pi) * 2.0 ** 64
    assert got.dtype == np.int64 and got.shape == (rot // 2,)
    # pow, log and a few products in double precision, then cut to a whole number
    assert np.all(np.abs(got.astype(np.float64) - want) <= 2.0 ** -46 * want + 1)


def test_scaled_frequencies_lie_between_plain_and_divided():
    plain = rope.frequencies(128, 10000.0)
    for scaling, kw in SCALINGS[3:]:
        f = rope.frequencies(128, 10000.0, scaling, **kw)
        assert np.all(f <= plain * (1 + 1e-12)) and np.all(f >= plain / kw["factor"] * (1 - 1e-12))
        assert f[0] == plain[0] and f[-1] == pytest.approx(plain[-1] / kw["factor"])


def test_a_quarter_turn_exchanges_the_pair():
    quarter = np.array([1 << 62] * 8, np.int64)
    x = np.arange(64, dtype=np.float16).reshape(1, 1, 64)
    for interleaved in (False, True):
        y, _ = rope.turned(x, [1], quarter, None, 0.0, 1.0, interleaved)
        a, b = (np.arange(0, 16, 2), np.arange(1, 16, 2)) if interleaved else (np.arange(8), np.arange(8, 16))
        assert np.allclose(y[0, 0, a], -x[0, 0, b].astype(float), atol=1e-14)
        assert np.allclose(y[0, 0, b], x[0, 0, a].astype(float), atol=1e-14)
        assert np.array_equal(y[0, 0, 16:], x[0, 0, 16:].astype(float))


@pytest.mark.parametrize("far", [0, 1000, 2 ** 31 - 60])
def test_products_depend_on_the_distance_alone(far):
    r = np.random.default_rng(0)
    f = sk.rope_frequencies(64, 10000.0, device="cpu").numpy()
    q, k = (r.standard_normal((1, 1, 64)).astype(np.float16) for _ in range(2))
    near = [(rope.turned(q, [7 + d], f, None, 0, 1.0, False)[0] * rope.turned(k, [d], f, None, 0, 1.0, False)[0]).sum()
            for d in (0, far)]
    assert near[0] == pytest.approx(near[1], abs=1e-9)


def test_norm():
    x = np.full((1, 1, 64), 3.0, np.float16)
    y, _ = rope.turned(x, [0], np.zeros(0, np.int64), np.full(64, 2.0, np.float32), 0.0, 1.0, False)
    assert np.allclose(y, 2.0, atol=1e-15)


def test_codes_are_those_of_the_rounded_steps_away_from_ties():
    """kv4_append's steps round a quotient to binary32 up to three times, 2^-24 of it each: where the exact one is
    further than 2^-22 from every border between two codes, both give the same code."""
    from oracle.quant import _E2M1_POS, _E4M3_POS

    def clear(q, table):
        border = (table[0][1:] + table[0][:-1]) / 2
        return np.all(np.abs(np.abs(q)[..., None] - border) > 2.0 ** -22 * border, -1)

    r = np.random.default_rng(1)
    w = r.standard_normal((200, 128)).astype(np.float16)
    G = float(np.float32(0.02))
    nib, sc = rope.encode(w.astype(np.float64), 0.02)
    nib2, sc2 = kv4.encode(w, 0.02)
    blocks = w.astype(np.float64).reshape(200, 8, 16)
    sure = clear(np.abs(blocks).max(-1) / (6 * G), _E4M3_POS)
    assert sure.mean() > 0.99 and np.array_equal(sc[sure], sc2[sure])
    unit = np.array([kv4.values(np.full((1, 16), 2), np.full((1, 1), c), 0.02)[0, 0] for c in sc.ravel()]).reshape(200, 8, 1)
    same = clear(blocks / unit, _E2M1_POS) & (sc == sc2)[..., None]
    assert same.mean() > 0.98 and np.array_equal(nib.reshape(blocks.shape)[same], nib2.reshape(blocks.shape)[same])


def test_chunks_of_rows_reproduce_the_round_form():
    r = np.random.default_rng(2)
    cache = r.integers(0, 0x70, (3, 2, 1, 18 * 64), dtype=np.uint8)
    table, lens = np.array([[2, 0, 1]], np.int32), np.array([37])
    q = r.standard_normal((4, 6, 64)).astype(np.float16)
    a = kv4.attention(q, cache, table, lens, 0.01, 0.01, 0.1, 4)
    b = rope.chunks(q, cache, table, lens, [0, 4], 0.01, 0.01, 0.1)
    for name in ("out", "lse", "absum", "zmax"):
        assert np.allclose(a[name], b[name], rtol=1e-12)
    c = rope.chunks(q, cache, table, lens, [0, 4], 0.01, 0.01, 0.1, window=64, sinks=2)
    assert np.allclose(b["out"], c["out"])
