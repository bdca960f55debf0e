"""Pins of the cache and log-probability oracle (no GPU): the record layout is
a permutation, codes round-trip, and attention, eviction and log probabilities
reproduce closed forms."""
import numpy as np
import pytest

from oracle import kv4


@pytest.mark.parametrize("D", [64, 128, 256])
def test_record_offsets_are_a_permutation_of_the_record(D):
    seen = np.concatenate([np.concatenate(kv4._where(D, i)) for i in range(16)])
    assert np.array_equal(np.sort(seen), np.arange(18 * D))


@pytest.mark.parametrize("D,page", [(64, 16), (128, 48)])
def test_write_then_read_returns_representable_values_exactly(D, page):
    r = np.random.default_rng(D)
    cache = r.integers(0, 255, (3, 2, page // 16, 18 * D), dtype=np.uint8)
    grid = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.5, -1, -6])
    slot, head = page + page - 3, 1
    want = []
    before = cache.copy()
    for _ in range(2):
        x = r.choice(grid, D)
        x[::16] = 6.0                                   # every block's scale is then 1 / G = 2, a power of two
        want.append(x.astype(np.float16))
    kv4.write(cache, slot, head, want[0], want[1], 0.5, 0.25)
    k, v = kv4.read(cache, slot, head, 0.5, 0.25)
    assert np.array_equal(k, want[0].astype(np.float64)) and np.array_equal(v, want[1].astype(np.float64))
    assert (cache != before).sum() <= 2 * (D // 2 + D // 16)
    other = before[:, 0]
    assert np.array_equal(cache[:, 0], other)           # the other head is untouched


def test_encode_rounds_to_nearest_even_and_saturates():
    w = np.zeros(16, np.float16)
    w[:8] = [6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    w[8:12] = [-0.0, -0.2, -5.5, 0.3]
    nib, sc = kv4.encode(w, 1.0)
    assert sc[0] == 0x38                                # 1.0
    assert list(nib[:12]) == [7, 0, 2, 2, 4, 4, 6, 6, 8, 8, 15, 1]
    nib, sc = kv4.encode(np.full(16, 60000.0, np.float16), 1e-3)
    assert sc[0] == 0x7E and (nib == 7).all()           # 448 and 6: the largest a block can hold
    nib, sc = kv4.encode(np.full(16, -1e-4, np.float16), 1.0)
    assert sc[0] == 0 and (nib == 8).all()


def test_attention_of_equal_keys_is_the_mean_of_the_seen_values():
    D, page = 64, 16
    r = np.random.default_rng(5)
    cache = np.zeros((2, 1, 1, 18 * D), np.uint8)
    for j in range(20):
        kv4.write(cache, j, 0, np.ones(D, np.float16), r.standard_normal(D).astype(np.float16), 0.01, 0.01)
    table = np.array([[0, 1]])
    q = np.ones((3, 2, D), np.float16)
    got = kv4.attention(q, cache, table, [20], 0.01, 0.01, 0.125, 3)
    _, v = kv4.sequence(cache, table[0], 20, 0, 0.01, 0.01)
    for m in range(3):
        assert np.allclose(got["out"][m], v[:18 + m].mean(0), atol=1e-12)
    assert np.allclose(got["weights"][0, 0, :18].sum() + got["weights"][0, 0, 18:].sum(), 6.0)
    empty = kv4.attention(q, cache, table, [1], 0.01, 0.01, 0.125, 3)
    assert (empty["out"][:2] == 0).all() and np.isneginf(empty["lse"][:2]).all()


def test_keep_prefers_weight_then_the_lower_position_and_protects_the_recent():
    acc = np.array([1.0, 3.0, 1.0, 0.0, 3.0, 0.0, 0.0])
    assert list(kv4.keep(acc, 7, 4, 2)) == [1, 4, 5, 6]
    assert list(kv4.keep(acc, 7, 3, 0)) == [0, 1, 4]
    assert list(kv4.keep(acc, 7, 2, 2)) == [5, 6]
    assert list(kv4.keep(acc, 3, 4, 2)) == [0, 1, 2]


def test_logprobs_of_a_uniform_and_a_masked_row():
    z = np.full(8, 2.0)
    lp, rank, ent, ids, top = kv4.logprobs(z, 3, 0.7, 3)
    assert np.isclose(lp, -np.log(8)) and rank == 4 and np.isclose(ent, np.log(8)) and list(ids) == [0, 1, 2]
    z[4:] = -np.inf
    lp, rank, ent, ids, top = kv4.logprobs(z, 5, 1.0, 10)
    assert np.isneginf(lp) and rank == 6 and np.isclose(ent, np.log(4)) and ids[8] == -1
    lp, rank, ent, _, _ = kv4.logprobs(np.full(4, -np.inf), 2, 1.0, 2)
    assert np.isneginf(lp) and rank == 3 and ent == 0.0
