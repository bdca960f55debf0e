"""Limits of the cache and log-probability entry points beyond which a call is refused before anything is launched
(no GPU needed): fake pointers that are never dereferenced."""
import pytest

import fp8_weight_only_skinny_gb300 as sk

INVALID, UNSUPPORTED = 1, 2
A = 0x10000


def _lp(N, rows=1, f16=0):
    return sk.lib.token_logprobs(A, f16, N, A, 1.0, 0, A, A, A, None, None, rows, N, None)


@pytest.mark.parametrize("N", [0x7FFF0001, 0x7FFFE000, 0x7FFFFFF0, 0x7FFFFFFF])
@pytest.mark.parametrize("f16", [0, 1])
def test_rows_of_logits_too_long_for_the_rounds_indices(N, f16):
    """A round's indices run up to two rounds of 8192 past the row's end and have to stay within 31 bits."""
    assert _lp(N, f16=f16) == UNSUPPORTED
    assert _lp(N, rows=0, f16=f16) == UNSUPPORTED
    assert _lp(0x7FFF0000, rows=0, f16=f16) == 0


def _attn(scale, kg, B=1):
    return sk.lib.kv4_attention(A, 6144, A, A, A, kg, 0.02, scale, A, A, None, None, B, 1, 48, 4, 128, 4, 64, 2, None)


@pytest.mark.parametrize("scale,kg", [(1e-30, 1e-20), (1e-24, 1e-20), (1e-18, 1e-20), (1e-37, 0.02), (1e-37, 4.0), (1e19, 1e20), (1e8, 1e20),
                                      (9e19, 2e7)])
def test_scale_times_key_scale_out_of_range(scale, kg):
    """Their product, by which scores are multiplied and the softmax's slack divided, is neither lost nor infinite, nor
    is it times the largest score (256 components of 65504 times 2688)."""
    assert _attn(scale, kg) == INVALID
    assert _attn(scale, kg, B=0) == INVALID


@pytest.mark.parametrize("scale,kg", [(0.1, 0.02), (1e-16, 1e-20), (1e6, 1e20), (1e-30, 1e-6), (1e-36, 1.0), (9e19, 1e7)])
def test_scale_times_key_scale_in_range(scale, kg):
    assert _attn(scale, kg, B=0) == 0
