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
