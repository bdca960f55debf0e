"""How near the log probabilities come, for rows of which a thread adds few terms.

Bound, derived before the first run.  With d = (z - max) log2 e / T, a term 2^d is off by |d| 1.5 2^-23 ln 2 (the rounded
factor, difference and product) and 2^-22 (the exponential) relative; weighed with the terms themselves that is below
20 2^-23 for the distributions here (the mean of |d| is below 19).  A thread adds at most 128 terms, and 16 joins follow:
144 2^-24.  The logarithm adds 2^-21.  So ln S is within 2^-16.8 + 2^-18.6 + 2^-21 < 2^-16, and a log probability within
2^-16 + 2^-21 |lp| (the difference, its factor 1 / T and their product)."""
import numpy as np
import pytest

from gpu_util import dev, host
from oracle import kv4

pytestmark = pytest.mark.gpu


# rows x logits: 64 threads a row; clusters of 16 with 512 and 256 threads; clusters of 8 and of 4
@pytest.mark.parametrize("M,N", [(5, 1000), (700, 1500), (1, 151936), (8, 32000), (40, 100003), (100, 50021)])
@pytest.mark.parametrize("dtype", [np.float32, np.float16])
@pytest.mark.parametrize("T", [1.0, 0.6, 1.7])
def test_error_of_log_probabilities(M, N, dtype, T):
    import torch

    import fp8_weight_only_skinny_gb300 as sk

    torch.cuda.set_device(0)
    sk.init()
    r = np.random.default_rng(M + N)
    z = (r.standard_normal((M, N), dtype=np.float32) * 2.2).astype(dtype)
    z[:, ::17] = -np.inf
    tok = r.integers(0, N, M)
    lp, _, _, ids, top = sk.token_logprobs(dev(z), dev(tok.astype(np.int32)), top_n=5, temperature=T)
    lp, ids, top = host(lp), host(ids), host(top)
    for m in range(0, M, max(1, M // 40)):
        want, _, _, wi, wt = kv4.logprobs(z[m], int(tok[m]), T, 5)
        assert lp[m] == want or abs(lp[m] - want) <= 2.0 ** -16 + 2.0 ** -21 * abs(want), (m, lp[m], want)
        assert np.array_equal(ids[m], wi)
        assert np.all(np.abs(top[m] - wt) <= 2.0 ** -16 + 2.0 ** -21 * np.abs(wt)), (m, top[m], wt)
