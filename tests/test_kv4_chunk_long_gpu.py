"""kv4_chunk_attention over hundreds of millions of positions: the costs of 32 tiles, by which the work is shared out, pass
31 bits. One page of 2^20 positions stands in the tables of all sequences over and over, so that the result is known: in
the page one key meets the queries (a score of 60, an exact product), the others are zero. What those weigh is
6 10^8 e^-60 < 2^-56 of the rest; so the output is the one position's value and the log sum 60 + log of how often it is seen.

Tolerances: the weights of equal scores are equal, FP32 sums of at most 600 of them in any order are within 600 2^-24 and
weights of a power of two (but for 2^-19 of their exponent's rounding) are not rounded in FP16: 2^-14 of the value; and
half a step of the FP16 output. The log sum is within that, 2^-14, and 2^-22 of itself."""
import math

import numpy as np
import pytest

from gpu_util import Guarded, dev
from oracle import kv4
from test_kv4_chunk_gpu import sk          # noqa: F401
from test_kv4_gpu import VG

pytestmark = pytest.mark.gpu

PAGE, AT = 1 << 20, 12345


@pytest.mark.parametrize("D,times", [(64, 600), (128, 530), (256, 480)])
def test_costs_beyond_31_bits(sk, D, times):       # noqa: F811
    import torch

    r = np.random.default_rng(D)
    cache = torch.zeros(1, 1, PAGE // 16, 18 * D, dtype=torch.uint8, device="cuda:0")
    gen = torch.Generator(device="cuda").manual_seed(D)
    cache[..., 9 * D:17 * D] = torch.randint(0, 256, (PAGE // 16, 8 * D), generator=gen, device="cuda", dtype=torch.uint8)
    cache[..., 17 * D:] = torch.randint(0x20, 0x38, (PAGE // 16, D), generator=gen, device="cuda", dtype=torch.uint8)
    one = np.zeros((1, 1, 1, 18 * D), np.uint8)
    value = r.standard_normal(D).astype(np.float16)
    kv4.write(one, AT % 16, 0, np.full(D, 6.0, np.float16), value, 1.0, VG)
    rec = cache[0, 0, AT // 16].cpu().numpy()
    where = kv4._where(D, AT % 16)
    for part in where:
        rec[part] = one[0, 0, 0][part]
    cache[0, 0, AT // 16] = dev(rec)
    key, want = kv4.read(one, AT % 16, 0, 1.0, VG)
    assert np.all(key == 6.0)

    B = 32
    # the last page of a sequence ends before that key, or behind it
    lens = np.array([times * PAGE - (PAGE - 64 * b if b % 2 else 0) for b in range(B)], np.int64)
    assert sum((n + 63) // 64 * (8 if D == 64 else 9 if D == 128 else 10) for n in lens) >= 1 << 31
    seen = lens // PAGE + (lens % PAGE > AT)
    q = torch.full((B, 1, D), 60.0 / (6 * D), dtype=torch.float16, device="cuda:0")
    assert float(q[0, 0, 0]) * 6 * D == 60.0
    out, lse = Guarded((B, 1, D), torch.float16), Guarded((B, 1), torch.float32)
    sk.kv4_chunk_attention(q, cache, torch.zeros(B, times, dtype=torch.int32, device="cuda:0"), dev(lens.astype(np.int32)),
                           dev(np.arange(B + 1, dtype=np.int32)), 1.0, VG, 1.0, out=out.t, lse=lse.t)
    y, z = out.host("out"), lse.host("lse")
    assert np.all(np.abs(y - want) <= (2.0 ** -14 + 2.0 ** -11) * np.abs(want) + 2.0 ** -25)
    for b in range(B):
        w = 60 + math.log(int(seen[b]))
        assert abs(z[b, 0] - w) <= 2.0 ** -14 + 2.0 ** -22 * w, b
