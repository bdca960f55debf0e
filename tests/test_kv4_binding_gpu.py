"""Strides that the binding hands on: a single row has no row stride, whatever its tensor says."""
import numpy as np
import pytest

from gpu_util import dev, host
from oracle import kv4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pitch", [4, 8, 3, 0])
@pytest.mark.parametrize("Hq,H,D", [(6, 2, 64), (4, 1, 128)])
def test_one_row_of_any_pitch(pitch, Hq, H, D):
    import torch

    import fp8_weight_only_skinny_gb300 as sk

    torch.cuda.set_device(0)
    sk.init()
    r = np.random.default_rng(pitch)
    k, v, q = (r.standard_normal((1, h * D + pitch)).astype(np.float16) for h in (H, H, Hq))
    views = [dev(x).as_strided((1, h, D), (h * D + pitch, D, 1)) for x, h in ((k, H), (v, H), (q, Hq))]
    cache = sk.kv4_cache(1, H, D, 16)
    slot = dev(np.array([0], np.int32))
    sk.kv4_append(views[0], views[1], slot, cache, 0.02, 0.02)
    want = np.zeros((1, H, 1, 18 * D), np.uint8)
    for h in range(H):
        kv4.write(want, 0, h, k[0, h * D:(h + 1) * D], v[0, h * D:(h + 1) * D], 0.02, 0.02)
    assert np.array_equal(host(cache), want)
    out, _ = sk.kv4_attention(views[2], cache, dev(np.zeros((1, 1), np.int32)), dev(np.array([1], np.int32)), 0.02, 0.02, 0.1)
    for x in range(Hq):                                     # one position has all the weight: its value, to half a ulp
        y = kv4.read(want, 0, x * H // Hq, 0.02, 0.02)[1]
        assert np.all(np.abs(host(out)[0, x] - y) <= 2.0 ** -11 * np.abs(y) + 2.0 ** -25)
