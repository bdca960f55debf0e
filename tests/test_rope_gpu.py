"""GPU parity of the rotation and of the rotated append (qk_norm_rope, kv4_append_rope) against the float64 oracle
(oracle/rope.py).

Tolerances, fixed before the first run.  With u = 2^-24 and a component made of two terms whose magnitudes, cosine and
sine taken as one, sum to `size`:  in FP32 the norm's factor is off by 11.5 u (a sum of 13 roundings and eps's two,
halved by the root, and rsqrt's two last places), an angle's cosine by 4.2 u, amplitude, weights, products and sum add
6 u: |dy| <= 24 u size, and half a step of the FP16 output: 2^-11 |y|, 2^-25 at least.  Key codes are those of exact
arithmetic and value codes kv4_append's: the cache is compared byte by byte.
"""
import numpy as np
import pytest

from gpu_util import Guarded, dev, host
from oracle import rope

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


def _inputs(seed, T, Hq, H, D, gap=0, norm=True, far=100000):
    """q, k and v as parts of one row of a projection's output, positions and weights."""
    r = np.random.default_rng(seed)
    x = (r.standard_normal((T, (Hq + 2 * H) * D + gap)) * np.where(r.random((Hq + 2 * H) * D + gap) < 0.05, 5, 1)).astype(np.float16)
    pos = r.integers(0, far + 1, T).astype(np.int32)
    w = [(1 + 0.2 * r.standard_normal(D)).astype(np.float32) for _ in range(2)] if norm else [None, None]
    return x, pos, w


def _parts(x, Hq, H, D):
    cut = [x[:, lo * D:hi * D] for lo, hi in ((0, Hq), (Hq, Hq + H), (Hq + H, Hq + 2 * H))]
    return [c.reshape(len(x), -1, D) if isinstance(x, np.ndarray) else c.unflatten(1, (-1, D)) for c in cut]


def _near(got, want, size, what):
    tol = 24 * 2.0 ** -24 * size + 2.0 ** -11 * np.abs(want) + 2.0 ** -25
    assert np.all(np.abs(got - want) <= tol), (what, np.max(np.abs(got - want) / tol))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("T,Hq,H,D,rot,gap", [(1, 24, 2, 256, 64, 0), (5, 7, 1, 64, 64, 8), (33, 3, 3, 128, 128, 0),
                                              (9, 12, 4, 64, 16, 64), (700, 5, 1, 128, 96, 0), (130, 2, 1, 256, 256, 8),
                                              (3, 1, 1, 64, 48, 0), (2, 9, 2, 128, 0, 0)])
def test_rotation(sk, T, Hq, H, D, rot, gap, norm, interleaved):
    import torch

    x, pos, w = _inputs(T * 7 + D, T, Hq, H, D, gap, norm)
    f = sk.rope_frequencies(rot, 1e6)
    amp = 1.21
    q, k, _ = _parts(dev(x), Hq, H, D)
    qo, ko = Guarded((T, Hq, D), torch.float16), Guarded((T, H, D), torch.float16)
    wd = [None if a is None else dev(a) for a in w]
    sk.qk_norm_rope(q, k, dev(pos), f, *wd, eps=1e-6, interleaved=interleaved, amplitude=amp, q_out=qo.t, k_out=ko.t)
    for a, out, wt in zip(_parts(x, Hq, H, D), (qo, ko), w):
        want, size = rope.turned(a, pos, f.cpu().numpy(), wt, 1e-6, amp, interleaved)
        _near(out.host(), want, size, (T, D))


@pytest.mark.parametrize("positions", [[0], [-1], [2 ** 31 - 1], [-2 ** 31], [1000003, 1000002, 0, 5]])
def test_far_and_negative_positions(sk, positions):
    T, Hq, H, D = len(positions), 2, 1, 128
    x, _, _ = _inputs(3, T, Hq, H, D)
    pos, f = np.array(positions, np.int32), sk.rope_frequencies(128, 10000.0)
    q, k, _ = _parts(dev(x), Hq, H, D)
    qo, ko = sk.qk_norm_rope(q, k, dev(pos), f)
    for a, out in zip(_parts(x, Hq, H, D), (qo, ko)):
        want, size = rope.turned(a, pos, f.cpu().numpy(), None, 0, 1.0, False)
        _near(host(out), want, size, positions)


@pytest.mark.parametrize("D,rot,interleaved", [(64, 64, False), (128, 32, True), (256, 128, False)])
def test_in_place(sk, D, rot, interleaved):
    """q_out and k_out that are q and k, within the projection's rows: the values beside them stay."""
    import torch

    T, Hq, H = 41, 6, 2
    x, pos, w = _inputs(D, T, Hq, H, D, 8)
    f, xd = sk.rope_frequencies(rot, 1e4), dev(x)
    q, k, v = _parts(xd, Hq, H, D)
    wd = [dev(a) for a in w]
    want = [t.clone() for t in sk.qk_norm_rope(q, k, dev(pos), f, *wd, interleaved=interleaved)]
    sk.qk_norm_rope(q, k, dev(pos), f, *wd, interleaved=interleaved, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert np.array_equal(xd[:, (Hq + H) * D:].cpu().numpy(), x[:, (Hq + H) * D:])


def test_a_head_of_zeros_and_the_smallest_numbers(sk):
    import torch

    x = np.zeros((3, 4, 64), np.float16)
    x[1] = 2.0 ** -24
    x[2, :, ::2] = -0.0
    w = torch.ones(64, device="cuda:0")
    f, pos = sk.rope_frequencies(64), np.array([0, 3, 9], np.int32)
    qo, _ = sk.qk_norm_rope(dev(x), dev(x), dev(pos), f, w, w, eps=1e-6)
    want, size = rope.turned(x, pos, f.cpu().numpy(), np.ones(64, np.float32), 1e-6, 1.0, False)
    _near(host(qo), want, size, "small")
    assert np.all(host(qo)[0] == 0)


# ------------------------------------------------------------------ append ---

def _check_append(sk, x, pos, w, Hq, H, D, rot, page, interleaved, amp=1.0, kG=KG, vG=VG, slots=None, eps=1e-6):
    import torch

    T = len(x)
    r = np.random.default_rng(T + D)
    pages = (T + page - 1) // page + 2
    cache = r.integers(0, 256, (pages, H, page // 16, 18 * D), dtype=np.uint8)
    if slots is None:
        slots = r.permutation(pages * page)[:T].astype(np.int32)
        if T > 4:
            slots[2], slots[3] = -1, pages * page + 7
    g, qo = Guarded(cache.shape, torch.uint8, fill=None), Guarded((T, Hq, D), torch.float16)
    g.t.copy_(torch.from_numpy(cache))
    q, k, v = _parts(dev(x), Hq, H, D)
    f = sk.rope_frequencies(rot, 1e6)
    wd = [None if a is None else dev(a) for a in w]
    sk.kv4_append_rope(q, k, v, dev(slots), dev(pos), f, g.t, kG, vG, *wd, eps=eps, interleaved=interleaved, amplitude=amp,
                       q_out=qo.t)
    xq, xk, xv = _parts(x, Hq, H, D)
    fq = f.cpu().numpy()
    want, size = rope.turned(xq, pos, fq, w[0], eps, amp, interleaved)
    _near(qo.host(), want, size, "q")
    key, _ = rope.turned(xk, pos, fq, w[1], eps, amp, interleaved)
    full = cache.copy()
    for t in range(T):
        if 0 <= slots[t] < pages * page:
            for h in range(H):
                rope.write(full, int(slots[t]), h, key[t, h], xv[t, h], kG, vG)
    got = g.host("cache")
    assert np.array_equal(got, full), np.argwhere(got != full)[:5]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("T,Hq,H,D,rot,page,gap", [(1, 24, 2, 256, 64, 64, 0), (5, 7, 1, 64, 64, 16, 8),
                                                   (37, 3, 3, 128, 128, 48, 0), (16, 4, 8, 64, 16, 32, 64),
                                                   (300, 2, 2, 256, 256, 16, 0), (65, 1, 5, 128, 0, 16, 8)])
def test_append_writes_the_oracles_bytes_and_no_others(sk, T, Hq, H, D, rot, page, gap, norm, interleaved):
    x, pos, w = _inputs(T * 5 + D, T, Hq, H, D, gap, norm)
    _check_append(sk, x, pos, w, Hq, H, D, rot, page, interleaved, amp=1.0 if T % 2 else 1.208)


@pytest.mark.parametrize("D,rot", [(64, 64), (128, 64), (256, 256)])
def test_codes_next_to_borders(sk, D, rot):
    """Thousands of keys: about one component in 10^5 lies so near a border that 32 bits leave its code open, and every
    one of them has to come out as in exact arithmetic."""
    T, Hq, H = 4000, 1, 2
    x, pos, w = _inputs(D, T, Hq, H, D)
    _check_append(sk, x, pos, w, Hq, H, D, rot, 64, False)


@pytest.mark.parametrize("kG", [2.0 ** -6, 1.0, 1e-4, 1e-19, 1e19])
def test_ties_saturation_and_vanishing_scales(sk, kG):
    """Keys that are not turned keep their ties under a scale that is a power of two; others saturate or vanish."""
    T, Hq, H, D = 40, 1, 1, 64
    r = np.random.default_rng(5)
    x = (r.integers(-24, 25, (T, 3 * D)) * 2.0 ** -4).astype(np.float16)
    x[3] = 0.0
    x[4] = -0.0
    x[5, ::3] = 60000.0
    x[6] = 6e-8
    _check_append(sk, x, np.zeros(T, np.int32), [None, None], Hq, H, D, 0, 16, False, kG=kG)
    _check_append(sk, x, np.arange(T, dtype=np.int32), [None, None], Hq, H, D, 64, 16, True, kG=kG)


def test_append_agrees_with_the_two_calls(sk):
    """The rotated queries are qk_norm_rope's bit for bit, the values kv4_append's."""
    import torch

    T, Hq, H, D, page = 50, 8, 2, 128, 32
    x, pos, w = _inputs(11, T, Hq, H, D)
    q, k, v = _parts(dev(x), Hq, H, D)
    f, wd = sk.rope_frequencies(128), [dev(a) for a in w]
    slots = dev(np.arange(T, dtype=np.int32))
    a, b = sk.kv4_cache(2, H, D, page), sk.kv4_cache(2, H, D, page)
    got = sk.kv4_append_rope(q, k, v, slots, dev(pos), f, a, KG, VG, *wd)
    want, _ = sk.qk_norm_rope(q, k, dev(pos), f, *wd)
    assert torch.equal(got, want)
    sk.kv4_append(k, v, slots, b, KG, VG)
    assert torch.equal(a[..., 9 * D:], b[..., 9 * D:])


def test_captured_and_on_another_stream(sk):
    import torch

    T, Hq, H, D, page = 20, 4, 1, 64, 16
    x, pos, w = _inputs(4, T, Hq, H, D)
    xd, pd = dev(x), dev(pos)
    q, k, v = _parts(xd, Hq, H, D)
    f, wd = sk.rope_frequencies(64), [dev(a) for a in w]
    slots, cache = dev(np.arange(T, dtype=np.int32)), sk.kv4_cache(2, H, D, page)
    qo = torch.empty(T, Hq, D, dtype=torch.float16, device="cuda:0")
    call = lambda **kw: sk.kv4_append_rope(q, k, v, slots, pd, f, cache, KG, VG, *wd, q_out=qo, **kw)      # noqa: E731
    call()
    want = [qo.clone(), cache.clone()]
    stream = torch.cuda.Stream()
    cache.zero_()
    torch.cuda.synchronize()
    call(stream=stream)
    stream.synchronize()
    assert torch.equal(qo, want[0]) and torch.equal(cache, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    pd.add_(5)
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(qo, want[0])
    pd.sub_(5)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(qo, want[0]) and torch.equal(cache, want[1])


def test_no_tokens_and_refused_shapes(sk):
    import torch

    z = lambda *s: torch.zeros(*s, dtype=torch.float16, device="cuda:0")      # noqa: E731
    f, cache = sk.rope_frequencies(64), sk.kv4_cache(1, 2, 64, 16)
    none = torch.zeros(0, dtype=torch.int32, device="cuda:0")
    assert sk.qk_norm_rope(z(0, 4, 64), z(0, 2, 64), none, f)[0].shape == (0, 4, 64)
    sk.kv4_append_rope(z(0, 4, 64), z(0, 2, 64), z(0, 2, 64), none, none, f, cache, KG, VG)
    one = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    with pytest.raises(ValueError):
        sk.qk_norm_rope(z(2, 4, 64), z(1, 2, 64), one, f)
    with pytest.raises(ValueError):
        sk.qk_norm_rope(z(1, 4, 64), z(1, 2, 64), one.long(), f)
    with pytest.raises(ValueError):
        sk.kv4_append_rope(z(1, 4, 64), z(1, 3, 64), z(1, 2, 64), one, one, f, cache, KG, VG)
    with pytest.raises(sk.SkinnyError):
        sk.qk_norm_rope(z(1, 4, 64), z(1, 2, 64), one, f, eps=-1.0)
