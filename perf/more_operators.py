"""Cases and plain forms of what stands between the fused qkv projection and the attention over the cache
held in 4 bits, and of that attention for chunks of new tokens and for windows.

    rope         norms of the query and key heads and their rotation by position, in FP16
    append_rope  the same, with the keys and values written to the cache's records
    chunk        a chunk of new tokens per sequence (any number, none among them) over the paged cache
    window       1..8 query rows per sequence that see the last positions and a few first ones

Each case is run in its plain form (elementary torch operations in 32 bits; keys on their way into 4 bits,
where a code is next to a border, and angles in 64) or, with `own` set, through the package's entry points.

The cache is u8 [pages][kv_heads][page_size / 16][18 D], one record of 18 D bytes per 16 positions
(D the head size): key codes [16][D/2], key scales [16][D/16], value codes [2][D/16][8][8] (half of
the positions, block of 16 components, position, byte), value scales [D/16][16].  Codes are E2M1,
low nibble first; scales are E4M3, one per 16 components of a position; one FP32 scale for all keys
and one for all values.

Frequencies are held as fractions of a turn per position in units of 2^-64: the angle of a position is the product
of two whole numbers modulo one turn, at any distance.
"""
import math

import numpy as np
import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
KG, VG, EPS = 0.02, 0.015, 1e-6


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # one decode token on its way from the projection to the cache: the smallest call of a decode step
        dict(name="append_rope_token", op="append_rope", tokens=1, q_heads=24, kv_heads=2, dim=256, rot=64, page=64,
             norm=True, interleaved=False, scaling="plain", far=100003),
        # 37 requests' speculative rounds of 8 rows, at far positions of a context that was lengthened
        dict(name="append_rope_rounds", op="append_rope", tokens=296, q_heads=48, kv_heads=4, dim=128, rot=128, page=32,
             norm=False, interleaved=False, scaling="turns", far=900001),
        # a long prompt
        dict(name="append_rope_prompt", op="append_rope", tokens=16387, q_heads=24, kv_heads=2, dim=256, rot=64, page=64,
             norm=True, interleaved=False, scaling="index", far=0),
        # a few rows of a small drafting model, whose cache is its own
        dict(name="rope_rows", op="rope", tokens=7, q_heads=28, kv_heads=4, dim=64, rot=64, norm=False, interleaved=True,
             scaling="base", far=5003),
        # a prompt whose keys and values are attended to before they are compressed
        dict(name="rope_prompt", op="rope", tokens=8191, q_heads=32, kv_heads=8, dim=128, rot=128, norm=True,
             interleaved=True, scaling="linear", far=0),
        # a prompt's attention over itself
        dict(name="chunk_prompt", op="chunk", seqs=1, most=4099, longest=4099, ragged=False, q_heads=24, kv_heads=2,
             dim=256, page=64, window=0, sinks=0),
        # the next piece of a long document, behind what is in the cache
        dict(name="chunk_long", op="chunk", seqs=1, most=2048, longest=61003, ragged=False, q_heads=24, kv_heads=2,
             dim=256, page=64, window=0, sinks=0),
        # a user's short turn at the end of a long conversation
        dict(name="chunk_turn", op="chunk", seqs=1, most=24, longest=100003, ragged=False, q_heads=48, kv_heads=4,
             dim=128, page=64, window=0, sinks=0),
        # a server's step over requests of mixed lengths, some with one new token, some with none
        dict(name="chunk_batch", op="chunk", seqs=23, most=333, longest=9001, ragged=True, q_heads=28, kv_heads=4,
             dim=64, page=16, window=0, sinks=0),
        # a prompt in a layer that keeps a window and the first few tokens
        dict(name="chunk_window", op="chunk", seqs=1, most=8195, longest=8195, ragged=False, q_heads=48, kv_heads=4,
             dim=128, page=64, window=1024, sinks=4),
        # one token of such a layer late in a conversation
        dict(name="window_token", op="window", seqs=1, rows=1, longest=100003, ragged=False, q_heads=48, kv_heads=4,
             dim=128, page=64, window=4096, sinks=4),
        # a server's decode step in such a layer
        dict(name="window_batch", op="window", seqs=64, rows=2, longest=16411, ragged=True, q_heads=24, kv_heads=2,
             dim=256, page=64, window=2000, sinks=20),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = ((48, 4, 128), (24, 2, 256), (28, 4, 64), (32, 8, 128), (8, 4, 128), (12, 4, 64), (16, 2, 256), (10, 1, 128))
SCALINGS = ("plain", "linear", "base", "turns", "index")


def draw(rng):
    op = rng.choice(("append_rope", "rope", "chunk", "chunk", "window"))
    hq, hkv, d = rng.choice(HEADS)
    page = rng.choice((16, 32, 64, 128, 48))
    if op in ("append_rope", "rope"):
        rot = rng.choice((d, d, d // 2, d // 4))
        c = dict(op=op, tokens=_log(rng, 1, 16387 * 24 * 256 // (hq * d)), q_heads=hq, kv_heads=hkv, dim=d, rot=rot,
                 norm=rng.random() < 0.5, interleaved=rng.random() < 0.5, scaling=rng.choice(SCALINGS),
                 far=rng.choice((0, 1, 5003, 100003, 900001)))
        return dict(c, page=page) if op == "append_rope" else c
    window = _log(rng, 1, 4096) if op == "window" or rng.random() < 0.4 else 0
    sinks = rng.choice((0, 1, 4, 20, 64)) if window else 0
    if op == "window":
        seqs = _log(rng, 1, 64)
        longest = _log(rng, 17, min(100003, 16411 * 64 * 512 // (seqs * hkv * d)))
        return dict(op=op, seqs=seqs, rows=rng.choice((1, 1, 2, 3, 5, 8)), longest=longest, ragged=rng.random() < 0.7,
                    q_heads=hq, kv_heads=hkv, dim=d, page=page, window=window, sinks=sinks)
    seqs = _log(rng, 1, 32)
    most = _log(rng, 1, 8195)
    # what the plain form computes: every row of a padded batch against every position
    top = 2048 * 61003 * 24 * 256
    most = max(1, min(most, top // (seqs * 17 * hq * d)))
    longest = _log(rng, 17, max(17, min(100003, top // (seqs * most * hq * d), 100003 * 512 // (seqs * hkv * d))))
    return dict(op=op, seqs=seqs, most=min(most, longest), longest=longest, ragged=rng.random() < 0.7, q_heads=hq,
                kv_heads=hkv, dim=d, page=page, window=window, sinks=sinks)


def _seen(c):
    """(pairs of a query row and a position it sees, positions that any row sees), over the sequences, for one head."""
    pairs = held = 0
    for n, m in zip(_lengths(c).tolist(), _rows(c).tolist()):
        last = np.arange(max(0, n - m), n, dtype=np.int64)              # positions of the rows
        seen = last + 1
        first = n                                                       # the first position that is seen beside the sinks
        if c["window"]:
            seen = np.minimum(seen, c["window"]) + np.clip(last + 1 - c["window"], 0, c["sinks"])
            first = max(0, n - m + 1 - c["window"]) if m else n
            held += (n - first) + min(first, c["sinks"]) if m else 0
        else:
            held += n if m else 0
        pairs += int(seen.sum())
    return pairs, held


def work(case):
    """Bytes: every input read once and every output written once.  Flops: products and sums of the definition."""
    c = case
    d = c["dim"]
    if c["op"] in ("append_rope", "rope"):
        q, k = c["tokens"] * c["q_heads"] * d, c["tokens"] * c["kv_heads"] * d
        by = 4 * q + (2 * k * (2 + 0.5625) + 4 * c["tokens"] if c["op"] == "append_rope" else 4 * k) + 4 * c["tokens"]
        return {"bytes": by, "flops": (q + k) * (3.0 + 4.0 * c["norm"])}
    pairs, held = _seen(c)
    rows = int(_rows(c).sum())
    return {"bytes": held * c["kv_heads"] * d * 1.125 + rows * c["q_heads"] * (4 * d + 4),
            "flops": 4.0 * pairs * c["q_heads"] * d}


# ----------------------------------------------------------------- inputs ---

def _lengths(c):
    """Tokens of each sequence: all the longest, or spread below it with an empty one and a short one among them."""
    b, longest = c["seqs"], c["longest"]
    n = np.full(b, longest, np.int64)
    if c["ragged"]:
        n = np.maximum(1, np.round(longest * np.random.RandomState(b * 7919 + longest).beta(1.2, 1.4, b))).astype(np.int64)
        n[0] = longest
        if b > 2:
            n[1], n[2] = 0, min(3, longest)
    return n


def _rows(c):
    """Query rows of each sequence, the last ones of its tokens."""
    if c["op"] == "window":
        return np.full(c["seqs"], c["rows"], np.int64)
    n, m = _lengths(c), np.full(c["seqs"], c["most"], np.int64)
    if c["ragged"]:
        r = np.random.RandomState(c["seqs"] * 104729 + c["most"])
        m = np.where(r.rand(c["seqs"]) < 0.3, 1, np.round(c["most"] * r.beta(1.0, 1.5, c["seqs"]))).astype(np.int64)
        m[0] = c["most"]
        if c["seqs"] > 3:
            m[3] = 0
    return np.minimum(m, n)


def _frequencies(c):
    """Fractions of a turn per position, in units of 2^-64, and what the rotated components are multiplied by."""
    r, base, factor, original = c["rot"], 1e6, 8.0, 32768
    if c["scaling"] == "base":
        base *= factor ** (r / (r - 2))
    i = np.arange(r // 2)
    f = base ** (-2.0 * i / r)
    amplitude = 1.0
    if c["scaling"] == "linear":
        f = f / factor
    elif c["scaling"] in ("turns", "index"):
        turns = original * f / (2 * math.pi)
        if c["scaling"] == "turns":        # by how often a frequency turns within the context it was made for
            keep = np.clip((turns - 1.0) / (4.0 - 1.0), 0, 1)
        else:                              # by its index, between those that turn 32 times and once
            at = lambda t: r * math.log(original / (t * 2 * math.pi)) / (2 * math.log(base))   # noqa: E731
            lo, hi = max(0, math.floor(at(32.0))), min(r // 2 - 1, math.ceil(at(1.0)))
            keep = 1 - np.clip((i - lo) / max(1e-3, hi - lo), 0, 1)
            amplitude = 0.1 * math.log(factor) + 1
        f = f * (keep + (1 - keep) / factor)
    return np.array([int(x / (2 * math.pi) * 2.0 ** 64) for x in f], np.int64), amplitude


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 2654435761 % (1 << 62) + 11)


def _tables(c, n, width, gen):
    """Pages of each sequence in a shuffled pool, and the pool's size."""
    need = torch.from_numpy((n + c["page"] - 1) // c["page"]).cuda()
    at = torch.arange(width, device="cuda")[None, :] < need[:, None]
    total = int(need.sum())
    order = torch.randperm(max(1, total), generator=gen, device="cuda").int()
    table = torch.zeros(c["seqs"], width, dtype=torch.int32, device="cuda")
    table[at] = order[:total]
    return table, max(1, total)


def _heads_like(shape, gen):
    """Keys or values as a model's projection makes them: near normal, a few channels much larger."""
    x = torch.randn(shape, generator=gen, device="cuda")
    loud = (torch.rand(shape[-1], generator=gen, device="cuda") < 0.03).float() * 4 + 1
    return x * loud


def _filled(c, pages, gen):
    """A cache whose positions all hold tokens."""
    h, d, page = c["kv_heads"], c["dim"], c["page"]
    cache = torch.empty(pages, h, page // 16, 18 * d, dtype=torch.uint8, device="cuda")
    for part, g in ((0, KG), (9 * d, VG)):
        codes, scales = _encode(_heads_like((pages, h, page // 16, 16, d), gen), g)
        rec = cache[..., part:part + 9 * d]
        if part:
            codes = codes.view(pages, h, page // 16, 2, 8, d // 16, 8).transpose(-3, -2).contiguous()
            scales = scales.transpose(-2, -1).contiguous()
        rec[..., :8 * d] = codes.reshape(pages, h, page // 16, 8 * d)
        rec[..., 8 * d:] = scales.reshape(pages, h, page // 16, d)
    return cache


def prepare(case, seed):
    c, gen = dict(case), _gen(seed)
    s = {"case": c}
    hq, h, d = c["q_heads"], c["kv_heads"], c["dim"]
    if c["op"] in ("append_rope", "rope"):
        t = c["tokens"]
        qkv = torch.empty(t, (hq + 2 * h) * d, dtype=torch.float16, device="cuda")    # the fused projection's output
        for lo, n in ((0, hq), (hq, h), (hq + h, h)):
            qkv[:, lo * d:(lo + n) * d] = _heads_like((t, n, d), gen).view(t, -1).half()
        s.update(q=qkv[:, :hq * d].view(t, hq, d), k=qkv[:, hq * d:(hq + h) * d].view(t, h, d),
                 v=qkv[:, (hq + h) * d:].view(t, h, d), q_out=torch.empty(t, hq, d, dtype=torch.float16, device="cuda"))
        freqs, s["amplitude"] = _frequencies(c)
        s["freqs"] = torch.from_numpy(freqs).cuda()
        # a prompt from its start, or rounds of eight rows of requests that are far along
        pos = torch.arange(t, device="cuda")
        if c["far"]:
            begin = torch.randint(0, c["far"], (t // 8 + 1,), generator=gen, device="cuda")
            pos = begin[pos // 8] + pos % 8
        s["positions"] = pos.int()
        for name in ("q_weight", "k_weight"):
            s[name] = torch.randn(d, generator=gen, device="cuda").mul_(0.2).add_(1.0) if c["norm"] else None
        if c["op"] == "rope":
            s["k_out"] = torch.empty(t, h, d, dtype=torch.float16, device="cuda")
            return s
        page = c["page"]
        pages = (t + page - 1) // page + 3
        s["cache"] = torch.zeros(pages, h, page // 16, 18 * d, dtype=torch.uint8, device="cuda")
        # tokens go to consecutive slots of shuffled pages, from an odd offset
        order = torch.randperm(pages, generator=gen, device="cuda")
        at = torch.arange(t, device="cuda") + 5
        s["slots"] = (order[at // page] * page + at % page).int()
        return s
    n, m = _lengths(c), _rows(c)
    width = int((n.max() + c["page"] - 1) // c["page"])
    table, used = _tables(c, n, width, gen)
    t = int(m.sum())
    qkv = torch.randn(t, (hq + 2 * h) * d, generator=gen, device="cuda").mul_(1.5).half()
    s.update(table=table, lens=torch.from_numpy(n).int().cuda(), scale=d ** -0.5, cache=_filled(c, used, gen),
             starts=torch.from_numpy(np.concatenate(([0], np.cumsum(m)))).int().cuda(), q=qkv[:, :hq * d].view(t, hq, d),
             out=torch.empty(t, hq, d, dtype=torch.float16, device="cuda"),
             lse=torch.empty(t, hq, dtype=torch.float32, device="cuda"))
    return s


# ------------------------------------------------------------ plain forms ---

def _e2m1(a):
    """The code of each magnitude: nearest, ties to the even code."""
    return ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte()
            + (a >= 3.5).byte() + (a > 5.0).byte())


def _encode(x, g):
    """FP32 [..., D] -> E2M1 codes u8 [..., D/2] and E4M3 scale codes u8 [..., D/16], each step a rounded FP32 operation."""
    six, gs = torch.full((), 6.0, device=x.device), torch.full((), g, device=x.device)
    blocks = x.unflatten(-1, (-1, 16))
    scales = (blocks.abs().amax(-1) / six / gs).clamp_max(448.0).to(torch.float8_e4m3fn)
    unit = (scales.float() * gs).unsqueeze(-1)
    a = torch.where(unit > 0, blocks.abs() / unit, torch.zeros_like(blocks))
    code = (_e2m1(a) + 8 * torch.signbit(blocks).byte()).flatten(-2)
    return code[..., 0::2] + 16 * code[..., 1::2], scales.view(torch.uint8)


def _encode_wide(x, g):
    """FP64 [..., D] -> the same codes, from the exact quotients."""
    g = float(np.float32(g))
    blocks = x.unflatten(-1, (-1, 16))
    want = blocks.abs().amax(-1) / (6 * g)
    half = torch.ldexp(torch.ones_like(want), torch.frexp(want.clamp_min(2.0 ** -6)).exponent - 4)    # E4M3's step there
    near = (torch.round(want / half) * half).clamp_max(448.0)
    scales = near.float().to(torch.float8_e4m3fn)                                                     # exact by now
    unit = (near * g).unsqueeze(-1)
    a = torch.where(unit > 0, blocks.abs() / unit, torch.zeros_like(blocks))
    code = (_e2m1(a) + 8 * torch.signbit(blocks).byte()).flatten(-2)
    return code[..., 0::2] + 16 * code[..., 1::2], scales.view(torch.uint8)


def _values(codes, scales, g):
    """What codes u8 [..., D/2] and scale codes u8 [..., D/16] stand for, FP32 [..., D]."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    w = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), -1).flatten(-2)
    return (w.unflatten(-1, (-1, 16)) * scales.view(torch.float8_e4m3fn).float().unsqueeze(-1)).flatten(-2) * g


def _views(cache):
    """Key codes, key scales, value codes and value scales of a cache's records, as views."""
    d = cache.shape[-1] // 18
    return (cache[..., :8 * d].unflatten(-1, (16, d // 2)), cache[..., 8 * d:9 * d].unflatten(-1, (16, d // 16)),
            cache[..., 9 * d:17 * d].unflatten(-1, (2, d // 16, 8, 8)), cache[..., 17 * d:].unflatten(-1, (d // 16, 16)))


def _rows_of(cache, table):
    """Codes and scales of every position of every sequence: four u8 tensors [B][H][positions][...]."""
    kc, ks, vc, vs = _views(cache[table.long()].transpose(1, 2))             # [B][H][width][records]...
    vc = vc.transpose(-3, -2).flatten(-2)                                    # [..][2][8][D/2]
    return kc.flatten(2, 4), ks.flatten(2, 4), vc.flatten(2, 5), vs.transpose(-2, -1).flatten(2, 4)


def _write_rows(cache, page, at, kc, ks, vc, vs):
    """Rows [n][H][...] into records of pages `page` at offsets `at` (both [n])."""
    k0, k1, v0, v1 = _views(cache)
    h = torch.arange(cache.shape[1], device=cache.device)
    page, at = page[:, None], at[:, None]
    r, i = at // 16, at % 16
    k0[page, h, r, i] = kc
    k1[page, h, r, i] = ks
    v0[page, h, r, i // 8, :, i % 8] = vc.unflatten(-1, (-1, 8))
    v1[page, h, r, :, i] = vs


def _angles(s):
    """Cosine and sine [T][1][R/2] in 64 bits: whole numbers of 2^-64 turns, which wrap around at a turn."""
    turn = (s["positions"].long()[:, None] * s["freqs"][None, :]).double() * 2.0 ** -64
    a = (turn * (2 * math.pi))[:, None, :]
    return torch.cos(a) * s["amplitude"], torch.sin(a) * s["amplitude"]


def _rotated(s, x, weight, cos, sin):
    """Normed and rotated heads [T][H][D], in the type of `cos`."""
    c, x = s["case"], x.to(cos.dtype)
    r = c["rot"]
    if c["norm"]:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.to(cos.dtype)
    turned = x[..., :r]
    a, b = (turned[..., 0::2], turned[..., 1::2]) if c["interleaved"] else (turned[..., :r // 2], turned[..., r // 2:])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((a, b), -1).flatten(-2) if c["interleaved"] else torch.cat((a, b), -1)
    return torch.cat((turned, x[..., r:]), -1)


def _plain_rope(s):
    cos, sin = _angles(s)
    cos, sin = cos.float(), sin.float()
    return {"q": _rotated(s, s["q"], s["q_weight"], cos, sin).half(), "k": _rotated(s, s["k"], s["k_weight"], cos, sin).half()}


def _plain_append_rope(s):
    cos, sin = _angles(s)
    page = s["case"]["page"]
    kc, ks = _encode_wide(_rotated(s, s["k"], s["k_weight"], cos, sin), KG)
    vc, vs = _encode(s["v"].float(), VG)
    slots = s["slots"].long()
    _write_rows(s["cache"], slots // page, slots % page, kc, ks, vc, vs)
    return {"q": _rotated(s, s["q"], s["q_weight"], cos.float(), sin.float()).half(), "cache": s["cache"]}


def _plain_attention(s):
    """Both kinds: the rows of a sequence are its last ones, padded to the most that a sequence has."""
    c, q, lens = s["case"], s["q"], s["lens"].long()
    b, hq, h, d = c["seqs"], c["q_heads"], c["kv_heads"], c["dim"]
    m = c["most"] if c["op"] == "chunk" else c["rows"]
    kc, ks, vc, vs = _rows_of(s["cache"], s["table"])
    at = torch.arange(kc.shape[2], device=q.device)
    row = torch.arange(m, device=q.device)
    begin, count = s["starts"][:-1].long(), s["starts"][1:].long() - s["starts"][:-1].long()
    there = row < count[:, None]                                                                       # [B][M]
    last = lens[:, None] - count[:, None] + row                                                        # a row's own position
    sees = at <= last[..., None]                                                                       # [B][M][positions]
    if c["window"]:
        sees = sees & ((at > last[..., None] - c["window"]) | (at < c["sinks"]))
    sees = (sees & (at < lens[:, None, None]))[:, None, :, None, :]
    of = torch.where(there, begin[:, None] + row, torch.zeros_like(last))
    qf = q[of].float().view(b, m, h, hq // h, d).permute(0, 2, 1, 3, 4)                                # [B][H][M][G][D]
    z = torch.einsum("bhmgd,bhnd->bhmgn", qf, _values(kc, ks, KG)) * s["scale"]
    z = z.masked_fill_(~sees, -math.inf)
    top = z.amax(-1, keepdim=True)
    p = z.sub_(torch.where(top > -math.inf, top, torch.zeros_like(top))).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.einsum("bhmgn,bhnd->bhmgd", p, _values(vc, vs, VG)) / torch.where(total > 0, total, torch.ones_like(total))
    lse = torch.where(total > 0, top + torch.log(total), torch.full_like(top, -math.inf))
    out, lse = out.permute(0, 2, 1, 3, 4).reshape(b, m, hq, d), lse.squeeze(-1).permute(0, 2, 1, 3).reshape(b, m, hq)
    return {"out": out[there].half(), "lse": lse[there]}


PLAIN = {"rope": _plain_rope, "append_rope": _plain_append_rope, "chunk": _plain_attention, "window": _plain_attention}


# -------------------------------------------------------- the entry points ---

_package = None


def _sk():
    global _package
    if _package is None:
        import fp8_weight_only_skinny_gb300 as package

        package.init()
        _package = package
    return _package


def run(state):
    s, c = state, state["case"]
    if not own:
        return PLAIN[c["op"]](s)
    sk = _sk()
    if c["op"] == "rope":
        q, k = sk.qk_norm_rope(s["q"], s["k"], s["positions"], s["freqs"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                               eps=EPS, interleaved=c["interleaved"], amplitude=s["amplitude"], q_out=s["q_out"],
                               k_out=s["k_out"])
        return {"q": q, "k": k}
    if c["op"] == "append_rope":
        q = sk.kv4_append_rope(s["q"], s["k"], s["v"], s["slots"], s["positions"], s["freqs"], s["cache"], KG, VG,
                               q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, interleaved=c["interleaved"],
                               amplitude=s["amplitude"], q_out=s["q_out"])
        return {"q": q, "cache": s["cache"]}
    if c["op"] == "chunk":
        out, lse = sk.kv4_chunk_attention(s["q"], s["cache"], s["table"], s["lens"], s["starts"], KG, VG, s["scale"],
                                          window=c["window"], sinks=c["sinks"], out=s["out"], lse=s["lse"])
        return {"out": out, "lse": lse}
    out, lse = sk.kv4_window_attention(s["q"], s["cache"], s["table"], s["lens"], KG, VG, s["scale"], c["window"],
                                       sinks=c["sinks"], rows=c["rows"], out=s["out"], lse=s["lse"])
    return {"out": out, "lse": lse}


# ------------------------------------------------ the definition, 64 bits ---

def _value64(code):
    """An E2M1 code's value from its sign, exponent and mantissa bits."""
    e, m = (code >> 1) & 3, (code & 1).double()
    mag = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2((e - 1).double()))
    return torch.where(code >= 8, -mag, mag)


def _scale64(code):
    """An E4M3 code's value (non-negative codes)."""
    e, m = (code >> 3) & 15, (code & 7).double()
    return torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2((e - 7).double()))


def _cache64(s, b, length, which):
    """Keys (which = 0) or values (1) of the first `length` positions of sequence b, FP64 [H][length][D]."""
    cache, c = s["cache"], s["case"]
    d, page = c["dim"], c["page"]
    pages = s["table"][b, :(length + page - 1) // page].long()
    rec = cache[pages].permute(1, 0, 2, 3).reshape(c["kv_heads"], -1, 18 * d)[..., 9 * d * which:9 * d * (which + 1)].long()
    codes, scales = rec[..., :8 * d], rec[..., 8 * d:]
    if which:
        codes = codes.reshape(*codes.shape[:2], 2, d // 16, 8, 8).permute(0, 1, 2, 4, 3, 5)
        scales = scales.reshape(*scales.shape[:2], d // 16, 16).permute(0, 1, 3, 2)
    codes, scales = codes.reshape(c["kv_heads"], -1, d // 2), scales.reshape(c["kv_heads"], -1, d // 16)
    x = torch.stack((_value64(codes & 15), _value64(codes >> 4)), -1).reshape(c["kv_heads"], -1, d)
    x = x * _scale64(scales).repeat_interleave(16, -1) * float(np.float32(VG if which else KG))
    return x[:, :length]


def _near64(x, mantissa, least, most):
    """x >= 0 to the nearest value with `mantissa` stored bits and exponents from `least`, ties to even, at most `most`."""
    e = torch.floor(torch.log2(x.clamp_min(2.0 ** least))).clamp_min(least)
    step = torch.exp2(e - mantissa)
    return (torch.round(x / step) * step).clamp_max(most)


def _heads64(s, x, weight):
    """Normed and rotated heads as products of complex numbers."""
    c = s["case"]
    r, y = c["rot"], x.double()
    if c["norm"]:
        y = y * torch.rsqrt((y * y).sum(-1, keepdim=True) / c["dim"] + EPS) * weight.double()
    # the fraction of a turn from the product's low 64 bits
    with np.errstate(over="ignore"):
        low = s["positions"].cpu().numpy().astype(np.int64).astype(np.uint64)[:, None] * s["freqs"].cpu().numpy().astype(np.uint64)
    turn = torch.from_numpy(low.astype(np.longdouble).astype(np.float64) / 2.0 ** 64).cuda()
    unit = torch.polar(torch.full_like(turn, s["amplitude"]), turn * (2 * math.pi))[:, None]
    head = y[..., :r]
    pairs = head.unflatten(-1, (r // 2, 2)) if c["interleaved"] else head.unflatten(-1, (2, r // 2)).transpose(-1, -2)
    turned = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * unit)
    turned = turned if c["interleaved"] else turned.transpose(-1, -2)
    y[..., :r] = turned.flatten(-2)
    return y


def _exact_rope(s):
    return {"q": _heads64(s, s["q"], s["q_weight"]), "k": _heads64(s, s["k"], s["k_weight"])}


def _exact_append_rope(s):
    # keys: codes of the exact quotients; values: each step a rounded binary32 operation (a quotient or product of two
    # binary32 numbers taken in 64 bits and rounded once more is that operation's result)
    c = s["case"]
    cache = s["cache"].clone()
    d, page, h = c["dim"], c["page"], c["kv_heads"]
    slots = s["slots"].long()
    rec = cache.view(-1, h, page // 16, 18 * d)
    p, r, i = slots // page, slots % page // 16, slots % 16
    byte, blk = torch.arange(8, device=cache.device), torch.arange(d // 16, device=cache.device)[:, None]
    same, r32 = (lambda y: y), (lambda y: y.float().double())
    for x, g, part, step in ((_heads64(s, s["k"], s["k_weight"]), KG, 0, same), (s["v"].double(), VG, 9 * d, r32)):
        g = float(np.float32(g))
        blocks = x.reshape(-1, h, d // 16, 16)
        sc = _near64(step(step(blocks.abs().amax(-1) / 6.0) / g), 3, -6, 448.0)
        unit = step(sc * g)[..., None]
        near = _near64(torch.where(unit > 0, step(blocks.abs() / unit.clamp_min(1e-300)), torch.zeros_like(blocks)), 1, 0, 6.0)
        e = torch.floor(torch.log2(near.clamp_min(0.25)))
        code = torch.where(near < 1, near * 2, 2 * (e + 1) + (near / torch.exp2(e) - 1) * 2).long()
        code = code + 8 * torch.signbit(blocks).long()
        pair = (code[..., 0::2] + 16 * code[..., 1::2]).byte()                          # [T][H][D/16][8]
        e = torch.floor(torch.log2(sc.clamp_min(2.0 ** -6)))
        scode = torch.where(sc < 2.0 ** -6, sc * 2 ** 9, (e + 7) * 8 + (sc / torch.exp2(e) - 1) * 8).long().byte()
        for head in range(h):
            if part == 0:
                where = i[:, None, None] * (d // 2) + blk * 8 + byte
                at = 8 * d + i[:, None] * (d // 16) + blk[:, 0]
            else:
                where = part + (i[:, None, None] // 8) * (4 * d) + blk * 64 + (i[:, None, None] % 8) * 8 + byte
                at = 17 * d + blk[:, 0] * 16 + i[:, None]
            rec[p[:, None, None], head, r[:, None, None], where] = pair[:, head]
            rec[p[:, None], head, r[:, None], at] = scode[:, head]
    return {"q": _heads64(s, s["q"], s["q_weight"]), "cache": cache}


def _exact_attention(s):
    c = s["case"]
    hq, h, d = c["q_heads"], c["kv_heads"], c["dim"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    row0 = 0
    for b, (n, m) in enumerate(zip(_lengths(c).tolist(), _rows(c).tolist())):
        if n and m:
            k, v = _cache64(s, b, n, 0), _cache64(s, b, n, 1)
            j = torch.arange(n, device="cuda")
            for lo in range(0, m, 128):
                hi = min(m, lo + 128)
                own_at = torch.arange(n - m + lo, n - m + hi, device="cuda")[:, None]
                hidden = j > own_at
                if c["window"]:
                    hidden = hidden | ((own_at - j >= c["window"]) & (j >= c["sinks"]))
                q = s["q"][row0 + lo:row0 + hi].double().view(-1, h, hq // h, d).permute(1, 2, 0, 3).reshape(h, -1, d)
                z = (q @ k.transpose(1, 2) * s["scale"]).view(h, hq // h, hi - lo, n).masked_fill_(hidden, -math.inf)
                total = torch.logsumexp(z, -1)
                lse[row0 + lo:row0 + hi] = total.permute(2, 0, 1).reshape(hi - lo, hq)
                # a row before the sequence's first position sees nothing
                p = torch.exp(z - torch.where(total > -math.inf, total, torch.zeros_like(total))[..., None])
                y = (p.view(h, -1, n) @ v).view(h, hq // h, hi - lo, d)
                out[row0 + lo:row0 + hi] = y.permute(2, 0, 1, 3).reshape(hi - lo, hq, d)
        row0 += m
    return {"out": out, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "append_rope": _exact_append_rope, "chunk": _exact_attention,
            "window": _exact_attention}[case["op"]](s)
