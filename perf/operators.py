"""Cases and plain forms of the operators around the key/value cache held in 4 bits and of the
log probabilities beside the vocabulary projection.

    append     keys and values of new tokens, FP16 -> NVFP4 records of a paged cache
    attention  1..8 query rows per sequence over that cache, with the weight each position got
    evict      keep the most attended positions of a cache within a budget, in other pages
    logprobs   log probability, rank, entropy and top alternatives of rows of logits

Each case is run in its plain form (elementary torch operations in 32 bits) or, with `own` set,
through the package's entry points.

The cache is u8 [pages][kv_heads][page_size / 16][18 D], one record of 18 D bytes per 16 positions
(D the head size): key codes [16][D/2], key scales [16][D/16], value codes [2][D/16][8][8] (half of
the positions, block of 16 components, position, byte), value scales [D/16][16].  Codes are E2M1,
low nibble first; scales are E4M3, one per 16 components of a position; one FP32 scale for all keys
and one for all values.
"""
import math

import numpy as np
import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # one decode token's key and value: the smallest call of a decode step
        dict(name="append_token", op="append", tokens=1, q_heads=48, kv_heads=4, dim=128, page=64, held=False),
        # 37 requests' speculative rounds of 8 rows, cut out of the fused projection's output
        dict(name="append_rounds", op="append", tokens=296, q_heads=24, kv_heads=2, dim=256, page=32, held=False),
        # a long prompt, with the values the cache then stands for (the prompt's own attention reads those)
        dict(name="append_prompt", op="append", tokens=32771, q_heads=48, kv_heads=4, dim=128, page=64, held=True),
        # one token of one request early in its answer
        dict(name="attention_token", op="attention", seqs=1, rows=1, longest=1031, ragged=False, q_heads=48, kv_heads=4,
             dim=128, page=64, weights=False),
        # the verify round (8 rows) of one request with a long context
        dict(name="attention_verify", op="attention", seqs=1, rows=8, longest=100003, ragged=False, q_heads=48,
             kv_heads=4, dim=128, page=64, weights=False),
        # a server's decode step: 64 requests of mixed lengths
        dict(name="attention_batch", op="attention", seqs=64, rows=1, longest=16411, ragged=True, q_heads=24, kv_heads=2,
             dim=256, page=64, weights=False),
        # short rounds over small heads and pages with the weights accumulated for eviction, empty requests among them
        dict(name="attention_weights", op="attention", seqs=23, rows=2, longest=9001, ragged=True, q_heads=32, kv_heads=8,
             dim=64, page=16, weights=True),
        # one request trimmed to a small budget
        dict(name="evict_one", op="evict", seqs=1, longest=1500, ragged=False, kv_heads=4, dim=128, page=64, budget=512,
             recent=128),
        # a server's caches trimmed at their high-water mark
        dict(name="evict_batch", op="evict", seqs=16, longest=16411, ragged=True, kv_heads=2, dim=256, page=64,
             budget=4096, recent=256),
        # the token just sampled, with five alternatives
        dict(name="logprobs_token", op="logprobs", rows=1, vocab=151936, half=False, top=5, temperature=1.0),
        # a verify round's eight rows of FP16 logits
        dict(name="logprobs_round", op="logprobs", rows=8, vocab=151936, half=True, top=20, temperature=0.6),
        # a scored prompt
        dict(name="logprobs_prompt", op="logprobs", rows=2048, vocab=151936, half=False, top=20, temperature=1.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = ((48, 4, 128), (24, 2, 256), (32, 8, 64), (32, 8, 128), (8, 8, 128), (12, 4, 64), (16, 2, 256), (10, 1, 128))


def draw(rng):
    op = rng.choice(("append", "attention", "attention", "evict", "logprobs"))
    hq, hkv, d = rng.choice(HEADS)
    page = rng.choice((16, 32, 64, 128, 48))
    if op == "append":
        most = 32771 * 4 * 128 // (hkv * d)
        return dict(op=op, tokens=_log(rng, 1, most), q_heads=hq, kv_heads=hkv, dim=d, page=page,
                    held=rng.random() < 0.5)
    if op == "attention":
        seqs = _log(rng, 1, 64)
        longest = _log(rng, 17, min(100003, 100003 * 512 // (seqs * hkv * d)))
        return dict(op=op, seqs=seqs, rows=rng.choice((1, 1, 2, 3, 5, 8)), longest=longest, ragged=rng.random() < 0.7,
                    q_heads=hq, kv_heads=hkv, dim=d, page=page, weights=rng.random() < 0.4)
    if op == "evict":
        seqs = _log(rng, 1, 16)
        longest = _log(rng, 40, 16411 * 512 // (hkv * d))
        budget = _log(rng, 16, min(4096, longest))
        return dict(op=op, seqs=seqs, longest=longest, ragged=rng.random() < 0.7, kv_heads=hkv, dim=d, page=page,
                    budget=budget, recent=rng.randrange(0, budget + 1))
    vocab = _log(rng, 300, 151936)
    return dict(op=op, rows=_log(rng, 1, 2048), vocab=vocab, half=rng.random() < 0.4, top=rng.choice((0, 1, 5, 8, 20)),
                temperature=rng.choice((1.0, 1.0, 0.6, 1.7)))


def work(case):
    """Bytes: every input read once and every output written once.  Flops: products and sums of the definition."""
    c = case
    if c["op"] == "append":
        n = c["tokens"] * c["kv_heads"] * c["dim"] * 2            # keys and values
        return {"bytes": n * (2 + 0.5625 + (2 if c["held"] else 0)) + 4 * c["tokens"], "flops": 4.0 * n}
    if c["op"] == "attention":
        positions = int(_lengths(c).sum())
        t = c["seqs"] * c["rows"]
        by = positions * c["kv_heads"] * c["dim"] * 1.125 + t * c["q_heads"] * (c["dim"] * 4 + 4)
        by += positions * c["kv_heads"] * 8 if c["weights"] else 0
        return {"bytes": by, "flops": 4.0 * positions * c["rows"] * c["q_heads"] * c["dim"]}
    if c["op"] == "evict":
        n = _lengths(c)
        kept = int(np.minimum(n, c["budget"]).sum())
        row = c["dim"] * 1.125
        return {"bytes": c["kv_heads"] * (int(n.sum()) * 4 + kept * (2 * row + 8)), "flops": float(c["kv_heads"] * int(n.sum()))}
    n = c["rows"] * c["vocab"]
    return {"bytes": n * (2 if c["half"] else 4) + c["rows"] * (16 + 8 * c["top"]), "flops": 6.0 * n}


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
        x = _heads_like((pages, h, page // 16, 16, d), gen)
        codes, scales = _encode(x, g)
        rec = cache[..., part:part + 9 * d]
        if part:
            codes = codes.view(pages, h, page // 16, 2, 8, d // 16, 8).transpose(-3, -2).contiguous()
            scales = scales.transpose(-2, -1).contiguous()
        rec[..., :8 * d] = codes.reshape(pages, h, page // 16, 8 * d)
        rec[..., 8 * d:] = scales.reshape(pages, h, page // 16, d)
    return cache


KG, VG = 0.02, 0.015


def prepare(case, seed):
    c, gen = dict(case), _gen(seed)
    s = {"case": c}
    if c["op"] == "append":
        t, hq, h, d, page = c["tokens"], c["q_heads"], c["kv_heads"], c["dim"], c["page"]
        qkv = torch.empty(t, (hq + 2 * h) * d, dtype=torch.float16, device="cuda")    # the fused projection's output
        qkv[:, :hq * d] = 0
        qkv[:, hq * d:(hq + h) * d] = _heads_like((t, h, d), gen).view(t, -1).half()
        qkv[:, (hq + h) * d:] = _heads_like((t, h, d), gen).view(t, -1).half()
        pages = (t + page - 1) // page + 3
        s.update(k=qkv[:, hq * d:(hq + h) * d].view(t, h, d), v=qkv[:, (hq + h) * d:].view(t, h, d),
                 cache=torch.zeros(pages, h, page // 16, 18 * d, dtype=torch.uint8, device="cuda"))
        # tokens go to consecutive slots of shuffled pages, from an odd offset
        order = torch.randperm(pages, generator=gen, device="cuda")
        at = torch.arange(t, device="cuda") + 5
        s["slots"] = (order[at // page] * page + at % page).int()
        if c["held"]:
            s["k_held"] = torch.empty(t, h, d, dtype=torch.float16, device="cuda")
            s["v_held"] = torch.empty_like(s["k_held"])
        return s
    if c["op"] in ("attention", "evict"):
        n = _lengths(c)
        h, d, page, b = c["kv_heads"], c["dim"], c["page"], c["seqs"]
        width = int((n.max() + page - 1) // page)
        table, used = _tables(c, n, width, gen)
        s.update(table=table, lens=torch.from_numpy(n).int().cuda())
        if c["op"] == "attention":
            hq, t = c["q_heads"], b * c["rows"]
            qkv = torch.randn(t, (hq + 2 * h) * d, generator=gen, device="cuda").mul_(1.5).half()
            s.update(q=qkv[:, :hq * d].view(t, hq, d), scale=d ** -0.5, cache=_filled(c, used, gen),
                     out=torch.empty(t, hq, d, dtype=torch.float16, device="cuda"),
                     lse=torch.empty(t, hq, dtype=torch.float32, device="cuda"))
            if c["weights"]:
                s["acc"] = torch.rand(b, h, width * page, generator=gen, device="cuda").square_()
                s["acc"] *= (torch.arange(width * page, device="cuda") < s["lens"][:, None])[:, None, :]
                s["acc_out"] = torch.zeros_like(s["acc"])
            return s
        per = (c["budget"] + page - 1) // page
        s["cache"] = _filled(c, used + b * per, gen)
        s["dst"] = (used + torch.randperm(b * per, generator=gen, device="cuda")).int().view(b, per)
        # a few positions carry most of the weight, some none at all
        u = torch.rand(b, h, width * page, generator=gen, device="cuda")
        s["acc"] = torch.where(u < 0.05, torch.zeros_like(u), u.clamp_min(1e-6) ** 6 * 40)
        s["kept"] = torch.empty(b, h, c["budget"], dtype=torch.int32, device="cuda")
        s["new_lens"] = torch.empty(b, dtype=torch.int32, device="cuda")
        s["acc_out"] = torch.empty(b, h, per * page, dtype=torch.float32, device="cuda")
        return s
    m, n = c["rows"], c["vocab"]
    z = torch.randn(m, n, generator=gen, device="cuda")
    z.mul_(2.2).sub_(1.0)
    some = (torch.randint(0, n, (m, 1), generator=gen, device="cuda") + torch.arange(12, device="cuda") * (n // 12 - 1)) % n
    z.scatter_(1, some, torch.rand(m, 12, generator=gen, device="cuda") * 9 + 6)      # the likely continuations
    z[:, ::17] = -math.inf                                                             # tokens that a grammar forbids
    s["logits"] = z.half() if c["half"] else z
    s["tokens"] = some[:, 3].int().contiguous()
    s["logprob"] = torch.empty(m, dtype=torch.float32, device="cuda")
    s["rank"] = torch.empty(m, dtype=torch.int32, device="cuda")
    s["entropy"] = torch.empty(m, dtype=torch.float32, device="cuda")
    s["top_ids"] = torch.empty(m, c["top"], dtype=torch.int32, device="cuda")
    s["top_logprobs"] = torch.empty(m, c["top"], dtype=torch.float32, device="cuda")
    return s


# ------------------------------------------------------------ plain forms ---

def _encode(x, g):
    """FP32 [..., D] -> E2M1 codes u8 [..., D/2] and E4M3 scale codes u8 [..., D/16], each step a rounded FP32 operation."""
    six, gs = torch.full((), 6.0, device=x.device), torch.full((), g, device=x.device)
    blocks = x.unflatten(-1, (-1, 16))
    scales = (blocks.abs().amax(-1) / six / gs).clamp_max(448.0).to(torch.float8_e4m3fn)
    unit = (scales.float() * gs).unsqueeze(-1)
    a = torch.where(unit > 0, blocks.abs() / unit, torch.zeros_like(blocks))
    code = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte()
            + (a >= 3.5).byte() + (a > 5.0).byte())
    code = (code + 8 * torch.signbit(blocks).byte()).flatten(-2)
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
    """Rows [n][H][...] into records of pages `page` at offsets `at` (both [n], or [n][H] with a head index)."""
    k0, k1, v0, v1 = _views(cache)
    h = torch.arange(cache.shape[1], device=cache.device)
    page, at = (page[:, None], at[:, None]) if page.dim() == 1 else (page, at)
    r, i = at // 16, at % 16
    k0[page, h, r, i] = kc
    k1[page, h, r, i] = ks
    v0[page, h, r, i // 8, :, i % 8] = vc.unflatten(-1, (-1, 8))
    v1[page, h, r, :, i] = vs


def _plain_append(s):
    k, v, cache, page = s["k"], s["v"], s["cache"], s["case"]["page"]
    kc, ks = _encode(k.float(), KG)
    vc, vs = _encode(v.float(), VG)
    slots = s["slots"].long()
    _write_rows(cache, slots // page, slots % page, kc, ks, vc, vs)
    if not s["case"]["held"]:
        return {"cache": cache}
    return {"cache": cache, "k_held": _values(kc, ks, KG).half(), "v_held": _values(vc, vs, VG).half()}


def _plain_attention(s):
    c, q, lens = s["case"], s["q"], s["lens"].long()
    b, m, hq, h, d = c["seqs"], c["rows"], c["q_heads"], c["kv_heads"], c["dim"]
    kc, ks, vc, vs = _rows_of(s["cache"], s["table"])
    at = torch.arange(kc.shape[2], device=q.device)
    sees = at < (lens[:, None] - (m - 1) + torch.arange(m, device=q.device))[:, :, None]               # [B][M][positions]
    sees = sees[:, None, :, None, :]
    qf = q.float().view(b, m, h, hq // h, d).permute(0, 2, 1, 3, 4)                                    # [B][H][M][G][D]
    z = torch.einsum("bhmgd,bhnd->bhmgn", qf, _values(kc, ks, KG)) * s["scale"]
    z = z.masked_fill(~sees, -math.inf)
    top = z.amax(-1, keepdim=True)
    p = torch.where(sees, torch.exp(z - top), torch.zeros_like(z))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, torch.ones_like(total))
    out = torch.einsum("bhmgn,bhnd->bhmgd", p, _values(vc, vs, VG)).permute(0, 2, 1, 3, 4).reshape(b * m, hq, d).half()
    lse = torch.where(total > 0, top + torch.log(total), torch.full_like(top, -math.inf))
    got = {"out": out, "lse": lse.squeeze(-1).permute(0, 2, 1, 3).reshape(b * m, hq)}
    if c["weights"]:
        got["acc"] = torch.where((at < lens[:, None])[:, None, :], s["acc"] + p.sum((2, 3)), s["acc_out"])
    return got


def _plain_evict(s):
    c, acc, lens = s["case"], s["acc"], s["lens"].long()
    b, h, page, budget = c["seqs"], c["kv_heads"], c["page"], c["budget"]
    kc, ks, vc, vs = _rows_of(s["cache"], s["table"])
    at = torch.arange(acc.shape[2], device=acc.device)
    n = lens[:, None, None]
    # larger first, ties to the lower position: the weight's bits (never negative) above the position counted down
    bits = torch.where(at >= n - c["recent"], 0x7F800000, acc.view(torch.int32).long())
    key = (bits << 32) + ((1 << 31) - at)
    key = torch.where(at < n, key, -1 - at)
    have = min(budget, acc.shape[2])
    idx = key.topk(have, dim=-1).indices
    new = torch.minimum(lens, torch.full_like(lens, budget))
    slot = torch.arange(budget, device=acc.device)
    idx = torch.where(slot[:have] < new[:, None, None], idx, torch.full_like(idx, 1 << 40)).sort(-1).values
    kept = torch.cat((idx, torch.full((b, h, budget - have), 1 << 40, device=acc.device)), -1)
    valid = slot < new[:, None, None]
    kept = torch.where(valid, kept, torch.full_like(kept, -1))
    take = kept.clamp_min(0)
    rows = [x.gather(2, take[..., None].expand(-1, -1, -1, x.shape[-1])).transpose(1, 2).flatten(0, 1) for x in (kc, ks, vc, vs)]
    dst = s["dst"].long()[:, slot // page].reshape(-1)                                                 # [B * budget]
    to = (slot % page).repeat(b)
    # slots past a sequence's new length keep what they hold
    old = [x[:, :, :budget].transpose(1, 2).flatten(0, 1) for x in _rows_of(s["cache"], s["dst"])]
    live = valid[:, 0].reshape(-1)[:, None, None]
    _write_rows(s["cache"], dst, to, *[torch.where(live, x, y) for x, y in zip(rows, old)])
    weight = torch.where(valid, acc.gather(2, take), torch.zeros((), device=acc.device))
    weight = torch.cat((weight, torch.zeros(b, h, s["acc_out"].shape[2] - budget, device=acc.device)), -1)
    return {"kept": kept.int(), "new_lens": new.int(), "acc": weight, "cache": s["cache"]}


def _plain_logprobs(s):
    c, tokens = s["case"], s["tokens"].long()
    z = s["logits"].float() + 0.0
    t = z / torch.full((), c["temperature"], device=z.device)
    top = t.amax(-1, keepdim=True)
    e = torch.exp(t - top)
    total = e.sum(-1, keepdim=True)
    lse = top + torch.log(total)
    entropy = torch.log(total) - torch.where(e > 0, e * (t - top), torch.zeros_like(t)).sum(-1, keepdim=True) / total
    mine, at = z.gather(1, tokens[:, None]), torch.arange(z.shape[1], device=z.device)
    rank = 1 + ((z > mine) | ((z == mine) & (at < tokens[:, None]))).sum(-1)
    bits = z.view(torch.int32)
    key = (torch.where(bits < 0, -1 - (bits & 0x7FFFFFFF), bits).long() << 32) + ((1 << 31) - at)
    ids = key.topk(c["top"], dim=-1).indices
    return {"logprob": (t.gather(1, tokens[:, None]) - lse).squeeze(-1), "rank": rank.int(),
            "entropy": entropy.squeeze(-1), "top_ids": ids.int(), "top_logprobs": t.gather(1, ids) - lse}


PLAIN = {"append": _plain_append, "attention": _plain_attention, "evict": _plain_evict, "logprobs": _plain_logprobs}


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
    if c["op"] == "append":
        if not c["held"]:
            sk.kv4_append(s["k"], s["v"], s["slots"], s["cache"], KG, VG)
            return {"cache": s["cache"]}
        sk.kv4_append(s["k"], s["v"], s["slots"], s["cache"], KG, VG, k_held=s["k_held"], v_held=s["v_held"])
        return {"cache": s["cache"], "k_held": s["k_held"], "v_held": s["v_held"]}
    if c["op"] == "attention":
        if not c["weights"]:
            sk.kv4_attention(s["q"], s["cache"], s["table"], s["lens"], KG, VG, s["scale"], rows=c["rows"],
                             out=s["out"], lse=s["lse"])
            return {"out": s["out"], "lse": s["lse"]}
        sk.kv4_attention(s["q"], s["cache"], s["table"], s["lens"], KG, VG, s["scale"], rows=c["rows"], out=s["out"],
                         lse=s["lse"], acc=s["acc"], acc_out=s["acc_out"])
        return {"out": s["out"], "lse": s["lse"], "acc": s["acc_out"]}
    if c["op"] == "evict":
        sk.kv4_evict(s["cache"], s["table"], s["lens"], s["acc"], s["dst"], c["budget"], c["recent"], kept=s["kept"],
                     new_lens=s["new_lens"], acc_out=s["acc_out"])
        return {"kept": s["kept"], "new_lens": s["new_lens"], "acc": s["acc_out"], "cache": s["cache"]}
    sk.token_logprobs(s["logits"], s["tokens"], top_n=c["top"], temperature=c["temperature"], logprob=s["logprob"],
                      rank=s["rank"], entropy=s["entropy"], top_ids=s["top_ids"], top_logprobs=s["top_logprobs"])
    return {"logprob": s["logprob"], "rank": s["rank"], "entropy": s["entropy"], "top_ids": s["top_ids"],
            "top_logprobs": s["top_logprobs"]}


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


def _exact_append(s):
    # the definition fixes each step to a rounded binary32 operation; a quotient or product of two binary32
    # numbers taken in 64 bits and rounded once more is that operation's result
    c, got = s["case"], {}
    cache = s["cache"].clone()
    d, page, h = c["dim"], c["page"], c["kv_heads"]
    slots = s["slots"].long()
    heads = torch.arange(h, device=cache.device)
    for name, x, g, part in (("k", s["k"], KG, 0), ("v", s["v"], VG, 9 * d)):
        g = float(np.float32(g))
        blocks = x.double().reshape(-1, h, d // 16, 16)
        r32 = lambda y: y.float().double()                                             # noqa: E731
        sc = _near64(r32(r32(blocks.abs().amax(-1) / 6.0) / g), 3, -6, 448.0)
        unit = r32(sc * g)[..., None]
        q = torch.where(unit > 0, r32(blocks.abs() / unit.clamp_min(1e-300)), torch.zeros_like(blocks))
        near = _near64(q, 1, 0, 6.0)
        if c["held"]:
            value = torch.where(torch.signbit(blocks), -near, near) * sc[..., None] * g
            got[name + "_held"] = value.reshape(-1, h, d)
        e = torch.floor(torch.log2(near.clamp_min(0.25)))
        code = torch.where(near < 1, near * 2, 2 * (e + 1) + (near / torch.exp2(e) - 1) * 2).long()
        code = code + 8 * torch.signbit(blocks).long()
        pair = (code[..., 0::2] + 16 * code[..., 1::2]).byte()                          # [T][H][D/16][8]
        e = torch.floor(torch.log2(sc.clamp_min(2.0 ** -6)))
        scode = torch.where(sc < 2.0 ** -6, sc * 2 ** 9, (e + 7) * 8 + (sc / torch.exp2(e) - 1) * 8).long().byte()
        rec = cache.view(-1, h, page // 16, 18 * d)
        p, r, i = slots // page, slots % page // 16, slots % 16
        byte = torch.arange(8, device=cache.device)
        blk = torch.arange(d // 16, device=cache.device)[:, None]
        for head in heads.tolist():
            if part == 0:
                where = i[:, None, None] * (d // 2) + blk * 8 + byte
                at = 8 * d + i[:, None] * (d // 16) + blk[:, 0]
            else:
                where = part + (i[:, None, None] // 8) * (4 * d) + blk * 64 + (i[:, None, None] % 8) * 8 + byte
                at = 17 * d + blk[:, 0] * 16 + i[:, None]
            rec[p[:, None, None], head, r[:, None, None], where] = pair[:, head]
            rec[p[:, None], head, r[:, None], at] = scode[:, head]
    return {"cache": cache, **got}


def _exact_attention(s):
    c = s["case"]
    b, m, hq, h, d = c["seqs"], c["rows"], c["q_heads"], c["kv_heads"], c["dim"]
    out = torch.zeros(b, m, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((b, m, hq), -math.inf, dtype=torch.float64, device="cuda")
    acc = s["acc_out"].double().clone() if c["weights"] else None
    for i, n in enumerate(_lengths(c).tolist()):
        if n == 0:
            continue
        k, v = _cache64(s, i, n, 0), _cache64(s, i, n, 1)
        weight = torch.zeros(h, n, dtype=torch.float64, device="cuda")
        for r in range(m):
            sees = n - (m - 1 - r)
            if sees <= 0:
                continue
            q = s["q"][i * m + r].double().view(h, hq // h, d)
            z = q @ k[:, :sees].transpose(1, 2) * s["scale"]
            lse[i, r] = torch.logsumexp(z, -1).reshape(-1)
            p = torch.softmax(z, -1)
            out[i, r] = (p @ v[:, :sees]).reshape(hq, d)
            weight[:, :sees] += p.sum(1)
        if c["weights"]:
            acc[i, :, :n] = s["acc"][i, :, :n].double() + weight
    got = {"out": out.reshape(b * m, hq, d), "lse": lse.reshape(b * m, hq)}
    return {**got, "acc": acc} if c["weights"] else got


def _exact_evict(s):
    c = s["case"]
    b, h, page, budget, d = c["seqs"], c["kv_heads"], c["page"], c["budget"], c["dim"]
    kept = torch.full((b, h, budget), -1, dtype=torch.int64)
    acc = torch.zeros(s["acc_out"].shape, dtype=torch.float64)
    cache, weights = s["cache"].cpu().numpy().copy(), s["acc"].cpu().numpy()
    table, dst = s["table"].cpu().numpy(), s["dst"].cpu().numpy()
    new = np.minimum(_lengths(c), budget)
    for i, n in enumerate(_lengths(c).tolist()):
        for head in range(h):
            w = weights[i, head, :n].astype(np.float64)
            w[max(0, n - c["recent"]):] = np.inf
            if c["recent"] == 0:
                w = weights[i, head, :n].astype(np.float64)
            idx = np.sort(np.argsort(-w, kind="stable")[:budget])
            kept[i, head, :len(idx)] = torch.from_numpy(idx)
            acc[i, head, :len(idx)] = torch.from_numpy(weights[i, head, idx].astype(np.float64))
            j = np.arange(len(idx))
            byte = np.arange(18 * d)
            # the position that a record's byte belongs to
            pos = np.concatenate((np.repeat(np.arange(16), d // 2), np.repeat(np.arange(16), d // 16),
                                  (np.arange(8 * d) // (4 * d)) * 8 + np.arange(8 * d) // 8 % 8, np.tile(np.arange(16), d // 16)))
            of = np.stack([byte[pos == p] for p in range(16)])
            sp, so, dp, do = table[i, idx // page], idx % page, dst[i, j // page], j % page
            cache[dp[:, None], head, (do // 16)[:, None], of[do % 16]] = cache[sp[:, None], head, (so // 16)[:, None], of[so % 16]]
    return {"kept": kept.int().cuda(), "new_lens": torch.from_numpy(new).int().cuda(), "acc": acc.cuda(),
            "cache": torch.from_numpy(cache).cuda()}


def _exact_logprobs(s):
    c, got = s["case"], {"logprob": [], "rank": [], "entropy": [], "top_ids": [], "top_logprobs": []}
    for lo in range(0, c["rows"], 256):
        z, tok = s["logits"][lo:lo + 256].double(), s["tokens"][lo:lo + 256].long()[:, None]
        lp = torch.log_softmax(z / float(np.float32(c["temperature"])), -1)
        mine = z.gather(1, tok)
        got["logprob"].append(lp.gather(1, tok)[:, 0])
        before = torch.arange(z.shape[1], device=z.device) < tok
        got["rank"].append((1 + (z > mine).sum(-1) + ((z == mine) & before).sum(-1)).int())
        got["entropy"].append(torch.special.entr(lp.exp()).sum(-1))
        ids = torch.sort(z, dim=-1, descending=True, stable=True).indices[:, :c["top"]]
        got["top_ids"].append(ids.int())
        got["top_logprobs"].append(lp.gather(1, ids))
    return {k: torch.cat(v) for k, v in got.items()}


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attention": _exact_attention, "evict": _exact_evict,
            "logprobs": _exact_logprobs}[case["op"]](s)
