"""Speculative decode rounds of one layer with its cache in 4 bits.

Each round projects M rows (the last token and M - 1 drafted ones), appends their keys and values
to the cache, attends over it, projects back, and verifies the drafts against the vocabulary
projection, whose picks are reported with their log probability, rank, entropy and alternatives.
The weight that the accepted rows give to each position is accumulated.  When the cache reaches its
high-water mark it is trimmed to the positions with the most weight (and the latest), in other pages.

    python examples/decode_round.py [rounds]

The weights are random: the example shows which call reads what, not a language model.
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

HIDDEN, Q_HEADS, KV_HEADS, DIM, VOCAB = 1024, 8, 2, 128, 4096
K_SCALE = V_SCALE = 0.002        # 1/2688 of the largest key and value expected


def decode(rounds=40, rows=4, page=32, high_water=256, budget=96, recent=32, top_n=5, seed=0):
    """Run `rounds` rounds; returns a dict with the committed tokens, what was reported of them, the cache and its
    bookkeeping at the end."""
    import torch

    import fp8_weight_only_skinny_gb300 as sk

    sk.init()
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=torch.float32)      # noqa: E731
    n_qkv = (Q_HEADS + 2 * KV_HEADS) * DIM
    qkv_w = sk.fp8_quantize((rand(n_qkv, HIDDEN) * HIDDEN ** -0.5).half())
    out_w = sk.fp8_quantize((rand(HIDDEN, Q_HEADS * DIM) * HIDDEN ** -0.5).half())
    head_codes, head_scales, head_g = sk.nvfp4_quantize((rand(VOCAB, HIDDEN) * HIDDEN ** -0.5).half())
    head_g = float(head_g)
    embed = rand(VOCAB, HIDDEN).half()

    per = high_water // page                       # pages of the sequence, twice: the trimmed cache goes to the others
    cache = sk.kv4_cache(2 * per, KV_HEADS, DIM, page)
    pages = [torch.arange(i * per, (i + 1) * per, dtype=torch.int32, device="cuda")[None] for i in (0, 1)]
    table, spare = pages
    acc = torch.zeros(1, KV_HEADS, high_water, device="cuda")
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    n, evictions = 0, 0
    tokens = [1]
    report = []
    for _ in range(rounds):
        if n + rows > high_water:
            lens.fill_(n)
            lens, kept, acc = sk.kv4_evict(cache, table, lens, acc, spare, budget, recent)
            table, spare = spare, table
            n = min(n, budget)
            evictions += 1
        draft = torch.randint(0, VOCAB, (rows - 1,), generator=gen, device="cuda", dtype=torch.int32)
        row_tokens = torch.cat((torch.tensor(tokens[-1:], dtype=torch.int32, device="cuda"), draft))
        x = embed[row_tokens.long()]
        qkv = sk.fp8_gemm(x, *qkv_w, f16_out=True)
        q, k, v = (qkv[:, a * DIM:b * DIM].unflatten(1, (b - a, DIM))
                   for a, b in ((0, Q_HEADS), (Q_HEADS, Q_HEADS + KV_HEADS), (Q_HEADS + KV_HEADS, Q_HEADS + 2 * KV_HEADS)))
        at = torch.arange(n, n + rows, device="cuda")
        sk.kv4_append(k, v, (table[0, at // page] * page + at % page).int(), cache, K_SCALE, V_SCALE)
        lens.fill_(n + rows)
        heads, _ = sk.kv4_attention(q, cache, table, lens, K_SCALE, V_SCALE, DIM ** -0.5, rows=rows)
        y = x + sk.fp8_gemm(heads.flatten(1), *out_w, f16_out=True)
        logits, picks, accept = sk.lm_head_verify(y, head_codes, head_scales, head_g, draft)
        logprob, rank, entropy, ids, top = sk.token_logprobs(logits, picks, top_n=top_n)
        agreed, bonus = (int(a) for a in accept)
        committed = draft[:agreed].tolist() + [bonus]
        for i, token in enumerate(committed):
            report.append((token, float(logprob[i]), int(rank[i]), float(entropy[i]), ids[i].tolist(), top[i].tolist()))
        tokens += committed
        n += agreed + 1
        # The weight of each position, from the accepted rows alone: which they are is known only now, so those rows
        # attend once more, as the last ones of a sequence that ends with them.
        lens.fill_(n)
        sk.kv4_attention(q[:agreed + 1], cache, table, lens, K_SCALE, V_SCALE, DIM ** -0.5, rows=agreed + 1, acc=acc,
                         acc_out=acc)
    assert sk.last_device_error() == sk.SK_OK
    return {"tokens": tokens, "report": report, "length": n, "evictions": evictions, "cache": cache, "table": table,
            "acc": acc}


def main():
    got = decode(int(sys.argv[1]) if len(sys.argv) > 1 else 300)
    for token, lp, rank, entropy, ids, top in got["report"][:8]:
        print(f"token {token:5d}  logprob {lp:8.4f}  rank {rank}  entropy {entropy:.3f}  alternatives {ids}")
    print(f"{len(got['tokens']) - 1} tokens, {got['evictions']} evictions, cache holds {got['length']} positions")


if __name__ == "__main__":
    main()
