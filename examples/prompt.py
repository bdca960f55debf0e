"""A prompt in pieces and the tokens after it, through two layers whose caches hold 4 bits: the first attends to
everything, the second to a window and the first few tokens.

Of every piece the queries and keys are normed and turned by position, the keys and values go to the cache in the same
pass (kv4_append_rope), and the piece's rows attend to what the cache holds (kv4_chunk_attention). The framework's linear
layers take 1 to 8 rows, so a piece is multiplied by a second, FP16 copy of the weights through PyTorch. Then tokens are
decoded one by one: the linear layers in FP8, the same append, and attention of single rows (kv4_attention,
kv4_window_attention).

    python examples/prompt.py [prompt tokens] [tokens per piece]

The weights are random: the example shows which call reads what, not a language model.
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

HIDDEN, Q_HEADS, KV_HEADS, DIM, ROT, VOCAB = 1024, 8, 2, 128, 64, 4096
K_SCALE = V_SCALE = 0.004        # 1/2688 of the largest key and value expected


def serve(prompt=300, piece=128, tokens=12, window=64, sinks=4, page=32, seed=0):
    """Returns a dict with the picked tokens and, per layer, the cache and its table, and of the prompt's last piece the
    queries and what they attended to."""
    import torch

    import fp8_weight_only_skinny_gb300 as sk

    sk.init()
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=torch.float32)      # noqa: E731
    n_qkv = (Q_HEADS + 2 * KV_HEADS) * DIM
    embed = rand(VOCAB, HIDDEN).half()
    head = sk.nvfp4_quantize((rand(VOCAB, HIDDEN) * HIDDEN ** -0.5).half())
    head_g = float(head[2])
    freqs = sk.rope_frequencies(ROT, 10000.0, "turns", factor=4.0, original=128, high=4.0)
    per = (prompt + tokens + page - 1) // page
    layers = []
    for i in range(2):
        qkv, out = (rand(n_qkv, HIDDEN) * HIDDEN ** -0.5).half(), (rand(HIDDEN, Q_HEADS * DIM) * HIDDEN ** -0.5).half()
        order = torch.randperm(per, generator=gen, device="cuda").int()
        layers.append({"qkv": qkv, "out": out, "qkv8": sk.fp8_quantize(qkv), "out8": sk.fp8_quantize(out),
                       "q_norm": 1 + 0.1 * rand(DIM), "k_norm": 1 + 0.1 * rand(DIM), "table": order[None].contiguous(),
                       "cache": sk.kv4_cache(per, KV_HEADS, DIM, page), "window": 0 if i == 0 else window})
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")

    def turn_and_append(layer, qkv, at):
        q, k, v = (qkv[:, a * DIM:b * DIM].unflatten(1, (b - a, DIM))
                   for a, b in ((0, Q_HEADS), (Q_HEADS, Q_HEADS + KV_HEADS), (Q_HEADS + KV_HEADS, Q_HEADS + 2 * KV_HEADS)))
        slots = (layer["table"][0, at // page] * page + at % page).int()
        # the queries are turned where they lie
        return sk.kv4_append_rope(q, k, v, slots, at.int(), freqs, layer["cache"], K_SCALE, V_SCALE,
                                  q_weight=layer["q_norm"], k_weight=layer["k_norm"], q_out=q)

    ids = torch.randint(0, VOCAB, (prompt,), generator=gen, device="cuda")
    for lo in range(0, prompt, piece):
        hi = min(prompt, lo + piece)
        x = embed[ids[lo:hi]]
        lens.fill_(hi)
        starts = torch.tensor([0, hi - lo], dtype=torch.int32, device="cuda")
        for layer in layers:
            q = turn_and_append(layer, x @ layer["qkv"].T, torch.arange(lo, hi, device="cuda"))
            heads, _ = sk.kv4_chunk_attention(q, layer["cache"], layer["table"], lens, starts, K_SCALE, V_SCALE, DIM ** -0.5,
                                              window=layer["window"], sinks=sinks)
            layer["last"] = (q.clone(), heads.clone())
            x = x + heads.flatten(1) @ layer["out"].T
    x = x[-1:]
    picked = []
    for n in range(prompt, prompt + tokens):
        _, token = sk.lm_head_argmax(x, head[0], head[1], head_g, want_logits=False)
        picked.append(int(token[0]))
        x = embed[token.long()]
        lens.fill_(n + 1)
        for layer in layers:
            q = turn_and_append(layer, sk.fp8_gemm(x, *layer["qkv8"], f16_out=True), torch.arange(n, n + 1, device="cuda"))
            if layer["window"]:
                heads, _ = sk.kv4_window_attention(q, layer["cache"], layer["table"], lens, K_SCALE, V_SCALE, DIM ** -0.5,
                                                   layer["window"], sinks=sinks)
            else:
                heads, _ = sk.kv4_attention(q, layer["cache"], layer["table"], lens, K_SCALE, V_SCALE, DIM ** -0.5)
            layer["token"] = (q.clone(), heads.clone())
            x = x + sk.fp8_gemm(heads.flatten(1), *layer["out8"], f16_out=True)
    assert sk.last_device_error() == sk.SK_OK
    return {"picked": picked, "layers": layers, "sinks": sinks, "positions": prompt + tokens}


def main():
    got = serve(*(int(a) for a in sys.argv[1:3]))
    print("picked", got["picked"])
    print(f"{got['positions']} positions in {[layer['cache'].numel() for layer in got['layers']]} bytes")


if __name__ == "__main__":
    main()
