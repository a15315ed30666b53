"""Serves a small random quantized decoder from a paged key-value cache.

Everything between the tokens going in and the log probabilities coming out runs
through the library: the quantized embedding rows, the quantized linear layers,
the cache and its pages, attention of the new token, and the numbers of the
answer. PyTorch does the norms and the activation, and holds the memory.

    python examples/serve_quantized.py

A user of the library with a scheduler of their own needs `Decoder.step` and the
page calls in `advance` and `main`. A pool may run out: a reserve or a fork says
for each sequence whether it was granted, and only granted tokens may be stored.
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import weight_only_int2_gb300 as wq  # noqa: E402


def norm(x):
    y = x.float()
    return (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)).bfloat16()


class Linear:
    """A random quantized layer: codes, a scale per row and 128 inputs."""

    def __init__(self, n, k, bits, g):
        self.n, self.k, self.bits = n, k, bits
        codes = torch.randint(0, 1 << bits, (n, k), generator=g, device="cuda", dtype=torch.uint8)
        scales = (torch.rand((n, k // 128), generator=g, device="cuda") + 0.5) * 2.0 / ((1 << bits) * k ** 0.5)
        self.packed, self.scales = wq.wna16_repack(codes, scales.bfloat16(), bits)

    def __call__(self, x):
        return wq.wna16_gemm(x, self.packed, self.scales, self.n, self.k, self.bits)


class Decoder:
    def __init__(self, layers=2, hidden=1024, heads=16, kv_heads=4, head_dim=64, inner=2048, vocab=4096, bits=6,
                 e4m3=False, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.heads, self.kv_heads, self.D, self.vocab, self.hidden = heads, kv_heads, head_dim, vocab, hidden
        self.e4m3 = e4m3
        q, kv = heads * head_dim, kv_heads * head_dim
        self.embed = Linear(vocab, hidden, 8, g)
        self.layers = [dict(qkv=Linear(q + 2 * kv, hidden, bits, g), o=Linear(hidden, q, bits, g),
                            up=Linear(2 * inner, hidden, bits, g), down=Linear(hidden, inner, bits, g))
                       for _ in range(layers)]
        self.head = Linear(vocab, hidden, 8, g)
        one = torch.ones(kv_heads, device="cuda")
        self.scales = dict(k_scale=one / 64, v_scale=one / 64) if e4m3 else {}

    def cache(self, pages, page_size):
        """The pages of all layers: [L, P, 2, Hkv, S, D]."""
        kv = torch.zeros((len(self.layers), pages, 2, self.kv_heads, page_size, self.D), device="cuda",
                         dtype=torch.bfloat16)
        return kv.to(torch.float8_e4m3fn) if self.e4m3 else kv

    def step(self, tokens, kv, table, lens):
        """Logits after one more token of every sequence. `lens` counts the
        tokens stored before; the new ones' pages are reserved already. A token
        of -1 leaves its sequence alone (its logits mean nothing)."""
        live = tokens >= 0
        now = torch.where(live, lens + 1, 0)           # what attention sees
        pos = torch.where(live, lens, -1)              # where the new token goes; -1: nowhere
        x = wq.qembed_gather(tokens, self.embed.packed, self.embed.scales, self.vocab, self.hidden, 8)
        q_dim, kv_dim = self.heads * self.D, self.kv_heads * self.D
        for layer, pages in zip(self.layers, kv):
            qkv = layer["qkv"](norm(x))
            q = qkv[:, :q_dim].unflatten(1, (self.heads, self.D))
            k = qkv[:, q_dim:q_dim + kv_dim].unflatten(1, (self.kv_heads, self.D))
            v = qkv[:, q_dim + kv_dim:].unflatten(1, (self.kv_heads, self.D))
            wq.kv_append(k, v, pos, table, pages, **self.scales)
            a = wq.kv_attn_decode(q, pages, table, now, **self.scales)
            x = x + layer["o"](a.view(-1, q_dim))
            gate, up = layer["up"](norm(x)).chunk(2, 1)
            x = x + layer["down"]((torch.nn.functional.silu(gate.float()) * up.float()).bfloat16())
        return self.head(norm(x))


def grow(table, lens, ref, page_size, tokens):
    """Reserves the page that each sequence's next token needs. Returns 1 for the
    sequences that have their page and 0 for those that the pool has none for:
    their token must not be stored, since its place in the table is not theirs."""
    _, _, granted = wq.kv_pages_reserve(table, lens, torch.where(tokens >= 0, lens + 1, lens), ref, page_size)
    return granted


def advance(model, tokens, kv, table, lens, ref, logits):
    """Stores each sequence's next token and computes what follows it. A sequence
    without a page waits: its token becomes -1, its logits stay. Returns the tokens
    that were stored and the logits; lens is updated."""
    granted = grow(table, lens, ref, kv.shape[4], tokens)
    tokens = torch.where(granted == 1, tokens, -1)
    after = model.step(tokens, kv, table, lens)
    lens += (tokens >= 0).int()
    return tokens, torch.where((tokens >= 0)[:, None], after, logits)


def main(e4m3=False, steps=6, verbose=True, pages=40):
    model = Decoder(e4m3=e4m3)
    B, W, S, P = 6, 8, 16, pages
    kv = model.cache(P, S)
    table = torch.full((B, W), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    ref = torch.zeros(P, dtype=torch.int32, device="cuda")
    logits = torch.zeros((B, model.vocab), dtype=torch.bfloat16, device="cuda")

    # two prompts, token by token, in sequences 0 and 1
    g = torch.Generator(device="cuda").manual_seed(1)
    prompts = torch.randint(0, model.vocab, (2, 21), generator=g, device="cuda", dtype=torch.int32)
    tokens = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    n = prompts.shape[1]
    for i in range(n):
        tokens[:2] = prompts[:, i]
        stored, logits = advance(model, tokens, kv, table, lens, ref, logits)
    if lens[:2].min() < n:
        raise RuntimeError("the pool has too few pages for the prompts")

    # each prompt is continued twice: sequences 2 and 3 start as copies, if there is a page for them
    ids = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
    _, _, _, granted = wq.kv_pages_fork(kv, table, lens, ref, ids[0], ids[1])
    logits[2:4] = logits[:2]
    alive = torch.zeros(B, dtype=torch.bool, device="cuda")
    alive[:2] = True
    alive[2:4] = granted == 1
    total = torch.zeros(B, device="cuda")
    history = []
    for i in range(steps):
        # the best token continues 0 and 1, the second best the first step of 2 and 3
        _, _, entropy, best, best_ids = wq.token_logprobs(logits, top_k=2)
        pick = torch.zeros(B, dtype=torch.int64, device="cuda")
        pick[2:4] = lens[2:4] == n
        tokens = torch.where(alive, best_ids.gather(1, pick[:, None])[:, 0], -1)
        lp, rank, _, _, _ = wq.token_logprobs(logits, tokens)
        tokens, logits = advance(model, tokens, kv, table, lens, ref, logits)
        total += torch.where(tokens >= 0, lp, 0.0)
        history.append((tokens, lp, rank, entropy))
        if i == steps // 2:
            # sequence 0 is finished: its pages go back, and the pool closes up
            alive[0] = False
            wq.kv_pages_free(table, lens, ref, torch.zeros(1, dtype=torch.int32, device="cuda"), S)
            _, _, _, n_live = wq.kv_pages_compact(kv, table, lens, ref)
    wq.check_status()
    if verbose:
        for tok, lp, rank, entropy in history:
            print(" ".join("%5d %7.3f (%d)" % x for x in zip(tok[:4].tolist(), lp[:4].tolist(), rank[:4].tolist())))
        print("log probability of each continuation:", [round(v, 3) for v in total[:4].tolist()])
        print("pages in use after compaction:", int(n_live))
    return dict(model=model, kv=kv, table=table, lens=lens, ref=ref, logits=logits, history=history, total=total)


if __name__ == "__main__":
    main(e4m3="--e4m3" in sys.argv[1:])
