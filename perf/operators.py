"""The serving operators around the quantized layers, as measured cases: writing
new keys and values into a paged cache, attention of one new token over it, the
cache's page management, and log probabilities from the logits.

`run` computes a case in its plain form (elementary torch operations in 32
bits) or, with `own` set, through the package's entry points; `exact` restates
each definition in 64 bits.

Shapes: the cache of L layers is kv [L, P, 2, Hkv, S, D] (keys, then values),
a page holding S tokens of every head; block_table [B, W] names the pages of
each sequence in order.
"""

import math

import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
#: The most bytes of keys and values that a drawn attention case reads (the largest listed one reads more).
MOST_KV = 1000 << 20


# ---------------------------------------------------------------- cases

def listed():
    return [
        # One user's short chat: latency of the smallest attention call.
        dict(name="attn one short", op="attn", B=1, Hq=32, Hkv=8, D=128, S=16, lo=77, hi=77, window=0, e4m3=False),
        # A full decode batch at mixed context lengths, one of them a single token.
        dict(name="attn batch", op="attn", B=64, Hq=32, Hkv=8, D=128, S=16, lo=1, hi=8192, window=0, e4m3=False),
        # One very long document: all SMs work on one sequence; five query heads share a key head.
        dict(name="attn one long", op="attn", B=1, Hq=40, Hkv=8, D=128, S=64, lo=131071, hi=131071, window=0,
             e4m3=False),
        # An 8-bit cache with wide heads, few key heads, pages of 48 tokens and a sliding window.
        dict(name="attn e4m3 window", op="attn", B=48, Hq=24, Hkv=4, D=256, S=48, lo=33, hi=20011, window=16384,
             e4m3=True),
        # A decode step's new tokens, the rows still inside the fused projection's output.
        dict(name="append decode", op="append", T=64, B=64, Hq=32, Hkv=8, D=128, S=16, W=2, e4m3=False),
        # Prompts of several sequences written into an 8-bit cache at once.
        dict(name="append prompts e4m3", op="append", T=12289, B=7, Hq=40, Hkv=8, D=128, S=16, W=129, e4m3=True),
        # Parallel samples start from prompts: full pages are shared, the partial last page of each is copied.
        dict(name="pages fork", op="fork", L=8, P=1024, Hkv=2, S=16, D=64, B=24, W=40, n=16, e4m3=False),
        # The bookkeeping of a scheduler step: finished sequences give their pages back, growing ones take new ones.
        dict(name="pages free reserve", op="turn", P=65536, B=256, W=300, S=16, n=40),
        # A half-empty pool is compacted so that its upper half can be given up.
        dict(name="pages compact", op="compact", L=8, P=4096, Hkv=8, S=16, D=128, B=64, W=64, live=2048, e4m3=False),
        # One decoded token over a large vocabulary with its twenty best alternatives: latency.
        dict(name="logprobs one", op="logprobs", T=1, V=248320, k=20, bf16=True, temp=1.0, masked=False),
        # A decode batch of 32-bit logits, some forbidden by a grammar, rows of an odd length.
        dict(name="logprobs batch fp32", op="logprobs", T=96, V=100003, k=8, bf16=False, temp=0.7, masked=True),
        # Every position of a prompt scored over a large vocabulary, as an evaluation does.
        dict(name="logprobs prompt", op="logprobs", T=2049, V=248320, k=5, bf16=True, temp=1.0, masked=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "fork", "turn", "compact", "copy", "logprobs", "logprobs"])
    e4m3 = rng.random() < 0.4
    D, S = rng.choice([64, 96, 128, 192, 256]), rng.choice([8, 16, 17, 32, 48, 64, 100, 128, 256])
    if op == "attn":
        Hkv, G, B = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16]), _log(rng, 1, 128)
        per = 2 * Hkv * D * (1 if e4m3 else 2)
        hi = min(_log(rng, 1, 131072), max(1, MOST_KV // (per * B)))
        lo = rng.randint(0, hi) if rng.random() < 0.7 else hi
        return dict(op=op, B=B, Hq=G * Hkv, Hkv=Hkv, D=D, S=S, lo=lo, hi=hi, e4m3=e4m3,
                    window=_log(rng, 1, hi) if rng.random() < 0.3 else 0)
    if op == "append":
        Hkv, B, W = rng.choice([1, 2, 3, 4, 8]), _log(rng, 1, 128), _log(rng, 1, 128)
        return dict(op=op, T=max(1, min(_log(rng, 1, 12289), B * W * S)), B=B, Hq=Hkv * rng.choice([1, 4, 5]),
                    Hkv=Hkv, D=D, S=S, W=W, e4m3=e4m3)
    if op == "turn":
        B, W, S = _log(rng, 2, 256), _log(rng, 2, 300), rng.choice([8, 16, 17, 64])
        return dict(op=op, P=max(B * W, _log(rng, 64, 65536)), B=B, W=W, S=S, n=rng.randint(1, B // 2))
    if op in ("fork", "compact", "copy"):
        L, Hkv = rng.choice([1, 2, 5, 8]), rng.choice([1, 2, 4, 8])
        page = 2 * Hkv * S * D * (1 if e4m3 else 2)
        P = min(_log(rng, 64, 8192), max(64, (1 << 30) // (L * page)))
        if op == "copy":
            return dict(op=op, L=L, P=P, Hkv=Hkv, S=S, D=D, n=_log(rng, 1, P // 2), e4m3=e4m3)
        if op == "fork":
            B, W = 2 * rng.randint(1, 8), rng.randint(1, 4)
            return dict(op=op, L=L, P=P, Hkv=Hkv, S=S, D=D, B=B, W=W, n=rng.randint(1, B // 2), e4m3=e4m3)
        live, B = rng.randint(1, P), rng.randint(1, 16)
        return dict(op=op, L=L, P=P, Hkv=Hkv, S=S, D=D, B=B, W=-(-live // B) + 1, live=live, e4m3=e4m3)
    V, bf16 = _log(rng, 100, 248320), rng.random() < 0.6
    return dict(op="logprobs", T=max(1, min(_log(rng, 1, 4096), (480_000_000 if bf16 else 240_000_000) // V)), V=V,
                k=rng.choice([0, 1, 5, 20, 32]), bf16=bf16, temp=rng.choice([1.0, 0.7, 1.3]), masked=rng.random() < 0.5)


def _lens(c):
    """An attention case's lengths: evenly spread from lo to hi."""
    return [c["lo"] + (c["hi"] - c["lo"]) * b // max(1, c["B"] - 1) for b in range(c["B"])] if c["B"] > 1 else [c["hi"]]


def _moves(c):
    """Live pages that a compact case has above its live count."""
    return min(c["P"] - c["live"], c["live"], round(c["live"] * (1 - c["live"] / c["P"])))


def _page_bytes(c):
    return 2 * c["Hkv"] * c["S"] * c["D"] * (1 if c["e4m3"] else 2)


# ---------------------------------------------------------------- inputs

def _kv(shape, e4m3, g):
    """A cache's content: N(0, 1) keys and values; in 8 bits with a scale per key head, codes = values / scale."""
    if not e4m3:
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16), None, None
    Hkv = shape[-3]
    ks, vs = ((torch.rand(Hkv, generator=g, device=DEV) + 0.5) / 64 for _ in range(2))
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
    x[..., 0, :, :, :] /= ks[:, None, None].bfloat16()
    x[..., 1, :, :, :] /= vs[:, None, None].bfloat16()
    return x.clamp_(-448, 448).to(E4M3), ks, vs


def _perm(n, g):
    return torch.randperm(n, generator=g, device=DEV).int()


def prepare(case, seed):
    c, op = dict(case), case["op"]
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    s = {"case": c}
    if op == "attn":
        lens = _lens(c)
        pages = [-(-n // c["S"]) for n in lens]
        W, P = max(1, max(pages)), sum(pages) + 3
        s["lens"] = torch.tensor(lens, device=DEV, dtype=torch.int32)[_perm(c["B"], g).long()].contiguous()
        have = (s["lens"] + c["S"] - 1) // c["S"]
        used = torch.arange(W, device=DEV)[None, :] < have[:, None]
        # pages in the random order that a pool in use hands them out; -1 beyond each sequence's last
        s["table"] = torch.full((c["B"], W), -1, device=DEV, dtype=torch.int32)
        s["table"][used] = _perm(P, g)[: sum(pages)]
        s["kv"], s["ks"], s["vs"] = _kv((P, 2, c["Hkv"], c["S"], c["D"]), c["e4m3"], g)
        s["q"] = torch.randn((c["B"], c["Hq"], c["D"]), generator=g, device=DEV, dtype=torch.bfloat16) * 1.5
        s["sm"] = 1.0 / math.sqrt(c["D"])
    elif op == "append":
        H, D, S, W, B, T = c["Hkv"], c["D"], c["S"], c["W"], c["B"], c["T"]
        P = B * W
        s["table"] = _perm(P, g).view(B, W)
        # T different places; a sequence's tokens follow one another where there are more tokens than sequences
        if T <= B:
            seq, pos = _perm(B, g)[:T], torch.randint(0, W * S, (T,), generator=g, device=DEV)
        else:
            each = -(-T // B)
            at = torch.arange(T, device=DEV)
            seq, pos = at // each, at % each
        s["seq"], s["pos"] = seq.int().contiguous(), pos.int().contiguous()
        qkv = torch.randn((T, (c["Hq"] + 2 * H) * D), generator=g, device=DEV, dtype=torch.bfloat16)
        s["k"] = qkv[:, c["Hq"] * D:(c["Hq"] + H) * D].unflatten(1, (H, D))
        s["v"] = qkv[:, (c["Hq"] + H) * D:].unflatten(1, (H, D))
        s["kv"] = torch.zeros((P, 2, H, S, D), device=DEV, dtype=torch.bfloat16)
        s["ks"] = s["vs"] = None
        if c["e4m3"]:
            s["kv"] = s["kv"].to(E4M3)
            s["ks"], s["vs"] = ((torch.rand(H, generator=g, device=DEV) + 0.5) / 64 for _ in range(2))
    elif op == "copy":
        s["kv"], _, _ = _kv((c["L"], c["P"], 2, c["Hkv"], c["S"], c["D"]), c["e4m3"], g)
        ids = _perm(c["P"], g)
        s["src"], s["dst"] = ids[: c["n"]].contiguous(), ids[c["n"]: 2 * c["n"]].contiguous()
    elif op == "fork":
        P, B, W, S, n = c["P"], c["B"], c["W"], c["S"], c["n"]
        s["kv"], _, _ = _kv((c["L"], P, 2, c["Hkv"], S, c["D"]), c["e4m3"], g)
        rows = _perm(B, g)
        child, parents = rows[:n].contiguous(), rows[n:]
        W = max(1, min(W, (P - n) // B))
        s["table"] = torch.full((B, c["W"]), -1, device=DEV, dtype=torch.int32)
        s["lens"] = torch.zeros(B, device=DEV, dtype=torch.int32)
        s["lens"][parents.long()] = torch.randint(1, W * S + 1, (B - n,), generator=g, device=DEV).int()
        used = torch.arange(c["W"], device=DEV)[None, :] < ((s["lens"] + S - 1) // S)[:, None]
        ids = _perm(P, g)
        s["table"][used] = ids[: int(used.sum())]
        s["ref"] = torch.zeros(P, device=DEV, dtype=torch.int32)
        s["ref"][s["table"][used].long()] = 1
        s["child"] = child
        s["parent"] = parents[torch.randint(0, B - n, (n,), generator=g, device=DEV)].contiguous()
        s["out"] = [torch.empty_like(s[k]) for k in ("table", "lens", "ref", "child")]
    elif op == "turn":
        P, B, W, S, n = c["P"], c["B"], c["W"], c["S"], c["n"]
        most = max(1, min(W - 1, P // B - 1))
        s["lens"] = torch.randint(1, most * S + 1, (B,), generator=g, device=DEV).int()
        used = torch.arange(W, device=DEV)[None, :] < ((s["lens"] + S - 1) // S)[:, None]
        s["table"] = torch.full((B, W), -1, device=DEV, dtype=torch.int32)
        s["table"][used] = _perm(P, g)[: int(used.sum())]
        s["ref"] = torch.zeros(P, device=DEV, dtype=torch.int32)
        s["ref"][s["table"][used].long()] = 1
        s["seqs"] = _perm(B, g)[:n].contiguous()
        # what every sequence wants next: its next few tokens; the finished ones nothing
        s["want"] = s["lens"] + torch.randint(1, S + 1, (B,), generator=g, device=DEV).int()
        s["want"][s["seqs"].long()] = 0
        s["out"] = [torch.empty_like(s[k]) for k in ("lens", "ref", "table", "ref", "lens")]
    elif op == "compact":
        P, B, W, S, live, m = c["P"], c["B"], c["W"], c["S"], c["live"], _moves(c)
        s["kv"], _, _ = _kv((c["L"], P, 2, c["Hkv"], S, c["D"]), c["e4m3"], g)
        low, high = _perm(live, g), _perm(P - live, g) + live
        pages = torch.cat([low[m:], high[:m]])[_perm(live, g).long()]
        s["ref"] = torch.zeros(P, device=DEV, dtype=torch.int32)
        # a few pages are shared by two sequences, as after a fork
        each = -(-live // B)
        s["table"] = torch.full((B, W), -1, device=DEV, dtype=torch.int32)
        at = torch.arange(live, device=DEV)
        s["table"][at // each, at % each] = pages
        s["ref"][pages.long()] = 1
        s["ref"][pages[: live // 8].long()] = 2
        count = torch.zeros(B, device=DEV, dtype=torch.int32).index_add_(
            0, at // each, torch.ones_like(at, dtype=torch.int32))
        s["lens"] = (count * S - torch.randint(0, S, (B,), generator=g, device=DEV).int()).clamp_(min=0)
        s["out"] = [torch.empty_like(s["table"]), torch.empty_like(s["ref"]), torch.empty_like(s["ref"]),
                    torch.empty(1, device=DEV, dtype=torch.int32)]
    else:
        T, V = c["T"], c["V"]
        x = torch.randn((T, V), generator=g, device=DEV) * 2.5
        # a few tokens of each row stand out, as a trained model's do
        x.scatter_add_(1, torch.randint(0, V, (T, 8), generator=g, device=DEV),
                       torch.rand((T, 8), generator=g, device=DEV) * 16)
        if c["masked"]:
            x.masked_fill_(torch.rand((T, V), generator=g, device=DEV) < 0.4, -math.inf)
        s["logits"] = x.bfloat16() if c["bf16"] else x
        s["ids"] = torch.randint(0, V, (T,), generator=g, device=DEV).int()
    return s


# ---------------------------------------------------------------- plain forms

def _attn(s):
    c, kv, table, lens = s["case"], s["kv"], s["table"].long(), s["lens"].long()
    B, W = table.shape
    H, S, D = c["Hkv"], c["S"], c["D"]
    got = kv.view(torch.uint8)[table.clamp(min=0)].view(kv.dtype)  # [B, W, 2, H, S, D]
    k, v = (got[:, :, i].permute(0, 2, 1, 3, 4).reshape(B, H, W * S, D).float() for i in (0, 1))
    if c["e4m3"]:
        k, v = k * s["ks"][:, None, None], v * s["vs"][:, None, None]
    at = torch.arange(W * S, device=DEV)[None, :]
    seen = at < lens[:, None]
    if c["window"]:
        seen &= at >= lens[:, None] - c["window"]
    q = s["q"].float().view(B, H, -1, D)
    x = torch.matmul(q, k.transpose(2, 3)) * s["sm"]
    x = torch.where(seen[:, None, None], x, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    l = p.sum(-1, keepdim=True)
    v = torch.where(seen[:, None, :, None], v, 0.0)
    out = torch.where(l > 0, torch.matmul(p, v) / l, 0.0)
    return out.view(B, -1, D).bfloat16(), (m + torch.log(l)).view(B, -1)


def _append(s):
    c, kv = s["case"], s["kv"]
    page = s["table"][s["seq"].long(), s["pos"].long() // c["S"]].long()
    slot = s["pos"].long() % c["S"]
    k, v = s["k"], s["v"]
    if c["e4m3"]:
        k, v = ((x.float() / w[:, None]).clamp(-448, 448).to(E4M3).view(torch.uint8)
                for x, w in ((k, s["ks"]), (v, s["vs"])))
        kv = kv.view(torch.uint8)
    kv[page, 0, :, slot] = k
    kv[page, 1, :, slot] = v
    return s["kv"]


def _bytes(kv):
    return kv.view(torch.uint8) if kv.dtype == E4M3 else kv


def _copy(s):
    kv = _bytes(s["kv"])
    kv[:, s["dst"].long()] = kv[:, s["src"].long()]
    return s["kv"]


def _free_pages(ref):
    """Page ids, the free ones first in ascending order, and how many are free."""
    return torch.argsort((ref != 0).int(), stable=True), (ref == 0).sum()


def _fork(s):
    S, W, P = s["case"]["S"], s["table"].shape[1], s["ref"].numel()
    parent, child, ref, kv = s["parent"].long(), s["child"].long(), s["ref"], _bytes(s["kv"])
    have = s["lens"][parent].long()
    full, need = have // S, (have % S != 0).long()
    ids, count = _free_pages(ref)
    upto = torch.cumsum(need, 0)
    ok = (need == 0) | (upto <= count)
    new = ids[(upto - need).clamp(max=P - 1)]
    rows = s["table"][parent]
    col = torch.arange(W, device=DEV)[None, :]
    shared = (col < full[:, None]) & ok[:, None]
    fresh = (col == full[:, None]) & (ok & (need > 0))[:, None]
    row = torch.where(shared, rows, s["table"][child])
    row = torch.where(fresh, new[:, None].int(), row)
    table, lens, ref = s["table"].clone(), s["lens"].clone(), ref.clone()
    table[child] = row
    lens[child] = torch.where(ok, have, 0).int()
    ref.index_add_(0, rows[shared].long(), torch.ones_like(rows[shared]))
    ref[row[fresh].long()] = 1
    kv[:, row[fresh].long()] = kv[:, rows[fresh].long()]
    return s["kv"], table, lens, ref, ok.int()


def _turn(s):
    S, W, P = s["case"]["S"], s["table"].shape[1], s["ref"].numel()
    seqs, col = s["seqs"].long(), torch.arange(W, device=DEV)[None, :]
    lens, ref = s["lens"].clone(), s["ref"].clone()
    gone = s["table"][seqs][col < ((lens[seqs] + S - 1) // S)[:, None]].long()
    ref.index_add_(0, gone, torch.full_like(gone, -1, dtype=torch.int32))
    lens[seqs] = 0
    have, want = ((x.long() + S - 1) // S for x in (lens, s["want"]))
    need = (want - have).clamp(min=0)
    ids, count = _free_pages(ref)
    upto = torch.cumsum(need, 0)
    ok = (need == 0) | (upto <= count)
    fresh = (col >= have[:, None]) & (col < want[:, None]) & ok[:, None]
    new = ids[((upto - need)[:, None] + col - have[:, None]).clamp(0, P - 1)].int()
    table, ref2 = torch.where(fresh, new, s["table"]), ref.clone()
    ref2[new[fresh].long()] = 1
    return lens, ref, table, ref2, ok.int()


def _compact(s):
    P, S, kv = s["ref"].numel(), s["case"]["S"], _bytes(s["kv"])
    live = s["ref"] != 0
    n = live.sum()
    page = torch.arange(P, device=DEV)
    dst, src = torch.nonzero(~live & (page < n))[:, 0], torch.nonzero(live & (page >= n))[:, 0]
    remap = torch.where(live, page, -1)
    remap[src] = dst
    col = torch.arange(s["table"].shape[1], device=DEV)[None, :]
    used = col < ((s["lens"].long() + S - 1) // S)[:, None]
    table = torch.where(used, remap[s["table"].long().clamp(min=0)].int(), s["table"])
    ref = s["ref"].clone()
    ref[dst] = ref[src]
    ref[src] = 0
    kv[:, dst] = kv[:, src]
    return s["kv"], table, ref, remap.int(), n.int().view(1)


def _logprobs(s):
    c, x, ids = s["case"], s["logits"].float(), s["ids"].long()[:, None]
    V = x.shape[1]
    xt = x.gather(1, ids)
    at = torch.arange(V, device=DEV)[None, :]
    rank = 1 + ((x > xt) | ((x == xt) & (at < ids))).sum(1)
    # the best k: value down, index up; 0.0 and -0.0 are one value
    bits = (x + 0.0).view(torch.int32)
    key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() * (1 << 32) + (V - 1 - at)
    top = (V - 1 - (torch.topk(key, c["k"], 1).values & 0xFFFFFFFF)) if c["k"] else ids[:, :0]
    del key, bits
    best = x.gather(1, top)
    m = x.amax(1, keepdim=True)
    d = (x - m) * (1.0 / c["temp"])
    e = torch.exp(d)
    l = e.sum(1, keepdim=True)
    log_l = torch.log(l)
    entropy = log_l - torch.where(e > 0, e * d, 0.0).sum(1, keepdim=True) / l
    lp = (xt - m) / c["temp"] - log_l
    return lp[:, 0], rank.int(), entropy[:, 0], (best - m) / c["temp"] - log_l, top.int()


PLAIN = {"attn": _attn, "append": _append, "copy": _copy, "fork": _fork, "turn": _turn, "compact": _compact,
         "logprobs": _logprobs}


# ---------------------------------------------------------------- the package's entry points

def _own(s):
    import weight_only_int2_gb300 as wq

    c, op = s["case"], s["case"]["op"]
    if op == "attn":
        return wq.kv_attn_decode(s["q"], s["kv"], s["table"], s["lens"], sm_scale=s["sm"], window=c["window"],
                                 k_scale=s["ks"], v_scale=s["vs"], return_lse=True)
    if op == "append":
        return wq.kv_append(s["k"], s["v"], s["pos"], s["table"], s["kv"], seq=s["seq"], k_scale=s["ks"],
                            v_scale=s["vs"])
    if op == "copy":
        return wq.kv_pages_copy(s["kv"], s["src"], s["dst"])
    if op == "fork":
        table, lens, ref, granted = s["out"]
        return (s["kv"],) + wq.kv_pages_fork(s["kv"], s["table"], s["lens"], s["ref"], s["parent"], s["child"],
                                             table_out=table, lens_out=lens, ref_out=ref, granted=granted)
    if op == "turn":
        lens, ref, table, ref2, granted = s["out"]
        wq.kv_pages_free(s["table"], s["lens"], s["ref"], s["seqs"], c["S"], lens_out=lens, ref_out=ref)
        wq.kv_pages_reserve(s["table"], lens, s["want"], ref, c["S"], table_out=table, ref_out=ref2, granted=granted)
        return lens, ref, table, ref2, granted
    if op == "compact":
        table, ref, remap, n = s["out"]
        return (s["kv"],) + wq.kv_pages_compact(s["kv"], s["table"], s["lens"], s["ref"], table_out=table, ref_out=ref,
                                                remap=remap, n_live=n)
    return wq.token_logprobs(s["logits"], s["ids"], top_k=c["k"], temperature=c["temp"])


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c, op = case, case["op"]
    if op == "attn":
        seen = sum(min(n, c["window"]) if c["window"] else n for n in _lens(c))
        return {"bytes": seen * 2 * c["Hkv"] * c["D"] * (1 if c["e4m3"] else 2)
                + c["B"] * c["Hq"] * (4 * c["D"] + 4) + 4 * (-(-seen // c["S"]) + c["B"]),
                "flops": 4 * seen * c["Hq"] * c["D"]}
    if op == "append":
        n = 2 * c["T"] * c["Hkv"] * c["D"]
        return {"bytes": n * (2 + (1 if c["e4m3"] else 2)) + 12 * c["T"], "flops": n if c["e4m3"] else 0}
    if op == "copy":
        return {"bytes": 2 * c["n"] * c["L"] * _page_bytes(c) + 8 * c["n"], "flops": 0}
    if op == "fork":
        # all but one in S prompts end inside a page; the refs and the rows are read and written
        return {"bytes": int(2 * c["n"] * c["L"] * _page_bytes(c) * (1 - 1 / c["S"])) + 8 * c["P"]
                + 8 * c["B"] * c["W"] + 16 * c["n"], "flops": 0}
    if op == "turn":
        return {"bytes": 16 * c["P"] + 8 * c["B"] * c["W"] + 24 * c["B"], "flops": 0}
    if op == "compact":
        return {"bytes": 2 * _moves(c) * c["L"] * _page_bytes(c) + 12 * c["P"] + 8 * c["B"] * c["W"], "flops": 0}
    n = c["T"] * c["V"]
    return {"bytes": n * (2 if c["bf16"] else 4) + c["T"] * (16 + 8 * c["k"]), "flops": 6 * n}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    c, op = dict(case), case["op"]
    if op in ("copy", "fork", "turn", "compact"):
        return None  # whole numbers, and values that are moved and not computed
    s = prepare(case, seed)
    if op == "append":
        if not c["e4m3"]:
            return None
        kv = s["kv"].double()
        for i, (x, w) in enumerate(((s["k"], s["ks"]), (s["v"], s["vs"]))):
            y = (x.double() / w.double()[:, None]).clamp(-448, 448)
            # round to 4 significant bits, not below the smallest step 2^-9, ties to even
            step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
            y = torch.round(y / step) * step
            p = s["pos"].long()
            kv[s["table"][s["seq"].long(), p // c["S"]].long(), i, :, p % c["S"]] = y
        return kv
    if op == "attn":
        H, G, D, S = c["Hkv"], c["Hq"] // c["Hkv"], c["D"], c["S"]
        out = torch.zeros((c["B"], H, G, D), dtype=torch.float64, device=DEV)
        lse = torch.full((c["B"], H, G), -math.inf, dtype=torch.float64, device=DEV)
        for b, n in enumerate(s["lens"].tolist()):
            first = max(0, n - c["window"]) if c["window"] else 0
            if n <= first:
                continue
            t = torch.arange(first, n, device=DEV)
            page = s["table"][b, t // S].long()
            flat = s["kv"].view(torch.uint8)[page, :, :, t % S].view(s["kv"].dtype).double()  # [t, 2, H, D]
            k, v = flat[:, 0].transpose(0, 1), flat[:, 1].transpose(0, 1)
            if c["e4m3"]:
                k, v = k * s["ks"].double()[:, None, None], v * s["vs"].double()[:, None, None]
            x = torch.bmm(s["q"][b].double().view(H, G, D), k.transpose(1, 2)) * s["sm"]
            lse[b] = torch.logsumexp(x, -1)
            out[b] = torch.bmm(torch.softmax(x, -1), v)
        return out.view(c["B"], -1, D), lse.view(c["B"], -1)
    T, k = c["T"], c["k"]
    lp, ent = (torch.empty(T, dtype=torch.float64, device=DEV) for _ in range(2))
    best = torch.empty((T, k), dtype=torch.float64, device=DEV)
    for t in range(0, T, 256):
        x = s["logits"][t:t + 256].double()
        y = torch.log_softmax(x / c["temp"], 1)
        lp[t:t + 256] = y.gather(1, s["ids"][t:t + 256].long()[:, None])[:, 0]
        ent[t:t + 256] = -torch.where(y > -math.inf, y.exp() * y, 0.0).sum(1)
        best[t:t + 256] = torch.topk(y, k, 1).values
    return lp, None, ent, best, None
