"""Operators that pick a small set of weights for each token, as measured cases: a
router's choice of experts and its gradient, tokens sorted by expert and brought
back with weights (and that gradient), and low-rank adapters of many requests
beside a shared projection.

`run` computes a case in its plain form (elementary torch operations in 32
bits) or, with `own` set, through the package's entry points; `exact` restates
each definition in 64 bits.

T tokens have K choices each among E experts; the sorted rows are [T * K, D].
An id of -1 is no choice (or no adapter).
"""

import math

import torch

own = False

DEV = "cuda"
#: The most bytes of rows that a drawn case reads or writes (the largest listed ones move more).
MOST = 400 << 20


# ---------------------------------------------------------------- cases

def listed():
    return [
        # A decode batch's gate: latency.
        dict(name="route decode", op="route", T=64, E=128, k=8, score="softmax", renorm=True, scale=1.0, bf16=True,
             masked=False, train=False),
        # The gate of long prompts, independent scores that are made to sum to a constant.
        dict(name="route prompt", op="route", T=16384, E=256, k=8, score="sigmoid", renorm=True, scale=2.5, bf16=False,
             masked=False, train=False),
        # A training step of the gate, some experts shut off: the choice and the gradient of the logits.
        dict(name="route train", op="route", T=8191, E=160, k=6, score="softmax", renorm=False, scale=1.0, bf16=False,
             masked=True, train=True),
        # A decode batch's tokens go to their experts: latency.
        dict(name="sort decode", op="sort", T=64, E=128, k=8, D=5120, out_of=0),
        # Prompts go to their experts.
        dict(name="sort prompt", op="sort", T=8192, E=128, k=8, D=5120, out_of=0),
        # A decode batch's results come back: latency.
        dict(name="combine decode", op="combine", T=64, E=128, k=8, D=5120, out_of=0, weighted=True, residual=True),
        # Prompts' results come back, added to the residual stream.
        dict(name="combine prompt", op="combine", T=8192, E=128, k=8, D=5120, out_of=0, weighted=True, residual=True),
        # A training step: gradients of the experts' rows and of the weights; a share of the choices lies elsewhere.
        dict(name="combine train", op="grad", T=4099, E=64, k=6, D=2048, out_of=5),
        # One user's token beside a large projection: latency.
        dict(name="adapters one token", op="lora", M=1, K=5120, N=17408, r=16, n=8, each=1, none=0, wide=0),
        # A decode batch, nearly every request with an adapter of its own, some without one.
        dict(name="adapters decode", op="lora", M=64, K=5120, N=17408, r=16, n=48, each=1, none=7, wide=0),
        # Prompts of five requests, each with its own adapter.
        dict(name="adapters prompts", op="lora", M=8192, K=5120, N=17408, r=16, n=5, each=1639, none=0, wide=0),
        # Larger adapters on the projection back, prompts of odd lengths, the base a slice of a wider output.
        dict(name="adapters ragged", op="lora", M=2049, K=17408, N=5120, r=64, n=9, each=111, none=4, wide=512),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["route", "route", "sort", "sort", "combine", "combine", "grad", "lora", "lora", "lora", "lora"])
    if op == "lora":
        K, N, r = 8 * _log(rng, 16, 2176), _log(rng, 100, 17408), rng.choice([8, 16, 24, 32, 48, 64, 128])
        N = N if rng.random() < 0.3 else max(8, N // 8 * 8)
        M = max(1, min(_log(rng, 1, 8192), MOST // (2 * K + 4 * N)))
        return dict(op=op, M=M, K=K, N=N, r=r, n=_log(rng, 1, 64), each=rng.choice([1, _log(rng, 1, M)]),
                    none=rng.choice([0, 0, 3, 7]), wide=rng.choice([0, 0, 8, 513]))
    E, T = _log(rng, 4, 512), _log(rng, 1, 16384)
    k = rng.randint(1, min(8, E))
    if op == "route":
        return dict(op=op, T=T, E=E, k=k, score=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.5,
                    scale=rng.choice([1.0, 2.5]), bf16=rng.random() < 0.5, masked=rng.random() < 0.4,
                    train=rng.random() < 0.5)
    D = _log(rng, 64, 8192)
    D = D if rng.random() < 0.3 else D // 8 * 8
    T = max(1, min(T, MOST // (2 * k * D)))
    c = dict(op=op, T=T, E=E, k=k, D=D, out_of=rng.choice([0, 0, 2, 5]))
    if op == "combine":
        c.update(weighted=rng.random() < 0.7, residual=rng.random() < 0.5)
    return c


def _held(c):
    """How many of the T * k choices name an expert (every out_of-th one lies elsewhere)."""
    n = c["T"] * c["k"]
    return n - (n // c["out_of"] if c["out_of"] else 0)


def _adapted(c):
    """Rows with an adapter (every none-th request has none), and the adapters in use."""
    req = torch.arange(c["M"]) // c["each"]
    has = (req + 1) % c["none"] != 0 if c["none"] else req >= 0
    rows = int(has.sum())
    return rows, min(c["n"], int(torch.unique(req[has]).numel()))


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    c, op = dict(case), case["op"]
    g = torch.Generator(device=DEV).manual_seed(int(seed))

    def rand(*shape):
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)

    s = {"case": c}
    if op == "lora":
        M, K, N, r, n = (c[x] for x in ("M", "K", "N", "r", "n"))
        s["x"] = rand(M, K)
        s["A"] = rand(n, r, K) * K ** -0.5
        s["B"] = rand(n, N, r) * r ** -0.5
        s["scale"] = torch.rand(n, generator=g, device=DEV) + 0.5
        s["base"] = rand(M, N + c["wide"])[:, :N]
        req = torch.arange(M, device=DEV) // c["each"]
        # requests take the adapters in a random order, around and around
        order = torch.randperm(n, generator=g, device=DEV)
        has = (req + 1) % c["none"] != 0 if c["none"] else req >= 0
        if c["none"]:
            req = req - (req + 1) // c["none"]
        s["adapter"] = torch.where(has, order[req % n], -1).int()
        return s
    T, E, k = c["T"], c["E"], c["k"]
    if op == "route":
        x = torch.randn((T, E), generator=g, device=DEV) * 1.5 + torch.randn(E, generator=g, device=DEV)
        if c["masked"]:
            x.masked_fill_(torch.rand((T, E), generator=g, device=DEV) < 0.3, -math.inf)
        s["logits"] = x.bfloat16() if c["bf16"] else x
        s["dw"] = torch.randn((T, k), generator=g, device=DEV)
        return s
    D, n = c["D"], T * k
    # different experts for each token, some of them chosen more often, as a gate does
    s["ids"] = torch.topk(torch.randn((T, E), generator=g, device=DEV) + torch.randn(E, generator=g, device=DEV), k,
                          1).indices.int()
    if c["out_of"]:
        s["ids"].view(-1)[c["out_of"] - 1::c["out_of"]] = -1
    if op == "sort":
        s["x"] = rand(T, D)
        s["out"] = torch.zeros((n, D), device=DEV, dtype=torch.bfloat16)
        return s
    s["slots"] = _slots(s["ids"], E)[0]
    s["y"] = rand(n, D)
    s["w"] = torch.rand((T, k), generator=g, device=DEV) / k
    if op == "combine":
        s["w"] = s["w"] if c["weighted"] else None
        s["residual"] = rand(T, D) if c["residual"] else None
    else:
        s["dout"] = rand(T, D)
        s["dy"] = torch.zeros((n, D), device=DEV, dtype=torch.bfloat16)
    return s


# ---------------------------------------------------------------- plain forms

def _slots(ids, E):
    """Each choice's row among those sorted by expert (-1 for no expert), and the experts' first rows."""
    e = ids.reshape(-1).long()
    held = (e >= 0) & (e < E)
    e = torch.where(held, e, E)
    order = torch.argsort(e, stable=True)
    slots = torch.empty_like(e)
    slots[order] = torch.arange(e.numel(), device=e.device)
    counts = torch.zeros(E + 1, device=e.device, dtype=torch.int64).index_add_(0, e, torch.ones_like(e))
    offsets = torch.cumsum(counts, 0) - counts
    return torch.where(held, slots, -1).int().view(ids.shape), offsets.int()


def _scores(x, c):
    """Scores of float logits over the last axis."""
    if c["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    m = x.amax(1, keepdim=True)
    e = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    l = e.sum(1, keepdim=True)
    return torch.where(l > 0, e / l, 0.0)


def _route(s):
    c, x = s["case"], s["logits"].float()
    E = x.shape[1]
    bits = (x + 0.0).view(torch.int32)
    key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() * (1 << 32) + (E - 1 - torch.arange(E, device=DEV))
    ids = E - 1 - (torch.topk(key, c["k"], 1).values & 0xFFFFFFFF)
    held = x.gather(1, ids) > -math.inf
    score = _scores(x, c)
    p = torch.where(held, score.gather(1, ids), 0.0)
    total = p.sum(1, keepdim=True)
    w = torch.where(total > 0, p / total, 0.0) if c["renorm"] else p
    out = (torch.where(held, ids, -1).int(), w * c["scale"])
    if not c["train"]:
        return out
    g = torch.where(held, s["dw"], 0.0) * c["scale"]
    if c["score"] == "softmax" and not c["renorm"]:
        d = score * (torch.zeros_like(x).scatter_add_(1, ids, g) - (g * p).sum(1, keepdim=True))
    else:
        if c["renorm"]:
            g = w * (g - (g * w).sum(1, keepdim=True))
        elif c["score"] == "sigmoid":
            g = g * p
        if c["score"] == "sigmoid":
            g = g * (1.0 / (1.0 + torch.exp(x.gather(1, ids))))
        d = torch.zeros_like(x).scatter_add_(1, ids, torch.where(held, g, 0.0))
    return out + (d.to(s["logits"].dtype),)


def _sort(s):
    c = s["case"]
    slots, offsets = _slots(s["ids"], c["E"])
    at = slots.view(-1)
    held = torch.nonzero(at >= 0)[:, 0]
    s["out"][at[held].long()] = s["x"][held // c["k"]]
    return s["out"], offsets, slots


def _rows(s):
    """The sorted rows of every choice, [T, k, D] in 32 bits; zeros for no expert."""
    y = s["y"][s["slots"].long().clamp(min=0)].float()
    return torch.where((s["slots"] >= 0)[:, :, None], y, 0.0)


def _combine(s):
    y = _rows(s)
    if s["w"] is not None:
        y = y * s["w"][:, :, None]
    y = y.sum(1)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.bfloat16()


def _grad(s):
    g = s["dout"].float()[:, None]
    dw = (_rows(s) * g).sum(2)
    held = s["slots"] >= 0
    s["dy"][s["slots"][held].long()] = (g * s["w"][:, :, None]).bfloat16()[held]
    return s["dy"], dw


def _lora(s):
    y = s["base"].float()
    for a in range(s["A"].shape[0]):
        rows = torch.nonzero(s["adapter"] == a)[:, 0]
        h = s["x"][rows].float() @ s["A"][a].float().T
        y[rows] += (h * s["scale"][a]) @ s["B"][a].float().T
    return y.bfloat16()


PLAIN = {"route": _route, "sort": _sort, "combine": _combine, "grad": _grad, "lora": _lora}


# ---------------------------------------------------------------- the package's entry points

def _own(s):
    import weight_only_int2_gb300 as wq

    c, op = s["case"], s["case"]["op"]
    if op == "route":
        how = dict(score=c["score"], renormalize=c["renorm"], scale=c["scale"])
        ids, w = wq.moe_route(s["logits"], c["k"], **how)
        if not c["train"]:
            return ids, w
        return ids, w, wq.moe_route_grad(s["logits"], ids, s["dw"], **how)
    if op == "sort":
        return wq.moe_sort(s["x"], s["ids"], c["E"], out=s["out"])
    if op == "combine":
        return wq.moe_combine(s["y"], s["slots"], s["w"], residual=s["residual"])
    if op == "grad":
        return wq.moe_combine_grad(s["dout"], s["y"], s["slots"], s["w"], dy=s["dy"])
    return wq.lora_gemm(s["x"], s["A"], s["B"], s["adapter"], s["base"], scale=s["scale"])


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c, op = case, case["op"]
    if op == "lora":
        rows, used = _adapted(c)
        return {"bytes": 2 * rows * c["K"] + 4 * c["M"] * c["N"] + 2 * used * c["r"] * (c["K"] + c["N"]) + 4 * c["M"],
                "flops": 2 * rows * c["r"] * (c["K"] + c["N"])}
    if op == "route":
        size = 2 if c["bf16"] else 4
        return {"bytes": c["T"] * (c["E"] * size * (2 if c["train"] else 1) + c["k"] * (12 if c["train"] else 8)),
                "flops": 5 * c["T"] * c["E"] * (2 if c["train"] else 1)}
    n, held, row = c["T"] * c["k"], _held(c), 2 * c["D"]
    if op == "sort":
        return {"bytes": c["T"] * row + held * row + 8 * n + 4 * c["E"], "flops": 0}
    if op == "combine":
        return {"bytes": held * row + c["T"] * row * (2 if c["residual"] else 1) + n * (8 if c["weighted"] else 4),
                "flops": 2 * held * c["D"]}
    return {"bytes": c["T"] * row + 2 * held * row + 12 * n, "flops": 3 * held * c["D"]}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    c, op = dict(case), case["op"]
    if op == "sort":
        return None  # whole numbers, and rows that are moved and not computed
    s = prepare(case, seed)
    if op == "lora":
        out = s["base"].double()
        for a in torch.unique(s["adapter"]).tolist():
            if a < 0:
                continue
            at = (s["adapter"] == a).nonzero().view(-1)
            for part in at.split(1024):
                low = torch.einsum("mk,rk->mr", s["x"][part].double(), s["A"][a].double())
                out[part] += s["scale"][a].double() * torch.einsum("mr,nr->mn", low, s["B"][a].double())
        return out
    if op == "route":
        x, k, scale = s["logits"].double(), c["k"], c["scale"]
        best, ids = torch.sort(x, dim=1, descending=True, stable=True)
        best, ids = best[:, :k], ids[:, :k]
        held = best > -math.inf
        if c["score"] == "softmax":
            # (a row of nothing but -inf has no scores: its sums are NaN, and not used)
            log_p = best - torch.logsumexp(best if c["renorm"] else x, 1, keepdim=True)
            slope = torch.ones_like(best)
        else:
            log_p = torch.nn.functional.logsigmoid(best)
            slope = torch.sigmoid(-best)
            if c["renorm"]:
                log_p = log_p - torch.logsumexp(log_p, 1, keepdim=True)
        p = torch.where(held, torch.exp(log_p), 0.0)
        if not c["train"]:
            return None, scale * p
        g = torch.where(held, s["dw"].double(), 0.0) * scale
        mean = (g * p).sum(1, keepdim=True) if c["renorm"] or c["score"] == "softmax" else 0.0
        d = torch.zeros_like(x)
        if c["score"] == "softmax" and not c["renorm"]:
            d -= torch.nan_to_num(torch.softmax(x, 1)) * mean
            mean = 0.0
        d.scatter_add_(1, ids, torch.where(held, p * (g - mean) * slope, 0.0))
        return None, scale * p, d
    T, k, D = c["T"], c["k"], c["D"]
    slots = s["slots"].long()
    if op == "combine":
        out = torch.zeros((T, D), dtype=torch.float64, device=DEV)
        if s["residual"] is not None:
            out += s["residual"].double()
        for j in range(k):
            at = (slots[:, j] >= 0).nonzero().view(-1)
            y = s["y"][slots[at, j]].double()
            out[at] += y if s["w"] is None else y * s["w"][at, j].double()[:, None]
        return out
    dy, dw = s["dy"].double(), torch.zeros((T, k), dtype=torch.float64, device=DEV)
    for j in range(k):
        at = (slots[:, j] >= 0).nonzero().view(-1)
        g = s["dout"][at].double()
        dw[at, j] = torch.linalg.vecdot(g, s["y"][slots[at, j]].double())
        dy[slots[at, j]] = g * s["w"][at, j].double()[:, None]
    return dy, dw
