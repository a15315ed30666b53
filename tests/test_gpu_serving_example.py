"""The serving operators together, as examples/serve_quantized.py runs them: the
cached step against attention over all tokens at once, and steps that must not
change when sequences are forked or pages move."""

import importlib.util
import os

import pytest
import torch

import weight_only_int2_gb300 as wq

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_quantized.py")


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("serve_quantized", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("e4m3", [False, True])
def test_example_runs(ex, e4m3):
    r = ex.main(e4m3=e4m3, steps=6, verbose=False)
    assert r["lens"].tolist()[1:4] == [27, 27, 27] and torch.isfinite(r["logits"][1:4].float()).all()
    first = r["history"][0]
    assert first[2][:4].tolist() == [1, 1, 2, 2]  # the best and the second best token
    # the pool is consistent: every page is counted once per sequence that holds it
    count = torch.zeros_like(r["ref"])
    for b, n in enumerate(r["lens"].tolist()):
        for j in range(-(-n // 16)):
            count[r["table"][b, j]] += 1
    assert torch.equal(count, r["ref"])


def test_step_equals_attention_over_all_tokens(ex):
    """Token by token through the cache gives what full causal attention in
    float32 over the same layers gives: the same bf16 layers around it, so the
    logits differ by the bf16 roundings of the attention's output only (2^-8 of
    it, through three more layers: within 2^-5 of the largest logit)."""
    m = ex.Decoder(layers=2)
    S, W, n = 16, 3, 37
    kv = m.cache(8, S)
    table = torch.tensor([[5, 2, 7]], dtype=torch.int32, device="cuda")
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    toks = torch.randint(0, m.vocab, (n,), device="cuda", dtype=torch.int32, generator=torch.Generator("cuda").manual_seed(5))
    got = []
    for i in range(n):
        got.append(m.step(toks[i:i + 1].clone(), kv, table, lens))
        lens += 1
    got = torch.cat(got).float()

    x = wq.qembed_gather(toks, m.embed.packed, m.embed.scales, m.vocab, m.hidden, 8)
    q_dim, kv_dim = m.heads * m.D, m.kv_heads * m.D
    mask = torch.ones((n, n), device="cuda", dtype=torch.bool).tril()
    for layer in m.layers:
        # (one token a call, as the steps ran the layers)
        rows = lambda f, y: torch.cat([f(y[i:i + 1]) for i in range(n)])  # noqa: E731
        qkv = rows(layer["qkv"], ex.norm(x)).float()
        q = qkv[:, :q_dim].view(n, m.heads, m.D)
        k, v = (y.view(n, m.kv_heads, m.D).repeat_interleave(m.heads // m.kv_heads, 1)
                for y in (qkv[:, q_dim:q_dim + kv_dim], qkv[:, q_dim + kv_dim:]))
        s = torch.einsum("qhd,khd->hqk", q, k) * m.D ** -0.5
        a = torch.einsum("hqk,khd->qhd", torch.softmax(s.masked_fill(~mask, -torch.inf), -1), v).bfloat16()
        x = x + rows(layer["o"], a.reshape(n, q_dim))
        gate, up = rows(layer["up"], ex.norm(x)).chunk(2, 1)
        x = x + rows(layer["down"], (torch.nn.functional.silu(gate.float()) * up.float()).bfloat16())
    want = torch.cat([m.head(ex.norm(x)[i:i + 1]) for i in range(n)]).float()
    assert (got - want).abs().max() <= 2.0 ** -5 * want.abs().max()


def test_forked_and_moved_pages_give_the_same_step(ex):
    """A fork's step has the bits of its parent's, and compaction changes none."""
    m = ex.Decoder(layers=2, seed=3)
    S, W, P = 16, 4, 30
    kv = m.cache(P, S)
    i32 = dict(dtype=torch.int32, device="cuda")
    table, lens, ref = torch.full((3, W), -1, **i32), torch.zeros(3, **i32), torch.zeros(P, **i32)
    ref[:7] = 1  # somebody else's
    g = torch.Generator("cuda").manual_seed(2)
    tokens = torch.full((3,), -1, **i32)
    for _ in range(21):
        tokens[0] = torch.randint(0, m.vocab, (1,), generator=g, **i32)
        ex.grow(table, lens, ref, S, tokens)
        m.step(tokens, kv, table, lens)
        lens += (tokens >= 0).int()
    wq.kv_pages_fork(kv, table, lens, ref, torch.tensor([0, 0], **i32), torch.tensor([1, 2], **i32))
    assert ref[table[0, 0]] == 3 and len({int(table[b, 1]) for b in range(3)}) == 3
    tokens[:] = 77
    assert ex.grow(table, lens, ref, S, tokens).tolist() == [1, 1, 1]
    before = m.step(tokens, kv, table, lens)
    assert torch.equal(before[0], before[1]) and torch.equal(before[0], before[2])
    ref[:7] = 0
    _, _, remap, n = wq.kv_pages_compact(kv, table, lens, ref)
    assert int(n) == 4 and sorted(set(table[:, :2].flatten().tolist())) == [0, 1, 2, 3]
    assert torch.equal(m.step(tokens, kv, table, lens), before)


@pytest.mark.parametrize("pages", [4, 5, 6, 7, 40])
def test_a_pool_that_runs_out(ex, pages):
    """Sequences that get no page wait, and nobody's tokens end up in another's pages: what each stored is the
    beginning of what it stores when there are pages for all, and the counts are right."""
    steps = 18
    r, full = (ex.main(steps=steps, verbose=False, pages=n) for n in (pages, 60))
    stored, want = ([[int(h[0][b]) for h in x["history"] if int(h[0][b]) >= 0] for b in range(6)] for x in (r, full))
    for b in range(6):
        assert stored[b] == want[b][:len(stored[b])], b
    lens, want_lens = r["lens"].tolist(), full["lens"].tolist()
    assert all(n <= m for n, m in zip(lens, want_lens))
    assert lens[1] == 21 + len(stored[1]) and lens[0] == 0
    count = torch.zeros_like(r["ref"])
    for b, n in enumerate(lens):
        for j in range(-(-n // 16)):
            count[r["table"][b, j]] += 1
    assert torch.equal(count, r["ref"]) and int((count > 0).sum()) <= pages
    if pages == 40:
        assert lens == want_lens == [0, 39, 39, 39, 0, 0]
    if pages == 4:
        assert lens[2:4] == [0, 0] and len(stored[0]) == steps // 2 + 1
    if pages == 5:
        assert lens[2] > 0 and lens[3] == 0


def test_prompts_that_do_not_fit(ex):
    with pytest.raises(RuntimeError, match="too few pages"):
        ex.main(verbose=False, pages=3)
