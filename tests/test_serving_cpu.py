"""CPU checks of the serving operators: pins of their oracle, and the argument
checks of the C ABI, which come before any CUDA call."""

import math
import os

import numpy as np
import pytest
import torch

from oracle import serving as R


# ---------------------------------------------------------------- oracle pins

def test_e4m3_grid_and_rounding():
    v = R.e4m3_values()
    assert v[0x38] == 1.0 and v[0x7E] == 448.0 and v[1] == 2.0 ** -9 and math.isnan(v[0x7F]) and v[0xB8] == -1.0
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(v, codes, equal_nan=True)
    x = np.concatenate([np.linspace(-500, 500, 20011), np.linspace(-0.1, 0.1, 4001), v[:127], (v[:126] + v[1:127]) / 2,
                        [2.0 ** -10, 3 * 2.0 ** -11, 1e-30, -0.0]])
    want = torch.from_numpy(np.clip(x, -448, 448)).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    exact = x.astype(np.float32) == x  # both round the same number
    assert np.array_equal(R.e4m3_codes(x)[exact], want[exact])


def test_attention_oracle_closed_forms():
    r = np.random.default_rng(0)
    kv = r.standard_normal((6, 2, 2, 4, 64))
    table = np.array([[2, 0, 5], [1, -1, -1]], dtype=np.int32)
    q = np.zeros((2, 4, 64))
    out, lse, bad, _ = R.attn_decode(q, kv, table, np.array([10, 3]), 0.5)  # equal scores: the mean, lse = ln n
    flat = np.concatenate([kv[2, 1], kv[0, 1], kv[5, 1][:, :2]], axis=1)
    assert np.allclose(out[0, 1], flat[0].mean(0)) and np.allclose(out[0, 2], flat[1].mean(0))
    assert np.allclose(lse, np.log([[10] * 4, [3] * 4])) and bad == 0
    q = r.standard_normal((2, 4, 64))
    out, lse, _, _ = R.attn_decode(q, kv, table, np.array([10, 1]), 0.5)
    assert np.allclose(out[1, 3], kv[1, 1, 1, 0]) and np.isclose(lse[1, 3], 0.5 * q[1, 3] @ kv[1, 0, 1, 0])
    # a window and the rest join to the whole, weighted by exp(lse)
    w, lw, _, _ = R.attn_decode(q, kv, table, np.array([10, 1]), 0.5, window=4)
    a, la, _, _ = R.attn_decode(q, kv, table, np.array([6, 1]), 0.5)
    f = 1 / (1 + np.exp(la[0] - lw[0]))[:, None]
    assert np.allclose(out[0], f * w[0] + (1 - f) * a[0]) and np.allclose(lse[0], np.logaddexp(lw[0], la[0]))
    # scales of the codes
    s, ls, _, _ = R.attn_decode(q, kv * 4, table, np.array([10, 1]), 0.5, k_scale=[0.25, 0.25], v_scale=[0.5, 0.25])
    assert np.allclose(ls, lse) and np.allclose(s[:, 2:], out[:, 2:]) and np.allclose(s[:, :2], 2 * out[:, :2])
    none, ln, _, _ = R.attn_decode(q, kv, table, np.array([0, -3]), 0.5)
    assert not none.any() and np.all(ln == -np.inf)


def test_logprob_oracle_against_log_softmax():
    x = torch.randn((4, 50), generator=torch.Generator().manual_seed(0), dtype=torch.float64)
    ids = np.array([3, 49, 0, 50])
    lp, rank, ent, top, top_ids, bad = R.token_logprobs(x.numpy(), ids, 5, 0.7)
    y = torch.log_softmax(x / 0.7, 1)
    assert np.allclose(lp[:3], y[torch.arange(3), ids[:3]]) and lp[3] == -np.inf and rank[3] == 0 and bad == 1
    assert np.allclose(ent, -(y.exp() * y).sum(1)) and np.allclose(top, y.topk(5).values)
    assert np.array_equal(top_ids, x.topk(5).indices) and all(rank[:3] == 1 + (x > x[torch.arange(4), [3, 49, 0, 0]][:, None]).sum(1).numpy()[:3])
    flat = R.token_logprobs(np.zeros((1, 8)), [5], 3, 1.0)
    assert np.isclose(flat[0][0], -math.log(8)) and flat[1][0] == 6 and list(flat[4][0]) == [0, 1, 2]
    assert np.isclose(flat[2][0], math.log(8))


def test_page_oracles_by_hand():
    table = np.array([[4, 1, -1], [-1, -1, -1], [3, -1, -1]], dtype=np.int32)
    lens, ref = np.array([6, 0, 4], dtype=np.int32), np.array([0, 1, 0, 1, 1, 0], dtype=np.int32)
    t, n, r, g, moves = R.pages_fork(table, lens, ref, 4, [0], [1])
    assert t[1].tolist() == [4, 0, -1] and n[1] == 6 and r.tolist() == [1, 1, 0, 1, 2, 0] and moves == [(1, 0)]
    t, r, g = R.pages_reserve(table, lens, np.array([13, 9, 8]), ref, 4)  # the first wants more than W * S
    assert g.tolist() == [0, 1, 0] and t[1].tolist() == [0, 2, 5] and r.tolist() == [1, 1, 1, 1, 1, 1]
    n, r, bad = R.pages_free(table, lens, ref, 4, [0, 9])
    assert n.tolist() == [0, 0, 4] and r.tolist() == [0, 0, 0, 1, 0, 0] and bad == 1
    t, r, m, live, moves = R.pages_compact(table, lens, ref, 4)
    assert live == 3 and moves == [(3, 0), (4, 2)] and m.tolist() == [-1, 1, -1, 0, 2, -1]
    assert t[0].tolist() == [2, 1, -1] and t[2].tolist() == [0, -1, -1] and r.tolist() == [1, 1, 1, 0, 0, 0]


# ---------------------------------------------------------------- refusals

@pytest.fixture(scope="module")
def lib():
    import weight_only_int2_gb300 as wq

    if not os.path.exists(wq.LIB_PATH):
        import __graft_entry__

        __graft_entry__.build()
    return wq.load()


@pytest.fixture(scope="module")
def fake():
    """An address that no check below lets a kernel use; with a GPU a real buffer."""
    if torch.cuda.is_available():
        buf = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
        yield buf.data_ptr()
        torch.cuda.synchronize()
    else:
        yield 1 << 20


def refused(lib, name, args, status, word):
    assert getattr(lib, name)(*args) == status, (name, lib.wq_last_error())
    assert word.encode() in lib.wq_last_error(), (word, lib.wq_last_error())


def changed(args, **kw):
    """args (an ordered dict of names) with some replaced, as a list."""
    assert set(kw) <= set(args)
    return list({**args, **kw}.values())


def test_append_refusals(lib, fake):
    p = fake
    ok = dict(k=p, v=p, ks=256, vs=256, T=2, seq=p, pos=p, table=p, B=2, W=2, kv=p, type=0, P=4, Hkv=2, S=16, D=128,
              k_scale=None, v_scale=None, bad=None, stream=None)
    for kw, status, word in [
            (dict(k=None), 1, "k is NULL"), (dict(v=p + 8), 1, "v is not 16"), (dict(ks=248), 1, "k_stride"),
            (dict(vs=260), 1, "v_stride"), (dict(T=-1), 1, "T must"), (dict(pos=None), 1, "pos"),
            (dict(table=p + 2), 1, "block_table"), (dict(B=0), 1, "B must"), (dict(W=0), 1, "W must"),
            (dict(kv=None), 1, "kv is NULL"), (dict(type=2), 1, "kv_type"), (dict(P=0), 1, "P must"),
            (dict(Hkv=0), 1, "Hkv"), (dict(S=0), 1, "S must"), (dict(D=80), 2, "D must"), (dict(type=1), 1, "k_scale"),
            (dict(k_scale=p), 1, "e4m3"), (dict(seq=None, T=3), 1, "seq"), (dict(W=2 ** 28), 1, "W * S"),
            (dict(S=2 ** 30), 1, "page"), (dict(bad=p + 1), 1, "bad_count")]:
        refused(lib, "kv_append", changed(ok, **kw), status, word)
    assert lib.kv_append(*changed(ok, T=0)) == 0


def test_attention_refusals(lib, fake):
    p = fake
    need = lib.kv_attn_workspace_bytes(2, 8, 2, 128)
    ok = dict(q=p, qs=1024, kv=p, type=0, table=p, lens=p, B=2, W=2, P=4, Hq=8, Hkv=2, S=16, D=128, k_scale=None,
              v_scale=None, sm=1.0, window=0, out=p, lse=p, bad=None, ws=p, ws_bytes=need, stream=None)
    for kw, status, word in [
            (dict(q=None), 1, "q is NULL"), (dict(qs=1016), 1, "q_stride"), (dict(qs=1025), 1, "q_stride"),
            (dict(kv=None), 1, "kv"), (dict(type=-1), 1, "kv_type"), (dict(table=None), 1, "block_table"),
            (dict(lens=None), 1, "lens"), (dict(B=-1), 1, "B must"), (dict(P=2 ** 31), 1, "P must"),
            (dict(Hq=7), 1, "multiple"), (dict(D=100), 2, "D must"), (dict(sm=math.inf), 1, "sm_scale"),
            (dict(sm=math.nan), 1, "sm_scale"), (dict(window=-1), 1, "window"), (dict(out=p + 4), 1, "out"),
            (dict(lse=p + 2), 1, "lse"), (dict(type=1, k_scale=p), 1, "v_scale"), (dict(v_scale=p), 1, "e4m3")]:
        refused(lib, "kv_attn_decode", changed(ok, **kw), status, word)
    if need:
        refused(lib, "kv_attn_decode", changed(ok, ws=None), 1, "workspace is NULL")
        refused(lib, "kv_attn_decode", changed(ok, ws_bytes=need - 1), 1, "workspace too small")
    assert lib.kv_attn_decode(*changed(ok, B=0)) == 0
    assert lib.kv_attn_workspace_bytes(0, 8, 2, 128) == 0


def test_page_refusals(lib, fake):
    p = fake
    copy = dict(kv=p, L=1, P=4, size=4096, src=p, dst=p, n=2, bad=None, stream=None)
    for kw, word in [(dict(kv=None), "kv"), (dict(L=0), "L must"), (dict(size=4100), "page_bytes"),
                     (dict(size=0), "page_bytes"), (dict(src=None), "src"), (dict(dst=p + 1), "dst"), (dict(n=-1), "n must")]:
        refused(lib, "kv_pages_copy", changed(copy, **kw), 1, word)
    assert lib.kv_pages_copy(*changed(copy, n=0)) == 0
    need = lib.kv_pages_scratch_bytes(2, 4, 3, 64)
    assert need > 0 and lib.kv_pages_scratch_bytes(-1, 4, 3, 64) == 0
    fork = dict(kv=p, L=1, P=64, size=4096, table=p, lens=p, ref=p, B=4, W=3, S=16, parent=p, child=p, n=2, t=p, l=p,
                r=p, g=p, scratch=p, bytes=need, stream=None)
    for kw, word in [(dict(table=None), "table"), (dict(lens=None), "lens"), (dict(ref=p + 3), "ref"),
                     (dict(n=5), "n must"), (dict(parent=None), "parent"), (dict(child=None), "child"),
                     (dict(t=None), "table_out"), (dict(l=None), "lens_out"), (dict(r=None), "ref_out"),
                     (dict(g=None), "granted"), (dict(scratch=None), "scratch"), (dict(bytes=need - 1), "scratch"),
                     (dict(S=0), "S must"), (dict(W=2 ** 28), "W * S")]:
        refused(lib, "kv_pages_fork", changed(fork, **kw), 1, word)
    need = lib.kv_pages_scratch_bytes(4, 4, 3, 64)
    res = dict(table=p, lens=p, new=p, ref=p, B=4, W=3, S=16, P=64, t=p, r=p, g=p, scratch=p, bytes=need, stream=None)
    for kw, word in [(dict(new=None), "new_lens"), (dict(g=None), "granted"), (dict(bytes=8), "scratch"),
                     (dict(B=0), "B must"), (dict(P=0), "P must")]:
        refused(lib, "kv_pages_reserve", changed(res, **kw), 1, word)
    free = dict(table=p, lens=p, ref=p, B=4, W=3, S=16, P=64, seqs=p, n=2, l=p, r=p, bad=None, stream=None)
    for kw, word in [(dict(seqs=None), "seqs"), (dict(n=5), "n must"), (dict(l=None), "lens_out"), (dict(r=None), "ref_out")]:
        refused(lib, "kv_pages_free", changed(free, **kw), 1, word)
    need = lib.kv_pages_scratch_bytes(0, 4, 3, 64)
    com = dict(kv=p, L=1, P=64, size=4096, table=p, lens=p, ref=p, B=4, W=3, S=16, t=p, r=p, remap=p, n=p, scratch=p,
               bytes=need, stream=None)
    for kw, word in [(dict(remap=None), "remap"), (dict(n=None), "n_live"), (dict(bytes=need - 1), "scratch"),
                     (dict(size=8), "page_bytes")]:
        refused(lib, "kv_pages_compact", changed(com, **kw), 1, word)


def test_logprob_refusals(lib, fake):
    p = fake
    need = lib.token_logprobs_workspace_bytes(2, 1000, 5)
    ok = dict(x=p, type=0, ld=1000, T=2, V=1000, ids=p, temp=1.0, k=5, lp=p, rank=p, ent=p, top=p, tids=p, bad=None,
              ws=p, bytes=need, stream=None)
    for kw, word in [(dict(x=None), "logits"), (dict(x=p + 2), "logits"), (dict(type=3), "logits_type"),
                     (dict(ld=999), "ld must"), (dict(T=-1), "T must"), (dict(V=0), "V must"), (dict(k=33), "top_k"),
                     (dict(k=-1), "top_k"), (dict(V=4, k=5), "top_k"), (dict(temp=0.0), "temperature"),
                     (dict(temp=-1.0), "temperature"), (dict(temp=math.nan), "temperature"),
                     (dict(temp=math.inf), "temperature"), (dict(temp=1e-40), "temperature"), (dict(lp=None), "logprob"),
                     (dict(rank=None), "rank"), (dict(top=None), "top_logprobs"), (dict(tids=p + 1), "top_ids")]:
        refused(lib, "token_logprobs", changed(ok, **kw), 1, word)
    if need:
        refused(lib, "token_logprobs", changed(ok, ws=None), 1, "workspace is NULL")
    assert lib.token_logprobs(*changed(ok, T=0)) == 0


def test_binding_refusals():
    """The Python checks, on CPU tensors, before the library is asked."""
    import weight_only_int2_gb300 as wq

    x = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="kv must be"):
        wq.kv_attn_decode(x, torch.zeros((3, 2, 2, 64)), torch.zeros((2, 1)), torch.zeros(2))
    with pytest.raises(TypeError, match="bfloat16 or float8"):
        wq.kv_append(x, x, x, x, torch.zeros((3, 2, 4, 8, 64)))
    with pytest.raises(ValueError, match="CUDA"):
        wq.kv_pages_copy(torch.zeros((1, 3, 2, 4, 8, 64), dtype=torch.bfloat16), x, x)
    with pytest.raises(ValueError, match="CUDA"):
        wq.token_logprobs(torch.zeros((2, 8)))
