"""GPU checks of kv_append and kv_attn_decode against the float64 oracle.

Tolerances, from the kernel's arithmetic (float32 scores, weights and sums,
weights kept to at least 16 bits in the products, one rounding to bf16):
 - a score is off by at most D 2^-24 A, A the largest sm_scale sum |q k|, and
   by 2^-22 |x| from the scaling, the exponential's argument and itself, so lse
   is off by at most e = (D 2^-24 + 2^-21) A + 2^-18;
 - the output's weights are off by 2 e + 2^-15 in all, its rounding by 2^-8:
   |out - ref| <= 2^-8 |ref| + (2 e + 2^-15) max |v|.
"""

import math

import numpy as np
import pytest
import torch

from oracle import serving as R
from tests.helpers import Guarded

import weight_only_int2_gb300 as wq

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


class Case:
    """A cache with the tables of sequences of the given lengths, its unused
    tokens and pages filled with NaN."""

    def __init__(self, lens, Hkv=2, G=4, D=128, S=16, e4m3=False, seed=0, W=None, spare=3, q_scale=1.0):
        r = np.random.default_rng(seed)
        self.S, self.e4m3 = S, e4m3
        pages = [max(0, -(-n // S)) for n in lens]
        self.W = W or max(1, max(pages, default=1))
        P = sum(pages) + spare
        ids = r.permutation(P)
        self.table = np.full((len(lens), self.W), -1, dtype=np.int32)
        self.lens = np.array(lens, dtype=np.int32)
        codes = np.full((P, 2, Hkv, S, D), 0x7F if e4m3 else 0x7FC0, dtype=np.uint8 if e4m3 else np.uint16)
        at = 0
        for b, n in enumerate(lens):
            for j in range(pages[b]):
                p = ids[at]
                at += 1
                self.table[b, j] = p
                m = min(S, n - j * S)
                x = r.standard_normal((2, Hkv, m, D))
                if e4m3:
                    codes[p, :, :, :m] = R.e4m3_codes(x * 40)
                else:
                    codes[p, :, :, :m] = bf16_bits(x)
        if e4m3:
            self.kv = R.e4m3_values()[codes]
            self.kv_dev = torch.from_numpy(codes).cuda().view(E4M3)
            self.ks, self.vs = ((r.random(Hkv) + 0.5).astype(np.float32) / 40 for _ in range(2))
        else:
            self.kv = bf16_values(codes)
            self.kv_dev = torch.from_numpy(codes.view(np.int16)).cuda().view(torch.bfloat16)
            self.ks = self.vs = None
        q = bf16_bits(r.standard_normal((len(lens), Hkv * G, D)) * q_scale)
        self.q = bf16_values(q)
        self.q_dev = torch.from_numpy(q.view(np.int16)).cuda().view(torch.bfloat16)
        self.sm = 1 / math.sqrt(D)

    def scales(self):
        if not self.e4m3:
            return {}
        return {"k_scale": torch.from_numpy(self.ks).cuda(), "v_scale": torch.from_numpy(self.vs).cuda()}

    def call(self, **kw):
        kw = {"sm_scale": self.sm, "return_lse": True, **self.scales(), **kw}
        return wq.kv_attn_decode(kw.pop("q", self.q_dev), self.kv_dev, torch.from_numpy(self.table).cuda(),
                                 torch.from_numpy(self.lens).cuda(), **kw)

    def check(self, out, lse, window=0, bad=None):
        ref, ref_lse, gone, A = R.attn_decode(self.q, self.kv, self.table, self.lens, self.sm, window, self.ks, self.vs)
        D = self.q.shape[2]
        e = (D * 2.0 ** -24 + 2.0 ** -21) * A + 2.0 ** -18
        top = np.nanmax(np.abs(self.kv[:, 1]), initial=0) * (1 if self.vs is None else self.vs.max())
        out, lse = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
        assert np.array_equal(np.isinf(lse), np.isinf(ref_lse))
        fin = np.isfinite(ref_lse)
        assert np.all(np.abs(lse[fin] - ref_lse[fin]) <= e), np.abs(lse[fin] - ref_lse[fin]).max()
        off = np.abs(out - ref) - 2.0 ** -8 * np.abs(ref)
        assert np.all(off <= (2 * e + 2.0 ** -15) * top), (off.max(), (2 * e + 2.0 ** -15) * top)
        assert np.all(out[~fin] == 0)
        if bad is not None:
            assert int(bad.item()) == gone


def bf16_bits(x):
    u = np.asarray(x, dtype=np.float32).view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def bf16_values(b):
    return (b.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


LENS = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 130, 300, 517]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("G,Hkv", [(1, 3), (5, 2), (8, 1), (12, 2), (16, 1), (23, 2)])
def test_attn_heads(D, G, Hkv, e4m3):
    c = Case(LENS, Hkv=Hkv, G=G, D=D, e4m3=e4m3, seed=D + G)
    c.check(*c.call())


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("S", [1, 3, 8, 17, 48, 64, 100, 256])
def test_attn_page_sizes(S, e4m3):
    c = Case([1, S - 1, S, S + 1, 3 * S + 2, 700, 0], S=S, e4m3=e4m3, seed=S)
    c.check(*c.call())


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 64, 100, 1000, 1 << 40])
def test_attn_window(window):
    c = Case(LENS, seed=window % 97, e4m3=window == 17)
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.check(*c.call(window=window, bad_count=bad), window=window, bad=bad)


@pytest.mark.parametrize("D,G", [(64, 4), (128, 12), (192, 5), (256, 16)])
@pytest.mark.parametrize("window", [1, 15, 16, 31, 32, 33, 127, 129, 1000])
def test_attn_window_of_an_e4m3_cache(window, D, G):
    c = Case(LENS + [31, 32, 33, 1500], S=7, G=G, D=D, seed=window + D, e4m3=True)
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.check(*c.call(window=window, bad_count=bad), window=window, bad=bad)


@pytest.mark.parametrize("B,n,e4m3", [(1, 1, False), (1, 5000, False), (1, 40000, False), (1, 40001, True),
                                     (3, 9001, False), (200, 37, False), (400, 3, True)])
def test_attn_long_and_many(B, n, e4m3):
    c = Case([max(1, n - 11 * b) for b in range(B)], Hkv=2, G=3, e4m3=e4m3, seed=n)
    c.check(*c.call())


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("B,G,Hkv,longest", [(200, 4, 4, 1100), (150, 23, 3, 1100), (200, 4, 4, 900), (450, 1, 2, 70)])
def test_attn_more_items_than_blocks(B, G, Hkv, longest, e4m3):
    """Uneven lengths, some zero, with more (sequence, head) items than blocks fit the GPU."""
    lens = np.random.default_rng(B).integers(0, 120, B)
    lens[[0, B // 2, B - 1]] = 0, longest, longest - 17
    c = Case([int(n) for n in lens], Hkv=Hkv, G=G, e4m3=e4m3, seed=G + longest)
    c.check(*c.call())


def test_attn_large_scores():
    """Scores of some hundreds: weights that differ by more than float32 holds."""
    c = Case([200, 64, 333], q_scale=40.0, seed=9)
    c.check(*c.call())


def test_attn_page_ids_and_lengths_out_of_range():
    c = Case([40, 64, 33, 100, 16], W=9, seed=3)
    P = c.kv.shape[0]
    c.table[0, 1] = -1
    c.table[1, 0] = P
    c.table[2, :] = [2 ** 31 - 1, -2 ** 31, -5, -1, -1, -1, -1, -1, -1]  # nothing left
    c.lens[3] = -7
    c.lens[4] = 2 ** 31 - 1  # counts as W * S: the other pages are out of range
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.check(*c.call(bad_count=bad), bad=bad)


@pytest.mark.parametrize("S", [3, 16, 40])
def test_attn_pages_out_of_range_of_an_e4m3_cache(S):
    c = Case([40, 64, 33, 100, 4 * S], W=-(-160 // S), S=S, D=128, seed=S, e4m3=True)
    c.table[0, 1] = -1
    c.table[1, 0] = c.kv.shape[0]
    c.table[2, :] = -5
    c.lens[4] = 2 ** 31 - 1  # counts as W * S (its last page is full: unused tokens are NaN)
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.check(*c.call(bad_count=bad), bad=bad)


def test_attn_scores_of_minus_infinity():
    c = Case([50, 20], Hkv=1, G=2, seed=4)
    c.kv[c.table[0, :4], 0, :, :, :] = -np.inf
    c.kv_dev[torch.from_numpy(c.table[0, :4].astype(np.int64)).cuda(), 0] = -math.inf
    c.q[:] = np.abs(c.q) + 1
    c.q = bf16_values(bf16_bits(c.q))
    c.q_dev = torch.from_numpy(bf16_bits(c.q).view(np.int16)).cuda().view(torch.bfloat16)
    out, lse = c.call()
    assert torch.all(out[0] == 0) and torch.all(lse[0] == -math.inf)
    ref, ref_lse, _, _ = R.attn_decode(c.q[1:], c.kv, c.table[1:], c.lens[1:], c.sm)
    assert np.abs(lse[1].cpu().numpy() - ref_lse[0]).max() < 1e-3
    # NaN in a stored value reaches the result of its sequence and no other's
    c.kv_dev[c.table[1, 0], 1, 0, 3, 5] = math.nan
    out2, _ = c.call()
    assert torch.isnan(out2[1, :, 5]).all() and not torch.isnan(out2[1, :, :5]).any()
    assert torch.equal(out2[0], out[0])


def test_attn_strided_queries_and_guarded_outputs():
    c = Case([5, 100, 33], Hkv=2, G=4, seed=5)
    wide = torch.full((3, 8 * 128 + 2 * 2 * 128), math.nan, dtype=torch.bfloat16, device="cuda")
    wide[:, :1024] = c.q_dev.view(3, 1024)
    out, lse = Guarded((3, 8, 128), torch.bfloat16), Guarded((3, 8), torch.float32)
    c.check(*c.call(q=wide[:, :1024].unflatten(1, (8, 128)), out=out.t, lse=lse.t))
    out.check("out")
    lse.check("lse")


def test_attn_repeats_and_streams():
    """The same bits again and again: alone, after other shapes on the same
    workspace, on another stream, and in a graph."""
    c = Case([3000, 1, 777, 12000], Hkv=2, G=5, seed=6)
    out, lse = c.call()
    other = Case([9, 2000], Hkv=1, G=16, D=256, e4m3=True, seed=7)
    for _ in range(5):
        other.check(*other.call())
        out2, lse2 = c.call()
        assert torch.equal(out, out2) and torch.equal(lse, lse2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out3, lse3 = c.call()
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, out3) and torch.equal(lse, lse3)
    table, lens = torch.from_numpy(c.table).cuda(), torch.from_numpy(c.lens).cuda()
    out4, lse4 = torch.empty_like(out), torch.empty_like(lse)
    need = wq.kv_attn_workspace_bytes(4, 10, 2, 128)
    ws = torch.zeros(max(16, need), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        wq.kv_attn_decode(c.q_dev, c.kv_dev, table, lens, out=out4, lse=lse4, ws=ws)
    for n in (c.lens, np.array([5, 4000 - 3001, 1, 0], dtype=np.int32), c.lens):
        lens.copy_(torch.from_numpy(n))
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, out4) and torch.equal(lse, lse4)


def test_attn_offsets_beyond_32_bits():
    """Pages whose elements lie beyond 2^31 (and bytes beyond 2^32)."""
    H, S, D = 8, 256, 256
    P = (1 << 31) // (2 * H * S * D) + 8
    kv = torch.zeros((P, 2, H, S, D), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    kv[P - 3:] = torch.randn((3, 2, H, S, D), generator=g, device="cuda").bfloat16()
    q = torch.randn((1, 8, D), generator=g, device="cuda").bfloat16()
    table = torch.tensor([[P - 1, P - 3]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([S + 77], dtype=torch.int32, device="cuda")
    out, lse = wq.kv_attn_decode(q, kv, table, lens, return_lse=True)
    small = kv[[P - 1, P - 3]].clone()
    out2, lse2 = wq.kv_attn_decode(q, small, torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"), lens,
                                   return_lse=True)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    x = torch.randn((1, 8, D), generator=g, device="cuda").bfloat16()
    wq.kv_append(x, x, torch.tensor([S + 5], dtype=torch.int32, device="cuda"), table, kv)
    assert torch.equal(kv[P - 3, 0, :, 5], x[0]) and torch.equal(kv[P - 3, 1, :, 5], x[0])


# ---------------------------------------------------------------- append

@pytest.mark.parametrize("D,S,Hkv,T", [(64, 16, 2, 1), (96, 7, 3, 37), (128, 16, 8, 64), (192, 1, 1, 5),
                                      (256, 100, 4, 211)])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("sliced", [False, True])
def test_append(D, S, Hkv, T, e4m3, sliced):
    r = np.random.default_rng(D + T)
    B, W = 5, -(-2 * T // (5 * S)) + 1
    P = B * W + 2
    table = r.permutation(P)[:B * W].reshape(B, W).astype(np.int32)
    at = r.permutation(B * W * S)[:T]
    seq, pos = (at // (W * S)).astype(np.int32), (at % (W * S)).astype(np.int32)
    if T > 8:  # tokens that have no place
        seq[1], seq[2], pos[3], pos[4] = -1, B, -1, W * S
        table[seq[5], pos[5] // S] = P
    bits = bf16_bits(r.standard_normal((T, 2, Hkv, D)) * 3)
    bits[0, 0, 0, :6] = [0x0000, 0x8000, 0x7F80, 0xFF80, 0x7FC0, 0x4780]  # 0, -0, inf, -inf, NaN, 65536
    ks, vs = ((r.random(Hkv) + 0.5).astype(np.float32) / 30 for _ in range(2))
    x = torch.from_numpy(bits.view(np.int16)).cuda().view(torch.bfloat16)
    k, v = (x[:, 0], x[:, 1]) if sliced else (x[:, 0].contiguous(), x[:, 1].contiguous())
    kv = Guarded((P, 2, Hkv, S, D), E4M3 if e4m3 else torch.bfloat16)
    want = kv.t.view(torch.uint8 if e4m3 else torch.int16).cpu().numpy().copy()
    vals = bf16_values(bits)
    bad = 0
    for t, (page, slot) in enumerate(R.token_places(table, P, S, seq, pos)):
        if page < 0:
            bad += 1
            continue
        for i, w in ((0, ks), (1, vs)):
            if e4m3:
                y = vals[t, i].astype(np.float32) / w[:, None]  # one IEEE division
                c = R.e4m3_codes(np.nan_to_num(y.astype(np.float64), nan=0.0))
                want[page, i, :, slot] = np.where(np.isnan(y), 0x7F, c)
            else:
                want[page, i, :, slot] = bits[t, i].view(np.int16)
    count = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = {"k_scale": torch.from_numpy(ks).cuda(), "v_scale": torch.from_numpy(vs).cuda()} if e4m3 else {}
    wq.kv_append(k, v, torch.from_numpy(pos).cuda(), torch.from_numpy(table).cuda(), kv.t,
                 seq=torch.from_numpy(seq).cuda(), bad_count=count, **kw)
    got = kv.t.view(torch.uint8 if e4m3 else torch.int16).cpu().numpy()
    if e4m3:  # either NaN code is a NaN
        got, want = (np.where((a & 127) == 127, 127, a) for a in (got, want))
    assert np.array_equal(got, want)
    assert int(count.item()) == bad
    kv.check("cache")


@pytest.mark.parametrize("Hkv", [2, 40])
def test_append_every_bf16_value(Hkv):
    """All 65536 patterns by scales from 2^-126 to 2^100, with one or two tokens a thread and an odd number of them."""
    T, D, S = 1025, 64, 16
    W = -(-T // S)
    r = np.random.default_rng(Hkv)
    bits = np.resize(np.arange(65536, dtype=np.uint16), (T, D))
    ks, vs = (np.exp2(r.uniform(-12, 4, Hkv)).astype(np.float32) for _ in range(2))
    ks[0], vs[0], ks[1], vs[1] = 2.0 ** -126, 2.0 ** 100, 1e-30, 1.0
    x = torch.from_numpy(np.broadcast_to(bits.view(np.int16)[:, None], (T, Hkv, D)).copy()).cuda().view(torch.bfloat16)
    kv = torch.zeros((W, 2, Hkv, S, D), dtype=torch.uint8, device="cuda").view(E4M3)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    wq.kv_append(x, x, pos, torch.arange(W, dtype=torch.int32, device="cuda")[None], kv,
                 seq=torch.zeros(T, dtype=torch.int32, device="cuda"),
                 k_scale=torch.from_numpy(ks).cuda(), v_scale=torch.from_numpy(vs).cuda())
    got = kv.view(torch.uint8).permute(0, 3, 1, 2, 4).reshape(W * S, 2, Hkv, D)[:T].cpu().numpy()
    vals = bf16_values(bits).astype(np.float32)
    for i, scales in ((0, ks), (1, vs)):
        for h in range(Hkv):
            with np.errstate(over="ignore", invalid="ignore"):
                y = vals / scales[h]
            want = np.where(np.isnan(y), 127, R.e4m3_codes(np.nan_to_num(y.astype(np.float64), nan=0.0, posinf=1e300, neginf=-1e300)))
            assert np.array_equal(np.where((got[:, i, h] & 127) == 127, 127, got[:, i, h]), want), (i, h)


def test_append_without_seq_and_empty():
    kv = torch.zeros((4, 2, 2, 8, 64), dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
    x = torch.randn((2, 2, 64), device="cuda").bfloat16()
    pos = torch.tensor([8, 3], dtype=torch.int32, device="cuda")
    wq.kv_append(x, x * 2, pos, table, kv)
    assert torch.equal(kv[1, 0, :, 0], x[0]) and torch.equal(kv[2, 1, :, 3], x[1] * 2)
    before = kv.clone()
    wq.kv_append(x[:0], x[:0], pos[:0], table, kv)
    assert torch.equal(kv, before)
    out = wq.kv_attn_decode(x[:0], kv, table[:0], pos[:0])
    assert out.shape == (0, 2, 64)


def test_a_captured_step_follows_its_inputs():
    """Append, attention and log probabilities in one CUDA graph, replayed after the inputs changed."""
    g = torch.Generator().manual_seed(3)
    B, W, S, Hkv, D = 3, 40, 16, 2, 64
    kv = torch.randn((B * W, 2, Hkv, S, D), generator=g).bfloat16().cuda()
    table = torch.randperm(B * W, generator=g).int().reshape(B, W).cuda()
    k, v, q = (torch.zeros((B, h, D), dtype=torch.bfloat16, device="cuda") for h in (Hkv, Hkv, 4 * Hkv))
    pos, lens, ids = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(3))
    logits = torch.zeros((B, 5003), dtype=torch.bfloat16, device="cuda")

    def step(kv):
        wq.kv_append(k, v, pos, table, kv)
        return wq.kv_attn_decode(q, kv, table, lens, return_lse=True) + wq.token_logprobs(logits, ids, top_k=3)

    mine = kv.clone()
    step(mine)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(mine)
    mine.copy_(kv)
    for n in (1, 17, 500, W * S):
        for x in (k, v, q, logits):
            x.copy_(torch.randn(x.shape, generator=g).bfloat16())
        lens.copy_(torch.tensor([n, max(0, n - 5), 1]))
        pos.copy_((lens - 1))
        ids.copy_(torch.randint(0, 5003, (B,), generator=g))
        graph.replay()
        want = step(kv)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert torch.equal(mine, kv)


def test_captured_calls_have_scratch_of_their_own():
    """A replay leaves the buffers of uncaptured calls alone, whatever ran on its stream before."""
    from weight_only_int2_gb300 import _lib

    g = torch.Generator().manual_seed(4)
    kv = torch.randn((64, 2, 2, 128, 64), generator=g).bfloat16().cuda()
    table = torch.randperm(64, generator=g).int()[None].cuda()
    lens = torch.tensor([64 * 128 - 3], dtype=torch.int32, device="cuda")
    q = torch.randn((1, 8, 64), generator=g).bfloat16().cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = wq.kv_attn_decode(q, kv, table, lens)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = wq.kv_attn_decode(q, kv, table, lens)
    for b in _lib._ws_cache.values():
        b.zero_()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert all(not bool(b.any()) for b in _lib._ws_cache.values())


@pytest.mark.parametrize("captured", [False, True])
def test_inputs_from_another_stream(captured):
    """Lengths and tokens that another stream's kernels have just written, behind an event."""
    g = torch.Generator().manual_seed(6)
    B, W, S, Hkv, D = 4, 64, 16, 2, 64
    kv = torch.randn((B * W, 2, Hkv, S, D), generator=g).bfloat16().cuda()
    table = torch.randperm(B * W, generator=g).int().reshape(B, W).cuda()
    q = torch.randn((B, 8, D), generator=g).bfloat16().cuda()
    k = torch.randn((B, Hkv, D), generator=g).bfloat16().cuda()
    lens, pos = (torch.ones(B, dtype=torch.int32, device="cuda") for _ in range(2))
    slow = torch.ones((2048, 2048), device="cuda")
    side = torch.cuda.Stream()

    def step(kv):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            y = slow @ slow  # 2048 in every place
            pos.copy_((y[0, :B] / 4).int() + torch.arange(B, device="cuda", dtype=torch.int32))
            lens.copy_(pos + 1)
        torch.cuda.current_stream().wait_stream(side)
        wq.kv_append(k, k, pos, table, kv)
        return wq.kv_attn_decode(q, kv, table, lens)

    mine = kv.clone()
    n = 512 + torch.arange(B, dtype=torch.int32, device="cuda")
    wq.kv_append(k, k, n, table, kv)
    want = wq.kv_attn_decode(q, kv, table, n + 1)
    torch.cuda.synchronize()
    if captured:
        step(mine.clone())
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step(mine)
        for _ in range(5):
            lens.fill_(1)
            pos.fill_(0)
            graph.replay()
            assert torch.equal(got, want)
        assert torch.equal(mine, kv)
    else:
        for _ in range(20):
            lens.fill_(1)
            pos.fill_(0)
            assert torch.equal(step(mine), want)
        assert torch.equal(mine, kv)


# ---------------------------------------------------------------- weights of very different sizes

GAPS = [12.0, 13.0, 14.5, 16.0, 17.25, 17.375, 18.5, 20.0, 22.0, 30.0, 45.0, 60.0]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D,G", [(64, 4), (128, 8), (128, 12), (256, 4)])
@pytest.mark.parametrize("n", [77, 1000, 32768])
@pytest.mark.parametrize("where", [0.0, 0.5, 1.0])
def test_attn_small_weights(where, n, D, G, e4m3):
    """One token whose weight is all but 1 and whose value is 0: the output is the others' alone, each with a weight
    of e^-gap. All values are positive, so the sum's relative error is at most a weight's: e as above (A the
    gap) for itself and for l, 2^-17 for its two parts, 2^-24 n for n additions' worst case, 2^-8 for the result."""
    S, B = 64, -(-len(GAPS) // G)
    W = -(-n // S)
    r = np.random.default_rng(n + D)
    codes = r.integers(0x30, 0x48, (W, 2, 1, S, D)).astype(np.uint8)  # 0.5 .. 4
    codes[:, 0] = 0
    top = int(where * (n - 1))
    codes[top // S, 0, 0, top % S, 0] = 0x38  # 1
    codes[top // S, 1, 0, top % S] = 0
    values = R.e4m3_values()[codes]
    kv = torch.from_numpy(codes).cuda().view(E4M3)
    kw = {"k_scale": torch.ones(1, device="cuda"), "v_scale": torch.ones(1, device="cuda")} if e4m3 else {}
    kv = kv if e4m3 else torch.from_numpy(values).bfloat16().cuda()
    gaps = np.resize(np.array(GAPS), (B, G))
    q = np.zeros((B, G, D))
    q[:, :, 0] = gaps
    table = torch.arange(W, dtype=torch.int32, device="cuda").expand(B, W).contiguous()
    out = wq.kv_attn_decode(torch.from_numpy(q).bfloat16().cuda(), kv, table,
                            torch.full((B,), n, dtype=torch.int32, device="cuda"), sm_scale=1.0, **kw)
    total = values[:, 1, 0].reshape(W * S, D)[:n].sum(0)
    w = np.exp(-gaps)[..., None]
    ref = w * total / (1 + (n - 1) * w)
    e = (D * 2.0 ** -24 + 2.0 ** -21) * gaps[..., None] + 2.0 ** -18
    off = np.abs(out.double().cpu().numpy() - ref) / ref
    assert np.all(off <= 2.0 ** -8 + 2 * e + 2.0 ** -17 + n * 2.0 ** -24), (off.max((0, 2)), gaps[0])


@pytest.mark.parametrize("D,G", [(64, 4), (128, 5), (128, 16), (192, 3), (256, 12)])
@pytest.mark.parametrize("spread", [3.0, 12.0, 40.0])
def test_attn_steep_scores_of_an_e4m3_cache(spread, D, G):
    """Scores from much less to much more than what came before, by the oracle: every weight in turn the largest."""
    c = Case([64, 333, 2500], G=G, D=D, e4m3=True, q_scale=spread, seed=D + G)
    c.check(*c.call())
    c.kv_dev[c.table[1, 0], 1, 0, 3, 5] = math.nan  # a value of NaN, whichever way the values are widened
    c.kv_dev[c.table[2, 9], 1, 1, 3, 7] = math.nan
    out, _ = c.call()
    assert torch.isnan(out[1, :G, 5]).all() and torch.isnan(out[2, G:, 7]).all()
    assert int(torch.isnan(out).sum()) == 2 * G


@pytest.mark.parametrize("D,G", [(64, 4), (128, 16), (256, 3)])
@pytest.mark.parametrize("power", [-118, -100, -94, 106, 108, 114])
def test_attn_very_large_and_small_queries_of_an_e4m3_cache(power, D, G):
    """Queries times a power of two and sm_scale divided by it: the same bits (2^114 times 8 is below 2^118, and
    no scale leaves the normal numbers)."""
    c = Case([64, 5, 333], G=G, D=D, e4m3=True, seed=D + G)
    # at least 2^-1, so that no query leaves the normal numbers either
    c.q = np.where(np.abs(c.q) < 0.5, np.copysign(0.5, c.q), c.q)
    c.q_dev = torch.from_numpy(c.q).bfloat16().cuda()
    out, lse = c.call()
    c.check(out, lse)
    out2, lse2 = c.call(q=c.q_dev * 2.0 ** power, sm_scale=c.sm * 2.0 ** -power)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("tokens", [1024, 2])
def test_append_every_bf16_value_by_extreme_scales(tokens):
    """All 65536 patterns by positive scales from the smallest number that float32 has to the largest."""
    r = np.random.default_rng(tokens)
    scales = [2.0 ** -149, 3 * 2.0 ** -149, 2.0 ** -141, 2.0 ** -133, 2.0 ** -128, 1e-38, 2.0 ** -126]
    scales += list(np.exp2(r.uniform(-149, -60, 13))) + list(np.exp2(r.uniform(60, 127.9, 11))) + [3.4028234e38]
    H, S, D = len(scales), 16, 64
    ks, vs = np.array(scales, dtype=np.float32), np.array(scales[::-1], dtype=np.float32)
    bits = np.arange(65536, dtype=np.uint16).reshape(1024, D)
    want = []
    for w in (ks, vs):
        with np.errstate(over="ignore", invalid="ignore"):
            y = bf16_values(bits).astype(np.float32)[:, None] / w[None, :, None]
            want.append(np.where(np.isnan(y), 127, R.e4m3_codes(np.nan_to_num(y.astype(np.float64), nan=0.0, posinf=1e300, neginf=-1e300))))
    table = torch.arange(64, dtype=torch.int32, device="cuda")[None]
    for t0 in range(0, 1024, tokens) if tokens > 2 else (0, 254, 510, 768):
        n = min(tokens, 1024 - t0)
        x = torch.from_numpy(np.broadcast_to(bits[t0:t0 + n].view(np.int16)[:, None], (n, H, D)).copy()).cuda().view(torch.bfloat16)
        kv = torch.zeros((64, 2, H, S, D), dtype=torch.uint8, device="cuda").view(E4M3)
        wq.kv_append(x, x, torch.arange(n, dtype=torch.int32, device="cuda"), table, kv,
                     seq=torch.zeros(n, dtype=torch.int32, device="cuda"), k_scale=torch.from_numpy(ks).cuda(),
                     v_scale=torch.from_numpy(vs).cuda())
        got = kv.view(torch.uint8).permute(1, 0, 3, 2, 4).reshape(2, 64 * S, H, D)[:, :n].cpu().numpy()
        for i in range(2):
            bad = np.where((got[i] & 127) == 127, 127, got[i]) != want[i][t0:t0 + n]
            assert not bad.any(), (i, np.unique(np.nonzero(bad)[1]), [scales[::1 - 2 * i][h] for h in np.unique(np.nonzero(bad)[1])])


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T,Hkv,D,S", [(1221, 8, 128, 16), (2501, 8, 128, 17), (2500, 3, 192, 100), (7001, 2, 96, 8)])
def test_append_of_prompts(T, Hkv, D, S, e4m3):
    """So many tokens that a thread has two, odd numbers of them among these, some without a place; the fused
    projection's rows."""
    r = np.random.default_rng(T)
    B = 4
    W = -(-T // (B * S)) + 1
    P = B * W + 1
    table = r.permutation(P)[:B * W].reshape(B, W).astype(np.int32)
    at = np.sort(r.permutation(B * W * S)[:T])
    seq, pos = (at // (W * S)).astype(np.int32), (at % (W * S)).astype(np.int32)
    seq[7], seq[8], pos[T - 1], pos[T - 4] = -1, B, W * S, -3
    table[2, W // 2] = P
    x = torch.from_numpy(r.standard_normal((T, (4 + 2) * Hkv * D)).astype(np.float32)).bfloat16().cuda()
    k = x[:, 4 * Hkv * D:5 * Hkv * D].unflatten(1, (Hkv, D))
    v = x[:, 5 * Hkv * D:].unflatten(1, (Hkv, D))
    ks, vs = ((r.random(Hkv) + 0.5).astype(np.float32) / 60 for _ in range(2))
    kv = Guarded((P, 2, Hkv, S, D), E4M3 if e4m3 else torch.bfloat16)
    raw = torch.uint8 if e4m3 else torch.int16
    want = kv.t.view(raw).cpu().numpy().copy()
    places = R.token_places(table, P, S, seq, pos)
    there = np.array([page >= 0 for page, _ in places])
    page, slot = (np.array(c)[there] for c in zip(*places))
    for i, (y, w) in enumerate(((k, ks), (v, vs))):
        if e4m3:
            q = y.float().cpu().numpy() / w[:, None]  # one IEEE division
            want[page, i, :, slot] = R.e4m3_codes(q.astype(np.float64))[there]
        else:
            want[page, i, :, slot] = y.contiguous().view(torch.int16).cpu().numpy()[there]
    count = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = {"k_scale": torch.from_numpy(ks).cuda(), "v_scale": torch.from_numpy(vs).cuda()} if e4m3 else {}
    wq.kv_append(k, v, torch.from_numpy(pos).cuda(), torch.from_numpy(table).cuda(), kv.t,
                 seq=torch.from_numpy(seq).cuda(), bad_count=count, **kw)
    assert np.array_equal(kv.t.view(raw).cpu().numpy(), want)
    assert int(count.item()) == int((~there).sum())
    kv.check("cache")


@pytest.mark.parametrize("e4m3", [False, True])
def test_every_replay_follows_the_lengths(e4m3):
    """A graph whose lengths change gives after each replay what a call gives that is not captured."""
    c = Case([3000, 1, 777, 12000], Hkv=2, G=5, e4m3=e4m3, seed=6)
    table, lens = torch.from_numpy(c.table).cuda(), torch.from_numpy(c.lens).cuda()
    out, lse = torch.empty_like(c.q_dev), torch.empty((4, 10), device="cuda")
    kw = {"sm_scale": c.sm, **c.scales()}
    wq.kv_attn_decode(c.q_dev, c.kv_dev, table, lens, **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wq.kv_attn_decode(c.q_dev, c.kv_dev, table, lens, out=out, lse=lse, **kw)
    for n in ([3000, 1, 777, 12000], [5, 1, 1, 0], [0, 0, 0, 0], [0, 0, 0, 12000], [2999, 0, 64, 3], [3000, 1, 777, 12000]):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        out.fill_(math.nan)
        lse.fill_(math.nan)
        graph.replay()
        c.lens = np.array(n, dtype=np.int32)
        c.check(out, lse)
        want = wq.kv_attn_decode(c.q_dev, c.kv_dev, table, lens, return_lse=True, **kw)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
