"""GPU checks of the page management calls against the oracle; every result is
a whole number or a moved value, so all comparisons are exact."""

import numpy as np
import pytest
import torch

from oracle import serving as R
from tests.helpers import Guarded

import weight_only_int2_gb300 as wq

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def host(t):
    return t.cpu().numpy()


def pool(L, P, seed, H=1, S=4, D=64, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randint(0, 256, (L, P, 2, H, S, D * (2 if dtype == torch.bfloat16 else 1)), generator=g, device="cuda",
                      dtype=torch.uint8)
    return x.view(dtype)


def raw(kv):
    return kv.view(torch.uint8)


def tables(B, W, S, P, fill, seed, shared=0):
    """Sequences with random lengths that hold about `fill` of the pool, some
    of their pages shared."""
    r = np.random.default_rng(seed)
    ids = list(r.permutation(P)[:int(P * fill)])
    table, lens, ref = np.full((B, W), -1), np.zeros(B), np.zeros(P)
    for b in range(B):
        n = min(int(r.integers(0, W + 1)), len(ids))
        for j in range(n):
            p = ids.pop()
            table[b, j] = p
            ref[p] += 1
        lens[b] = max(0, n * S - int(r.integers(0, S))) if n else 0
    for b in range(min(shared, B)):
        have = -(-int(lens[b]) // S)
        for j in range(have // 2):
            ref[table[b, j]] += 1
    return table.astype(np.int32), lens.astype(np.int32), ref.astype(np.int32)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,W,S,P,fill,n", [(2, 1, 4, 2, 0.5, 1), (9, 7, 4, 40, 0.7, 4), (40, 12, 5, 300, 0.97, 17),
                                           (40, 12, 4, 5000, 0.05, 20), (3000, 3, 1, 9000, 0.5, 1400),
                                           (30, 6, 4, 90, 1.0, 9)])
def test_fork(B, W, S, P, fill, n, in_place):
    table, lens, ref = tables(B, W, S, P, fill, B + P, shared=3)
    r = np.random.default_rng(7)
    rows = r.permutation(B)
    child, parent = rows[:n], r.choice(rows[n:], n)
    for c in child:  # a child holds nothing before
        for j in range(-(-int(lens[c]) // S)):
            ref[table[c, j]] -= 1
        lens[c] = 0
    ref = np.maximum(ref, 0)
    child, parent = child.copy(), parent.copy()
    if n >= 9:
        child[1], parent[2], parent[3], child[4] = -1, B, -7, parent[4]
    want_t, want_l, want_r, want_g, moves = R.pages_fork(table, lens, ref, S, parent, child)
    kv = pool(2, P, 3, S=S)
    want = raw(kv).clone()
    for s, d in moves:
        want[:, d] = raw(kv)[:, s]
    t, l, f = dev(table), dev(lens), dev(ref)
    outs = {} if in_place else {"table_out": torch.empty_like(t), "lens_out": torch.empty_like(l),
                                "ref_out": torch.empty_like(f)}
    got = wq.kv_pages_fork(kv, t, l, f, dev(parent), dev(child), **outs)
    for a, b, what in zip(got, (want_t, want_l, want_r, want_g), ("table", "lens", "ref", "granted")):
        assert np.array_equal(host(a), b), what
    assert torch.equal(raw(kv), want)
    if not in_place:
        assert np.array_equal(host(t), table) and np.array_equal(host(f), ref) and np.array_equal(host(l), lens)
    else:
        assert got[0].data_ptr() == t.data_ptr() and got[2].data_ptr() == f.data_ptr()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,W,S,P,fill", [(1, 1, 1, 1, 0.0), (9, 7, 4, 40, 0.6), (50, 20, 16, 700, 0.9),
                                         (1500, 5, 3, 8000, 0.4), (20, 100, 1, 40000, 0.02), (5, 9, 4, 30, 1.0),
                                         (3, 60000, 2, 200000, 0.3)])
def test_reserve(B, W, S, P, fill, in_place):
    table, lens, ref = tables(B, W, S, P, fill, B + W)
    r = np.random.default_rng(2)
    new = np.minimum(lens + r.integers(0, 3 * S + 1, B), W * S).astype(np.int32)
    new[::3] = np.minimum(W * S, 2 * lens[::3])
    if B > 4:
        new[1], new[2], new[3] = -5, W * S + 1, 2 ** 31 - 1
    want_t, want_r, want_g = R.pages_reserve(table, lens, new, ref, S)
    t, f = dev(table), dev(ref)
    outs = {} if in_place else {"table_out": torch.empty_like(t), "ref_out": torch.empty_like(f)}
    got = wq.kv_pages_reserve(t, dev(lens), dev(new), f, S, **outs)
    for a, b, what in zip(got, (want_t, want_r, want_g), ("table", "ref", "granted")):
        assert np.array_equal(host(a), b), what


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,W,S,P,n", [(1, 1, 4, 3, 1), (9, 7, 4, 40, 5), (300, 40, 16, 9000, 120), (4, 3000, 1, 20000, 3),
                                      (6, 5, 4, 40, 0)])
def test_free(B, W, S, P, n, in_place):
    table, lens, ref = tables(B, W, S, P, 0.8, B, shared=2)
    if n >= 5:
        table[1, 0], table[2, 1] = P, -3
        ref[table[3, 0]] = 0
    seqs = np.random.default_rng(1).permutation(B)[:n].astype(np.int32)
    if n >= 5:
        seqs[0], seqs[1] = -1, B
    want_l, want_r, want_bad = R.pages_free(table, lens, ref, S, seqs)
    l, f, bad = dev(lens), dev(ref), torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = {} if in_place else {"lens_out": torch.empty_like(l), "ref_out": torch.empty_like(f)}
    got = wq.kv_pages_free(dev(table), l, f, dev(seqs), S, bad_count=bad, **outs)
    assert np.array_equal(host(got[0]), want_l) and np.array_equal(host(got[1]), want_r)
    assert int(bad.item()) == want_bad


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,W,S,P,fill", [(1, 1, 4, 1, 1.0), (3, 4, 4, 50, 0.0), (9, 7, 4, 40, 0.6), (50, 20, 16, 700, 0.9),
                                         (700, 5, 3, 3000, 0.4), (5, 900, 1, 30000, 0.2), (30, 40, 4, 1025, 1.0),
                                         (4, 60000, 2, 200000, 0.5)])
def test_compact(B, W, S, P, fill, in_place):
    table, lens, ref = tables(B, W, S, P, fill, B + P, shared=4)
    if B >= 9:
        table[2, 0] = P + 5
    want_t, want_r, want_m, n, moves = R.pages_compact(table, lens, ref, S)
    kv = pool(2 if P < 100000 else 1, P, 3, S=S)
    want = raw(kv).clone()
    if moves:
        s, d = (torch.tensor(v, device="cuda") for v in zip(*moves))
        want[:, d] = raw(kv)[:, s]
    t, f = dev(table), dev(ref)
    outs = {} if in_place else {"table_out": torch.empty_like(t), "ref_out": torch.empty_like(f)}
    got = wq.kv_pages_compact(kv, t, dev(lens), f, **outs)
    for a, b, what in zip(got, (want_t, want_r, want_m, np.array([n])), ("table", "ref", "remap", "n_live")):
        assert np.array_equal(host(a), b), what
    assert torch.equal(raw(kv), want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("L,P,H,S,D,n", [(1, 2, 1, 1, 64, 1), (3, 50, 2, 5, 96, 20), (2, 30, 8, 128, 128, 11),
                                        (1, 4000, 1, 1, 64, 1999)])
def test_copy(L, P, H, S, D, n, dtype):
    kv = pool(L, P, 1, H, S, D, dtype)
    ids = np.random.default_rng(0).permutation(P).astype(np.int32)
    src, dst = ids[:n].copy(), ids[n:2 * n].copy()
    want = raw(kv).clone()
    if n > 4:
        src[0], dst[1], dst[2] = -1, P, -2 ** 31
    ok = (src >= 0) & (dst >= 0) & (dst < P)
    want[:, torch.from_numpy(dst[ok].astype(np.int64)).cuda()] = raw(kv)[:, torch.from_numpy(src[ok].astype(np.int64)).cuda()]
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert wq.kv_pages_copy(kv, dev(src), dev(dst), bad_count=bad).data_ptr() == kv.data_ptr()
    assert torch.equal(raw(kv), want) and int(bad.item()) == int((~ok).sum())
    one = kv[0]
    if n > 4:
        wq.kv_pages_copy(one, dev([3]), dev([4]))
        assert torch.equal(raw(one)[4], raw(one)[3])
        wq.kv_pages_copy(one, dev([]), dev([]))


def test_copy_offsets_beyond_32_bits():
    P, S, D = 5, 2048, 256
    L = (1 << 32) // (P * 2 * 8 * S * D * 2) + 2
    kv = torch.zeros((L, P, 2, 8, S, D), dtype=torch.bfloat16, device="cuda")
    kv[:, 1] = 3.0
    kv[-1, 1, 1, 7, S - 1, D - 1] = 5.0
    wq.kv_pages_copy(kv, dev([1]), dev([4]))
    assert torch.equal(kv[:, 4], kv[:, 1]) and not kv[:, 3].any()


def test_outputs_stay_in_bounds():
    B, W, S, P = 33, 5, 4, 211
    table, lens, ref = tables(B, W, S, P, 0.5, 1)
    t, l, f = Guarded((B, W), torch.int32), Guarded((B,), torch.int32), Guarded((P,), torch.int32)
    m, n, g = Guarded((P,), torch.int32), Guarded((1,), torch.int32), Guarded((B,), torch.int32)
    kv = Guarded((2, P, 2, 1, S, 64), torch.bfloat16)
    wq.kv_pages_compact(kv.t, dev(table), dev(lens), dev(ref), table_out=t.t, ref_out=f.t, remap=m.t, n_live=n.t)
    wq.kv_pages_reserve(dev(table), dev(lens), dev(lens + 9), dev(ref), S, table_out=t.t, ref_out=f.t, granted=g.t)
    wq.kv_pages_free(dev(table), dev(lens), dev(ref), dev(np.arange(B)), S, lens_out=l.t, ref_out=f.t)
    wq.kv_pages_fork(kv.t, dev(table), dev(lens), dev(ref), dev([1, 2]), dev([3, 4]), table_out=t.t, lens_out=l.t,
                     ref_out=f.t)
    for x in (t, l, f, m, n, g, kv):
        x.check()


def test_a_pool_through_its_life():
    """Reserve, fork, free and compact in turn: the counts always equal the
    number of sequences that hold each page, and every sequence keeps its data."""
    L, P, S, B, W = 2, 64, 4, 8, 10
    r = np.random.default_rng(11)
    kv = torch.zeros((L, P, 2, 1, S, 64), dtype=torch.bfloat16, device="cuda")
    table, lens, ref = dev(np.full((B, W), -1)), dev(np.zeros(B)), dev(np.zeros(P))
    content = {b: [] for b in range(B)}  # the value written to each token

    def verify():
        t, n, c = host(table), host(lens), np.zeros(P, dtype=np.int32)
        k = kv[:, :, 0, 0, :, 0].float().cpu().numpy()
        for b in range(B):
            assert n[b] == len(content[b])
            for j in range(-(-int(n[b]) // S)):
                c[t[b, j]] += 1
            for i, v in enumerate(content[b]):
                assert np.all(k[:, t[b, i // S], i % S] == v), (b, i)
        assert np.array_equal(c, host(ref))

    for step in range(40):
        do = ("grow", "grow", "fork", "free", "compact")[step % 5]
        n = host(lens)
        if do == "grow":
            new = np.minimum(n + r.integers(0, 6, B), W * S).astype(np.int32)
            _, _, ok = wq.kv_pages_reserve(table, lens, dev(new), ref, S)
            ok = host(ok)
            seq = [b for b in range(B) if ok[b] for _ in range(n[b], new[b])]
            pos = [i for b in range(B) if ok[b] for i in range(n[b], new[b])]
            if seq:
                vals = torch.arange(len(seq)).float() + step
                x = vals.bfloat16().cuda()[:, None, None].expand(-1, 1, 64).contiguous()
                for layer in range(L):
                    wq.kv_append(x, x, dev(pos), table, kv[layer], seq=dev(seq))
                for b, v in zip(seq, x[:, 0, 0].float().tolist()):
                    content[b].append(v)
            lens.copy_(dev(np.where(ok == 1, np.maximum(n, new), n)))
        elif do == "fork":
            empty = [b for b in range(B) if n[b] == 0]
            full = [b for b in range(B) if n[b] > 0]
            if empty and full:
                child, parent = empty[:2], [int(v) for v in r.choice(full, len(empty[:2]))]
                _, _, _, ok = wq.kv_pages_fork(kv, table, lens, ref, dev(parent), dev(child))
                for a, c, o in zip(parent, child, host(ok)):
                    content[c] = list(content[a]) if o else []
        elif do == "free":
            gone = r.permutation(B)[:3]
            wq.kv_pages_free(table, lens, ref, dev(gone), S)
            for b in gone:
                content[int(b)] = []
        else:
            _, _, _, live = wq.kv_pages_compact(kv, table, lens, ref)
            assert not host(ref)[int(live.item()):].any() and host(ref)[:int(live.item())].all()
        verify()


def test_guarded_outputs_have_the_oracles_values():
    """The calls of test_outputs_stay_in_bounds, one after another into the same outputs, with their values."""
    B, W, S, P = 33, 5, 4, 211
    table, lens, ref = tables(B, W, S, P, 0.5, 1)
    lens[3] = lens[4] = 0
    t, l, f = Guarded((B, W), torch.int32), Guarded((B,), torch.int32), Guarded((P,), torch.int32)
    m, n, g = Guarded((P,), torch.int32), Guarded((1,), torch.int32), Guarded((B,), torch.int32)
    kv = Guarded((2, P, 2, 1, S, 64), torch.bfloat16)

    def equal(*pairs):
        for x, want in pairs:
            x.check()
            assert np.array_equal(host(x.t), want)

    wq.kv_pages_compact(kv.t, dev(table), dev(lens), dev(ref), table_out=t.t, ref_out=f.t, remap=m.t, n_live=n.t)
    want_t, want_r, want_m, live, _ = R.pages_compact(table, lens, ref, S)
    equal((t, want_t), (f, want_r), (m, want_m), (n, [live]))
    wq.kv_pages_reserve(dev(table), dev(lens), dev(lens + 9), dev(ref), S, table_out=t.t, ref_out=f.t, granted=g.t)
    want_t, want_r, want_g = R.pages_reserve(table, lens, lens + 9, ref, S)
    equal((t, want_t), (f, want_r), (g, want_g))
    wq.kv_pages_free(dev(table), dev(lens), dev(ref), dev(np.arange(B)), S, lens_out=l.t, ref_out=f.t)
    want_l, want_r, _ = R.pages_free(table, lens, ref, S, range(B))
    equal((l, want_l), (f, want_r))
    got = wq.kv_pages_fork(kv.t, dev(table), dev(lens), dev(ref), dev([1, 2]), dev([3, 4]), table_out=t.t, lens_out=l.t,
                           ref_out=f.t)
    want_t, want_l, want_r, want_g, _ = R.pages_fork(table, lens, ref, S, [1, 2], [3, 4])
    equal((t, want_t), (l, want_l), (f, want_r))
    assert np.array_equal(host(got[3]), want_g)
