"""GPU checks of token_logprobs against the float64 oracle.

Tolerances: with R the row's largest finite |x - m| / temperature, a term's
exponent is off by at most 4 R 2^-24, the sums' terms by 2^-21 of themselves
and their additions by 2^-18, so ln l is off by at most e = 4 R 2^-24 + 2^-17;
a log probability by e + |lp| 2^-22, the entropy by (1 + R) e. Ids and ranks are
exact.
"""

import math

import numpy as np
import pytest
import torch

from oracle import serving as O

import weight_only_int2_gb300 as wq

pytestmark = pytest.mark.gpu


def rows(T, V, bf16, seed, kind="normal"):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, V), generator=g) * 3
    if kind == "masked":
        x[torch.rand((T, V), generator=g) < 0.7] = -math.inf
    elif kind == "ties":
        x = torch.randint(-3, 4, (T, V), generator=g).float() * 0.5
    elif kind == "ascending":
        x = x.sort(1).values
    elif kind == "constant":
        x = torch.full((T, V), 1.5)
    elif kind == "steep":
        x = x * 100
    return x.bfloat16() if bf16 else x


def check(x, ids, k, temp, got, bad=None):
    lp, rank, ent, top, top_ids, gone = O.token_logprobs(x.double().numpy(), ids.numpy(), k, temp)
    a = x.double().numpy()
    with np.errstate(invalid="ignore"):
        d = a - a.max(1, keepdims=True)
    R = np.array([np.max(np.abs(r[np.isfinite(r)]), initial=0.0) / temp for r in d])
    e = 4 * R * 2.0 ** -24 + 2.0 ** -17
    glp, grank, gent, gtop, gids = (v.cpu().numpy() for v in got)
    assert np.array_equal(gids, top_ids)
    assert np.array_equal(grank, rank)

    def near(u, v, tol):
        u = u.astype(np.float64)
        assert np.array_equal(np.isnan(u), np.isnan(v)) and np.array_equal(np.isinf(u), np.isinf(v))
        f = np.isfinite(v)
        assert np.all(np.abs(u - v)[f] <= np.broadcast_to(tol, v.shape)[f]), np.max(np.abs(u - v)[f])

    near(glp, lp, e + np.nan_to_num(np.abs(lp), posinf=0) * 2.0 ** -22)
    near(gtop, top, e[:, None] + np.nan_to_num(np.abs(top), posinf=0) * 2.0 ** -22)
    near(gent, ent, (1 + R) * e)
    if bad is not None:
        assert int(bad.item()) == gone


def run(x, ids, k=0, temp=1.0, **kw):
    return wq.token_logprobs(x.cuda(), ids.cuda(), top_k=k, temperature=temp, **kw)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,V,k", [(1, 1, 1), (3, 2, 2), (2, 31, 5), (5, 33, 32), (4, 1000, 0), (7, 1001, 1),
                                  (1, 50001, 20), (3, 65536, 32), (2, 248320, 8), (200, 4099, 5), (700, 517, 3)])
def test_sizes(T, V, k, bf16):
    x = rows(T, V, bf16, T + V)
    ids = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(V)).int()
    check(x, ids, k, 1.0, run(x, ids, k))


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("kind", ["masked", "ties", "ascending", "constant", "steep"])
@pytest.mark.parametrize("T,V", [(1, 70001), (3, 2050), (170, 9001)])
def test_kinds(kind, T, V, bf16):
    x = rows(T, V, bf16, 5, kind)
    ids = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(V)).int()
    check(x, ids, 32, 0.7, run(x, ids, 32, 0.7))


@pytest.mark.parametrize("temp", [0.05, 0.7, 1.0, 1.9, 100.0])
def test_temperature(temp):
    x = rows(6, 5003, True, 8)
    ids = torch.tensor([0, 5002, 17, 4096, 4095, 1], dtype=torch.int32)
    check(x, ids, 4, temp, run(x, ids, 4, temp))


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,V", [(8, 300), (8, 60000), (400, 300)])
def test_rows_without_weight_and_special_values(T, V, bf16):
    x = rows(T, V, bf16, 3)
    x[0] = -math.inf
    x[1] = -math.inf
    x[1, V // 2] = -5.0
    x[2, 7] = math.nan
    x[2, 3] = math.nan
    x[3, V - 1] = math.inf
    x[4, 5] = math.inf
    x[4, 250] = math.nan
    x[5] = -math.inf
    x[5, 0], x[5, 9], x[5, 20] = -0.0, 0.0, -0.0
    x[6, :] = -1e30
    ids = torch.zeros(T, dtype=torch.int32)
    ids[:8] = torch.tensor([5, V // 2, 7, 0, 250, 20, 299, 4])
    check(x, ids, 6, 1.0, run(x, ids, 6))


def test_ids_out_of_range_and_none():
    x = rows(5, 999, False, 4)
    ids = torch.tensor([-1, 999, 2 ** 31 - 1, -2 ** 31, 998], dtype=torch.int32)
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(x, ids, 3, bad_count=bad)
    check(x, ids, 3, 1.0, got, bad)
    lp, rank, ent, top, top_ids = wq.token_logprobs(x.cuda(), top_k=3)
    assert lp is None and rank is None
    assert torch.equal(ent, got[2]) and torch.equal(top, got[3]) and torch.equal(top_ids, got[4])
    empty = wq.token_logprobs(x[:0].cuda(), ids[:0].cuda(), top_k=2)
    assert empty[0].shape == (0,) and empty[3].shape == (0, 2)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("pad", [1, 3, 8, 13])
@pytest.mark.parametrize("T,V", [(6, 1003), (2, 90007)])
def test_padded_rows(pad, T, V, bf16):
    """Rows of any alignment inside a wider array whose padding holds +inf and NaN."""
    wide = torch.full((T, V + pad), math.inf)
    wide[:, V + pad // 2:] = math.nan
    wide = wide.bfloat16() if bf16 else wide
    x = rows(T, V, bf16, pad)
    wide[:, :V] = x
    ids = torch.full((T,), V - 1, dtype=torch.int32)
    dev = wide.cuda()
    check(x, ids, 7, 1.0, wq.token_logprobs(dev[:, :V], ids.cuda(), top_k=7))


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("kind", ["normal", "masked", "ties", "ascending", "constant"])
@pytest.mark.parametrize("T,V,k", [(9, 700, 32), (1100, 4001, 7), (1040, 2050, 32), (4100, 515, 0)])
def test_many_rows(T, V, k, kind, bf16):
    x = rows(T, V, bf16, 11, kind)
    ids = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(V)).int()
    check(x, ids, k, 1.3, run(x, ids, k, 1.3))


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,V", [(5, 70001), (5, 900), (900, 40003)])
def test_few_logits_above_minus_infinity(T, V, bf16):
    """Less than top_k of a row have weight, wherever they are: -inf follows by id."""
    x = torch.full((T, V), -math.inf)
    x[1, [0, V // 2, V - 1]] = torch.tensor([1.0, -2.0, 1.0])
    x[2, :31] = torch.arange(31.0)
    x[3, V - 40:] = torch.arange(40.0)
    x[4, ::V // 33] = 0.5
    x = x.bfloat16() if bf16 else x
    ids = torch.zeros(T, dtype=torch.int32)
    ids[:5] = torch.tensor([V - 1, 1, 31, V - 40, V // 33])
    check(x, ids, 32, 1.0, run(x, ids, 32))


@pytest.mark.parametrize("V", [62080, 65537, 8193, 16400])
def test_rows_that_end_in_a_short_piece(V):
    x = rows(3, V, True, V)
    ids = torch.tensor([0, V - 1, V // 2], dtype=torch.int32)
    check(x, ids, 32, 1.0, run(x, ids, 32))


def test_repeats_and_streams():
    x, y = rows(3, 130001, True, 1).cuda(), rows(64, 3001, False, 2).cuda()
    ids = torch.tensor([3, 1, 2], dtype=torch.int32, device="cuda")
    first = wq.token_logprobs(x, ids, top_k=9)
    for _ in range(5):
        wq.token_logprobs(y, top_k=32)
        assert all(torch.equal(a, b) for a, b in zip(first, wq.token_logprobs(x, ids, top_k=9)))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = wq.token_logprobs(x, ids, top_k=9)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_offsets_beyond_32_bits():
    V = 250001
    T = (1 << 31) // V + 3
    x = torch.zeros((T, V), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    x[-2:] = torch.randn((2, V), generator=g, device="cuda").bfloat16()
    ids = torch.full((T,), 17, dtype=torch.int32, device="cuda")
    got = wq.token_logprobs(x, ids, top_k=4)
    tail = x[-2:].cpu()
    check(tail, ids[-2:].cpu(), 4, 1.0, [v[-2:] for v in got])
    assert math.isclose(float(got[0][0]), -math.log(V), rel_tol=1e-6)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("S", [250, 1002])
@pytest.mark.parametrize("shares", [1, 2])
def test_rows_that_no_share_cuts(shares, S, captured):
    """As many rows as shares (three blocks an SM), so that no row is joined from parts: the library's next
    kernel, which writes over the logits, begins only after the last of them has been read."""
    T, V = shares * 3 * torch.cuda.get_device_properties(0).multi_processor_count, 128 * S
    g = torch.Generator(device="cuda").manual_seed(S)
    x = torch.randn((2 * T, V), generator=g, device="cuda").bfloat16()
    ids = torch.randint(0, V, (T,), generator=g, device="cuda").int()
    want = wq.token_logprobs(x[:T].clone(), ids, top_k=5)
    torch.cuda.synchronize()
    work = x.clone()
    pages = work.view(2 * T, 2, 1, S, 64)  # a row is a page
    here = torch.arange(T, dtype=torch.int32, device="cuda")

    def step():
        got = wq.token_logprobs(work[:T], ids, top_k=5)
        wq.kv_pages_copy(pages, here + T, here)
        return got

    step()
    torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step()
    for _ in range(10):
        work.copy_(x)
        if captured:
            graph.replay()
        else:
            got = step()
        assert torch.equal(work[:T], x[T:])
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("temp", [0.7, 1.0, 1.3])
@pytest.mark.parametrize("T,V", [(6, 300), (1, 70001), (6, 60000), (700, 4099)])
def test_masks_of_the_lowest_value(T, V, temp, bf16):
    """Logits forbidden by the type's lowest value weigh as little as by -inf, wherever the others lie.

    With R the largest |x - m| / temperature of the others, the tolerances are those above. A forbidden logit's
    log probability is within 2^-20 of (x - m) / temperature - ln l, and -inf where float32 cannot hold it."""
    dtype = torch.bfloat16 if bf16 else torch.float32
    low = torch.finfo(dtype).min
    x = rows(T, V, bf16, 17)
    forbidden = torch.zeros((T, V), dtype=torch.bool)
    for t in range(T):
        kind = t % 6
        if kind == 0:
            forbidden[t, : V // 2] = True
        elif kind == 1:
            forbidden[t, :-1] = True
        elif kind == 2:
            forbidden[t, V // 3:] = True
        elif kind == 3:
            forbidden[t, ::2] = True
        elif kind == 4:
            forbidden[t] = True
            forbidden[t, [V // 2, V - 3]] = False
    x[forbidden] = low
    ids = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(V)).int()
    k = 8
    lp, rank, ent, top, top_ids, _ = O.token_logprobs(x.double().numpy(), ids.numpy(), k, temp)
    glp, grank, gent, gtop, gids = (v.cpu().numpy().astype(np.float64) for v in run(x, ids, k, temp))
    assert np.array_equal(gids, top_ids) and np.array_equal(grank, rank)
    a = np.where(forbidden.numpy(), np.nan, x.double().numpy())
    R = np.nanmax(np.abs(a - np.nanmax(a, 1, keepdims=True)), 1) / temp
    e = 4 * R * 2.0 ** -24 + 2.0 ** -17
    assert np.all(np.abs(gent - ent) <= (1 + R) * e), np.abs(gent - ent).max()
    for got, want, far in ((glp[:, None], lp[:, None], forbidden.gather(1, ids[:, None].long()).numpy()),
                           (gtop, top, forbidden.gather(1, torch.from_numpy(top_ids).long()).numpy())):
        tol = np.where(far, np.abs(want) * 2.0 ** -20, e[:, None] + np.abs(want) * 2.0 ** -22)
        fits = np.abs(want) <= float(torch.finfo(torch.float32).max)
        assert np.all(got[~fits] == -np.inf)
        assert np.all(np.abs(got - want)[fits] <= tol[fits])
