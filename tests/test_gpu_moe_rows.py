"""GPU checks of the rows of a mixture of experts: sorted by expert, brought back
with weights, and that gradient, against the float64 oracle. Places, offsets and
moved rows are exact; so is dy, one float32 product rounded once.

Tolerances: combine's sum of k products and the residual, each step rounded, is off
by (k + 2) 2^-24 of the terms' sizes and its bf16 rounding 2^-8; a product of
dweights sums at most 8 (D / 2048 + 1) or D / 256 + 1 terms a thread, 5 steps of a
warp and 8 of the block: (D / 128 + 32) 2^-24 of the products' sizes."""

import threading

import numpy as np
import pytest
import torch

from oracle import choice as R
from tests.helpers import Guarded

import weight_only_int2_gb300 as wq

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def choices(T, k, E, seed, out_of=0.0, skew=False):
    r = np.random.default_rng(seed)
    ids = r.integers(0, E, (T, k))
    if skew:
        ids = np.minimum(ids, r.integers(0, E, (T, k)) // 7)
    ids[r.random((T, k)) < out_of] = -1
    far = r.random((T, k)) < out_of / 4
    ids[far] = r.choice([E, E + 1, -2, 2 ** 31 - 1, -2 ** 31], far.sum())
    return ids.astype(np.int32)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def rows(shape, seed):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").bfloat16()


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy()


def f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("T,k,E,out_of", [
    (1, 1, 1, 0), (1, 8, 128, 0), (3, 2, 4, 0.3), (64, 8, 128, 0), (64, 8, 1024, 0.1), (33, 1, 1, 0), (31, 32, 3, 0.5),
    (100, 6, 7, 1.0), (1024, 8, 64, 0), (2048, 1, 1024, 0.2), (2731, 3, 256, 0.05), (1366, 6, 160, 0), (700, 4, 50, 0.1), (4096, 1, 1024, 0.1), (4097, 1, 8, 0),
    (20000, 8, 1024, 0.1),
    (8193, 1, 1, 0.5), (70001, 2, 333, 0)])
@pytest.mark.parametrize("skew", [False, True])
def test_sort_places(T, k, E, out_of, skew):
    ids = choices(T, k, E, T + k + E, out_of, skew)
    go, gs = Guarded((E + 1,), torch.int32), Guarded((T, k), torch.int32)
    bad = torch.full((1,), 5, dtype=torch.int32, device="cuda")
    # (the ids lie anywhere: 4-byte aligned)
    place = torch.empty(T * k + 1, dtype=torch.int32, device="cuda")[1:].view(T, k).copy_(dev(ids))
    none, offsets, slots = wq.moe_sort(None, place, E, offsets=go.t, slots=gs.t, bad_count=bad)
    go.check("offsets")
    gs.check("slots")
    want_offsets, want_slots, want_bad = R.sort(ids, E)
    assert none is None
    assert np.array_equal(offsets.cpu().numpy(), want_offsets) and np.array_equal(slots.cpu().numpy(), want_slots)
    assert int(bad) == 5 + want_bad


@pytest.mark.parametrize("T,k,E,D,out_of", [
    (1, 1, 1, 1, 0), (1, 8, 16, 5120, 0), (5, 3, 4, 7, 0.3), (64, 8, 128, 2048, 0), (64, 9, 128, 136, 0.2), (33, 32, 40, 72, 0.4),
    (7, 2, 3, 8, 1.0), (300, 4, 8, 1001, 0.1), (2000, 6, 64, 264, 0)])
def test_sort_rows(T, k, E, D, out_of):
    ids = choices(T, k, E, D + T, out_of)
    x = rows((T, D + 24), D)[:, 8:8 + D] if D % 8 == 0 else rows((T, D), D)  # strided where 16-byte aligned
    g = Guarded((T * k, D), torch.bfloat16)
    before = bits(g.t.clone())
    out, offsets, slots = wq.moe_sort(x, dev(ids), E, out=g.t)
    g.check("out")
    want_offsets, want_slots, _ = R.sort(ids, E)
    want, xb = before.copy(), bits(x)
    for t, j in np.argwhere(want_slots >= 0):
        want[want_slots[t, j]] = xb[t]
    assert np.array_equal(bits(out), want)  # (rows behind the last expert's are as they were)
    assert np.array_equal(offsets.cpu().numpy(), want_offsets) and np.array_equal(slots.cpu().numpy(), want_slots)


def test_sort_rows_of_an_odd_stride():
    x = rows((40, 19), 1)[:, :16]
    ids = choices(40, 2, 5, 3)
    out, _, slots = wq.moe_sort(x, dev(ids), 5)
    assert torch.equal(out[slots.long()], x[:, None].expand(-1, 2, -1))


@pytest.mark.parametrize("weighted,residual", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("T,k,E,D,out_of", [
    (1, 1, 1, 1, 0), (1, 8, 16, 5120, 0), (5, 3, 4, 7, 0.3), (64, 8, 128, 2048, 0), (33, 32, 40, 72, 0.4), (7, 2, 3, 8, 1.0),
    (300, 9, 8, 1001, 0.1), (500, 6, 64, 264, 0)])
def test_combine(T, k, E, D, out_of, weighted, residual):
    _, slots, _ = R.sort(choices(T, k, E, D + T, out_of), E)
    n = T * k
    y = rows((n, D), 2)
    unused = np.setdiff1d(np.arange(n), slots[slots >= 0])
    y[dev(unused).long()] = float("nan")  # rows of no expert are not read
    w = torch.rand((T, k), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda") - 0.3
    if weighted:
        w[dev(slots) < 0] = float("nan")  # nor do their weights count
    res = rows((T, D), 4) if residual else None
    g = Guarded((T, D), torch.bfloat16)
    out = wq.moe_combine(y, dev(slots), w if weighted else None, residual=res, out=g.t)
    g.check("out")
    want, size = R.combine(f64(y), slots, f64(w) if weighted else None, f64(res) if residual else None)
    assert np.all(np.abs(f64(out) - want) <= (k + 2) * U * size + 2.0 ** -8 * np.abs(want))
    if residual:  # in place
        wq.moe_combine(y, dev(slots), w if weighted else None, residual=res, out=res)
        assert torch.equal(res, out)


@pytest.mark.parametrize("T,k,E,D,out_of", [
    (1, 1, 1, 1, 0), (1, 8, 16, 5120, 0), (5, 3, 4, 7, 0.3), (64, 8, 128, 2048, 0), (33, 32, 40, 72, 0.4), (7, 2, 3, 8, 1.0),
    (300, 9, 8, 1001, 0.1), (500, 6, 64, 264, 0), (20, 10, 16, 4104, 0)])
def test_combine_grad(T, k, E, D, out_of):
    _, slots, _ = R.sort(choices(T, k, E, D + T, out_of), E)
    n = T * k
    y, dout = rows((n, D), 5), rows((T, D), 6)
    unused = np.setdiff1d(np.arange(n), slots[slots >= 0])
    y[dev(unused).long()] = float("nan")
    w = torch.rand((T, k), generator=torch.Generator(device="cuda").manual_seed(7), device="cuda") - 0.3
    gy, gw = Guarded((n, D), torch.bfloat16), Guarded((T, k), torch.float32)
    before = gy.t.clone()
    dy, dw = wq.moe_combine_grad(dout, y, dev(slots), w, dy=gy.t, dweights=gw.t)
    gy.check("dy")
    gw.check("dweights")
    want_dy = before
    for t, j in np.argwhere(slots >= 0):
        want_dy[slots[t, j]] = (w[t, j] * dout[t].float()).bfloat16()
    assert np.array_equal(bits(dy), bits(want_dy))
    _, want, size = R.combine_grad(f64(dout), f64(y), slots, f64(w), np.zeros((n, D)))
    assert np.all(np.abs(f64(dw) - want) <= (D / 128 + 32) * U * size)


def test_combine_slots_out_of_range_and_shared():
    y = rows((6, 40), 1)
    slots = np.array([[0, 6], [-1, 5], [2, 2], [2 ** 31 - 1, -2 ** 31]], np.int32)
    out = wq.moe_combine(y, dev(slots))
    want, size = R.combine(f64(y), slots)
    assert np.all(np.abs(f64(out) - want) <= 4 * U * size + 2.0 ** -8 * np.abs(want))


def test_gradients_against_differences():
    """<dout, combine> along each direction, in float64 differences of the oracle."""
    T, k, E, D = 6, 3, 4, 10
    _, slots, _ = R.sort(choices(T, k, E, 1, 0.2), E)
    y, dout, w = rows((T * k, D), 2), rows((T, D), 3), torch.rand((T, k), device="cuda")
    dy, dw = wq.moe_combine_grad(dout, y, dev(slots), w, dy=torch.zeros_like(y))
    f = lambda yy, ww: (R.combine(yy, slots, ww)[0] * f64(dout)).sum()  # noqa: E731
    y64, w64 = f64(y), f64(w)
    r = np.random.default_rng(4)
    vy, vw = r.standard_normal(y64.shape), r.standard_normal(w64.shape)
    along = (f(y64 + 1e-4 * vy, w64) - f(y64 - 1e-4 * vy, w64)) / 2e-4
    assert abs(along - (f64(dy) * vy).sum()) <= 2.0 ** -8 * np.abs(f64(dy) * vy).sum() + 1e-8
    along = (f(y64, w64 + 1e-4 * vw) - f(y64, w64 - 1e-4 * vw)) / 2e-4
    assert abs(along - (f64(dw) * vw).sum()) <= 1e-5 * np.abs(f64(dw) * vw).sum() + 1e-8
    # the gradient of sort: every choice's gradient back to its token
    ids = choices(T, k, E, 1, 0.2)
    x = rows((T, D), 5)
    out, _, at = wq.moe_sort(x, dev(ids), E, out=torch.zeros((T * k, D), dtype=torch.bfloat16, device="cuda"))
    dx = wq.moe_combine(y, at)
    assert abs((f64(out) * y64).sum() - (f64(x) * f64(dx)).sum()) <= 2.0 ** -8 * np.abs(f64(x) * f64(dx)).sum() + 1e-8


def test_offsets_beyond_32_bits():
    T, k, E, D = 70000, 8, 16, 4096  # 2.3e9 values
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    x = rows((T, D), 2)
    out, offsets, slots = wq.moe_sort(x, ids, E)
    assert int(offsets[-1]) == T * k and int(slots.max()) == T * k - 1
    for t in (0, 1, 34567, T - 1):
        assert torch.equal(out[slots[t].long()], x[t].expand(k, D))
    back = wq.moe_combine(out, slots, torch.full((T, k), 1 / 8, device="cuda"))
    assert torch.equal(back, x)  # eight eighths
    dy, dw = wq.moe_combine_grad(x, out, slots, torch.ones((T, k), device="cuda"))
    assert torch.equal(dy[-1], out[-1]) and torch.equal(dy[: 1 << 12], out[: 1 << 12])
    want = x.double().square().sum(1)
    assert bool(((dw.double() - want[:, None]).abs() <= (D / 128 + 32) * U * want[:, None]).all())


def test_no_tokens():
    ids = torch.empty((0, 4), dtype=torch.int32, device="cuda")
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    out, offsets, slots = wq.moe_sort(x, ids, 9, offsets=torch.full((10,), 7, dtype=torch.int32, device="cuda"))
    assert out.shape == (0, 64) and slots.shape == (0, 4) and not offsets.any()
    assert wq.moe_combine(rows((3, 64), 1), slots).shape == (0, 64)
    assert not wq.moe_sort(None, ids, 9)[1].any()


def test_no_tokens_from_the_sort_to_the_gradients():
    ids = torch.empty((0, 4), dtype=torch.int32, device="cuda")
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.empty((0, 4), device="cuda")
    out, _, slots = wq.moe_sort(x, ids, 9)
    assert wq.moe_combine(out, slots, w, x).shape == (0, 64)
    dy, dw = wq.moe_combine_grad(x, out, slots, w)
    assert dy.shape == (0, 64) and dw.shape == (0, 4)
    assert wq.moe_combine(dy, slots).shape == (0, 64)


def test_same_bits_every_time_and_on_another_stream():
    T, k, E, D = 3000, 6, 64, 512
    ids, x = dev(choices(T, k, E, 1, 0.1)), rows((T, D), 2)
    first = wq.moe_sort(x, ids, E, out=torch.zeros((T * k, D), dtype=torch.bfloat16, device="cuda"))
    w = torch.rand((T, k), device="cuda")
    want = wq.moe_combine(first[0], first[2], w)
    grad = wq.moe_combine_grad(x, first[0], first[2], w, dy=torch.zeros_like(first[0]))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for _ in range(20):
            got = wq.moe_sort(x, ids, E, out=torch.zeros((T * k, D), dtype=torch.bfloat16, device="cuda"))
            again = wq.moe_combine(got[0], got[2], w)
            g2 = wq.moe_combine_grad(x, got[0], got[2], w, dy=torch.zeros_like(got[0]))
            for a, b in zip((*got, again, *g2), (*first, want, *grad)):
                assert torch.equal(a, b)
    s.synchronize()


def test_refusals():
    y, slots = rows((8, 16), 1), torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    w = torch.zeros((4, 2), device="cuda")
    for call, err in [
            (lambda: wq.moe_sort(y, slots, 4), ValueError), (lambda: wq.moe_sort(y[:4], slots.long(), 4), TypeError),
            (lambda: wq.moe_sort(y[:4].float(), slots, 4), TypeError), (lambda: wq.moe_sort(y[:4], slots, 0), (wq.WQError, RuntimeError)),
            (lambda: wq.moe_sort(y[:4], slots[0], 4), ValueError), (lambda: wq.moe_sort(y[:4], slots, 4, out=y[:6]), ValueError),
            (lambda: wq.moe_sort(None, slots, 4, out=y), ValueError), (lambda: wq.moe_sort(y[:4].T.contiguous().T, slots, 4), ValueError),
            (lambda: wq.moe_combine(y.float(), slots), TypeError), (lambda: wq.moe_combine(y, slots, w[:3]), ValueError),
            (lambda: wq.moe_combine(y, slots, w.double()), TypeError), (lambda: wq.moe_combine(y, slots, residual=y), ValueError),
            (lambda: wq.moe_combine(y[:0], slots), wq.WQError), (lambda: wq.moe_combine_grad(y, y, slots, w), ValueError),
            (lambda: wq.moe_combine_grad(y[:4], y, slots, None), TypeError)]:
        with pytest.raises(err):
            call()


# ---------------------------------------------------------------- a whole layer

def layer(E, N, K, seed, bits_=6):
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 1 << bits_, (E * N, K), generator=g, device="cuda", dtype=torch.uint8)
    scales = ((torch.rand((E * N, K // 128), generator=g, device="cuda") + 0.5) * 2 / ((1 << bits_) * K ** 0.5)).bfloat16()
    dense = (codes.double() - (1 << (bits_ - 1))) * scales.double().repeat_interleave(128, 1)
    return (*wq.wna16_repack(codes, scales, bits_), dense.view(E, N, K))


@pytest.mark.parametrize("T", [1, 5, 64, 700])
def test_expert_layer(T):
    """Gate, choice, rows to the experts, their products, rows back onto the residual stream: against the same layer
    in float64. The chain rounds to bf16 twice (the products, the sum), each to 2^-8 of a value, and the product's own
    documented error is 5e-3 of its norm."""
    E, k, D = 8, 2, 256
    packed, scales, dense = layer(E, D, D, 1)
    x = rows((T, D), 2)
    gate = rows((E, D), 3) * 0.1
    logits = x.float() @ gate.float().T
    ids, w = wq.moe_route(logits, k, renormalize=True)
    xs, offsets, slots = wq.moe_sort(x, ids, E)
    y = wq.wna16_moe_gemm(xs, offsets, packed, scales, E, D, D, 6)
    out = wq.moe_combine(y, slots, w, residual=x)
    x64, p = x.double(), torch.softmax(logits.double(), 1)
    best = torch.topk(p, k, 1)
    want = x64.clone()
    for j in range(k):
        term = torch.einsum("tnd,td->tn", dense[best.indices[:, j]], x64)
        want += term * (best.values[:, j] / best.values.sum(1))[:, None]
    assert torch.equal(ids, best.indices.int())
    err = (out.double() - want).norm() / want.norm()
    assert err <= 5e-3 + 2 * 2.0 ** -8, float(err)


@pytest.mark.parametrize("T", [200, 1500])
def test_captured_layer_with_changing_inputs(T):
    """Route, sort, combine and both gradients in one graph, replayed with other inputs; two graphs captured on one
    stream share nothing."""
    E, k, D = 16, 4, 384
    x, logits = rows((T, D), 1), torch.randn((T, E), device="cuda")
    x2, logits2 = rows((T, D), 3), torch.randn((T, E), device="cuda")

    def step(x, logits):
        ids, w = wq.moe_route(logits, k, score="sigmoid", renormalize=True)
        xs, offsets, slots = wq.moe_sort(x, ids, E)
        out = wq.moe_combine(xs, slots, w, residual=x)
        dy, dw = wq.moe_combine_grad(out, xs, slots, w)
        dl = wq.moe_route_grad(logits, ids, dw, score="sigmoid", renormalize=True)
        return [ids, w, xs, offsets, slots, out, dy, dw, dl]

    step(x, logits)
    torch.cuda.synchronize()
    graphs, results = [], []
    for a, b in ((x, logits), (x2, logits2)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            results.append(step(a, b))
        graphs.append(graph)
    for seed in range(4):
        for t in (x, x2):
            t.copy_(rows((T, D), 10 + seed))
        logits.copy_(torch.randn((T, E), device="cuda"))
        logits2.copy_(torch.randn((T, E), device="cuda"))
        for graph in graphs:
            graph.replay()
        for (a, b), got in zip(((x, logits), (x2, logits2)), results):
            want = step(a, b)
            for p, q in zip(got, want):
                assert torch.equal(p, q)


def test_host_threads_on_one_stream():
    jobs = []
    for i, (T, k, E, D) in enumerate([(64, 8, 128, 512), (3000, 4, 64, 256), (1, 2, 8, 1024), (500, 6, 700, 100)]):
        ids, x, w = dev(choices(T, k, E, i, 0.1)), rows((T, D), i), torch.rand((T, k), device="cuda")

        def job(ids=ids, x=x, w=w, E=E):
            xs, offsets, slots = wq.moe_sort(x, ids, E)
            return [offsets, slots, wq.moe_combine(xs, slots, w, residual=x)]

        jobs.append(job)
    want = [job() for job in jobs]
    torch.cuda.synchronize()
    wrong, errors = [0] * len(jobs), []
    start = threading.Barrier(len(jobs))

    def work(i):
        try:
            start.wait()
            got = [jobs[i]() for _ in range(40)]
            wrong[i] = sum(not torch.equal(a, b) for r in got for a, b in zip(r, want[i]))
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors and wrong == [0] * len(jobs), (errors, wrong)
