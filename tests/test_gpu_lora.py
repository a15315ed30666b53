"""GPU checks of the low-rank adapters against the float64 oracle.

Tolerance, per value: y's rounding 2^-8; the first product's K terms go 16 at a time
into a float32 sum (each step at worst cut off, 2^-23), then at most 32 shares and 4
warps are added: (K / 16 + 40) 2^-23 of the terms' sizes, carried through B; its two
bf16 numbers leave 2^-17, its scale 2^-24; base begins the second product's sum, whose
r / 8 steps are cut off likewise: (r / 8 + 4) 2^-23 of base's and the terms' sizes."""

import threading

import numpy as np
import pytest
import torch

from oracle import choice as R
from tests.helpers import Guarded

import weight_only_int2_gb300 as wq

pytestmark = pytest.mark.gpu


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def rows(shape, seed, size=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * size).bfloat16()


def f64(t):
    return t.double().cpu().numpy()


def ids_of(M, n, seed, none=0.15, each=1):
    r = np.random.default_rng(seed)
    ids = np.repeat(r.integers(0, n, -(-M // each)), each)[:M]
    ids[r.random(M) < none] = -1
    return ids.astype(np.int32)


def tolerance(want, first, second, base, K, r):
    return (2.0 ** -8 * np.abs(want) + (K / 16 + 40) * 2.0 ** -23 * first + 2.0 ** -17 * second
            + (r / 8 + 4) * 2.0 ** -23 * (np.abs(base) + second))


def check(M, K, N, r, n, ids, scaled=True, base_wide=0, y_wide=0, x_wide=0, seed=0):
    x = rows((M, K + x_wide), seed)[:, :K]
    A, B = rows((n, r, K), seed + 1, K ** -0.5), rows((n, N, r), seed + 2, r ** -0.5)
    scale = torch.rand(n, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda") + 0.5 if scaled else None
    base = rows((M, N + base_wide), seed + 3)[:, base_wide:]
    g = Guarded((M, N + y_wide), torch.bfloat16)
    before = g.t.clone()
    y = wq.lora_gemm(x, A, B, dev(ids), base, scale=scale, y=g.t[:, y_wide // 2:y_wide // 2 + N])
    g.check("y")
    if y_wide:
        edge = torch.ones(N + y_wide, dtype=torch.bool, device="cuda")
        edge[y_wide // 2:y_wide // 2 + N] = False
        assert torch.equal(g.t[:, edge].view(torch.int16), before[:, edge].view(torch.int16))
    want, first, second = R.lora(f64(x), f64(A), f64(B), ids, f64(base), f64(scale) if scaled else None)
    err = np.abs(f64(y) - want) - tolerance(want, first, second, f64(base), K, r)
    assert np.all(err <= 0), (err.max(), np.argwhere(err > 0)[:4])
    assert np.linalg.norm(f64(y) - want) <= 1.01 * 2.0 ** -8 * np.linalg.norm(want)
    none = (ids < 0) | (ids >= n)
    assert torch.equal(y[dev(none)].contiguous().view(torch.int16), base[dev(none)].contiguous().view(torch.int16))
    # in place, rows without an adapter untouched
    again = wq.lora_gemm(x, A, B, dev(ids), base, scale=scale, y=base)
    assert again is base and torch.equal(base.contiguous().view(torch.int16), y.contiguous().view(torch.int16))
    return y


@pytest.mark.parametrize("r", [8, 16, 24, 32, 40, 64, 72, 128])
@pytest.mark.parametrize("M,K,N,n", [(1, 128, 64, 1), (5, 1024, 200, 3), (40, 136, 1000, 40), (600, 256, 136, 5)])
def test_ranks(M, K, N, n, r):
    check(M, K, N, r, n, ids_of(M, n, M + r), seed=r)


@pytest.mark.parametrize("M,K,N,r,n", [
    (1, 8, 1, 8, 1), (2, 5120, 33, 16, 4), (15, 264, 31, 16, 2), (16, 512, 32, 16, 1), (17, 520, 129, 32, 1), (64, 1024, 257, 16, 64),
    (511, 72, 96, 16, 1), (512, 72, 96, 16, 1), (513, 64, 40, 64, 9), (1000, 1032, 127, 16, 1000), (700, 128, 8, 128, 1024)])
def test_shapes(M, K, N, r, n):
    check(M, K, N, r, n, ids_of(M, n, M + N), scaled=M % 2 == 0, seed=M)


@pytest.mark.parametrize("M", [40, 640])
@pytest.mark.parametrize("base_wide,y_wide,x_wide", [(64, 16, 8), (3, 0, 16), (0, 7, 0), (8, 8, 1024)])
def test_strides_and_alignment(M, base_wide, y_wide, x_wide):
    check(M, 256, 104, 16, 6, ids_of(M, 6, M, each=7), base_wide=base_wide, y_wide=y_wide, x_wide=x_wide, seed=M + y_wide)


@pytest.mark.parametrize("M", [9, 530])
def test_adapters_out_of_range_and_none(M):
    ids = ids_of(M, 3, M)
    ids[::4] = np.resize(np.array([3, 1024, 2 ** 31 - 1, -2 ** 31, -2], np.int32), ids[::4].size)
    check(M, 128, 72, 16, 3, ids, seed=M)
    check(M, 128, 72, 16, 3, np.full(M, -1, np.int32), seed=M)
    check(M, 128, 72, 16, 3, np.full(M, 2, np.int32), seed=M)
    one = np.full(M, -1, np.int32)
    one[M // 2] = 1
    check(M, 2048, 72, 32, 3, one, seed=M)


def test_prompts_and_tokens_mixed():
    ids = np.concatenate([np.full(300, 4), np.full(1, 2), np.full(511, -1), np.full(200, 2), ids_of(100, 6, 1)]).astype(np.int32)
    check(len(ids), 640, 328, 16, 6, ids, seed=5)


@pytest.mark.parametrize("M", [4, 600])
def test_infinite_and_nan_values(M):
    """An infinite product stays infinite; NaN and infinities stay in their rows."""
    K, N, r, n = 128, 64, 16, 2
    x, A, B = rows((M, K), 1), rows((n, r, K), 2).abs() + 0.1, rows((n, N, r), 3).abs() + 0.1
    x[0], x[1, 5], x[2] = float("inf"), float("nan"), 1e38
    base, ids = rows((M, N), 4), torch.zeros(M, dtype=torch.int32, device="cuda")
    ids[3] = -1
    x[3] = float("nan")
    y = wq.lora_gemm(x, A, B, ids, base)
    assert bool((y[0] == float("inf")).all() and y[1].isnan().all() and (y[2] == float("inf")).all())
    assert torch.equal(y[3], base[3]) and bool(y[4:].isfinite().all())


@pytest.mark.parametrize("M,N", [(5, 64), (5, 33), (700, 64), (700, 33)])
def test_rows_without_an_adapter_are_copied_bit_by_bit(M, N):
    """Every bf16 pattern (NaN payloads, infinities, -0.0) of base, beside rows with an adapter."""
    K, r, n = 64, 8, 2
    g = torch.Generator(device="cuda").manual_seed(M + N)
    base = torch.randint(-2 ** 15, 2 ** 15, (M, N), generator=g, device="cuda", dtype=torch.int16).view(torch.bfloat16)
    ids = torch.where(torch.arange(M, device="cuda") % 3 == 1, 1, -1).int()
    y = wq.lora_gemm(rows((M, K), 1), rows((n, r, K), 2), rows((n, N, r), 3), ids, base)
    assert torch.equal(y[ids < 0].view(torch.int16), base[ids < 0].view(torch.int16))


def test_offsets_beyond_32_bits():
    """Rows of y behind 2^31 values, and adapters behind 2^31 values of B."""
    M, K, N, r, n = 70000, 64, 32768, 16, 2  # 2.3e9 values of y
    x, A, B = rows((M, K), 1), rows((n, r, K), 2, K ** -0.5), rows((n, N, r), 3)
    ids = (torch.arange(M, device="cuda") % 3 - 1).int()
    base = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    wq.lora_gemm(x, A, B, ids, base, y=base)
    for m in (0, 1, 2, 65535, 65536, M - 2, M - 1):
        a = int(ids[m])
        want = torch.zeros(N, dtype=torch.float64, device="cuda")
        size = want
        if a >= 0:
            h = A[a].double() @ x[m].double()
            want, size = B[a].double() @ h, B[a].double().abs() @ h.abs()
        assert bool(((base[m].double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-4 * size).all()), m
    del base, x, A
    n, N, r, K, M = 1024, 17408, 128, 64, 3  # 2.28e9 values
    B = torch.zeros((n, N, r), dtype=torch.bfloat16, device="cuda")
    B[n - 1] = rows((N, r), 4)
    A, x, base = rows((n, r, K), 5, K ** -0.5), rows((M, K), 6), rows((M, N), 7)
    y = wq.lora_gemm(x, A, B, torch.tensor([n - 1, 0, n - 1], dtype=torch.int32, device="cuda"), base)
    h = x.double() @ A[n - 1].double().T
    want, size = base.double() + h @ B[n - 1].double().T, base.double().abs() + h.abs() @ B[n - 1].double().abs().T
    ok = (y.double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-4 * size
    assert bool(ok[0].all() and ok[2].all()) and torch.equal(y[1], base[1])


def test_no_rows_and_refusals():
    w = rows((2, 16, 16), 1)
    empty = torch.empty((0, 16), dtype=torch.bfloat16, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    assert wq.lora_gemm(empty, w, w, none, empty).shape == (0, 16)
    x, ids = rows((3, 16), 2), torch.zeros(3, dtype=torch.int32, device="cuda")
    for call, err in [
            (lambda: wq.lora_gemm(x, w, w[:1], ids, x), ValueError), (lambda: wq.lora_gemm(x, w, w[0], ids, x), ValueError),
            (lambda: wq.lora_gemm(x.float(), w, w, ids, x), TypeError), (lambda: wq.lora_gemm(x, w, w, ids.long(), x), TypeError),
            (lambda: wq.lora_gemm(x, w, w, ids[:2], x), ValueError), (lambda: wq.lora_gemm(x, w, w, ids, x[:, :8]), ValueError),
            (lambda: wq.lora_gemm(x[:, :8], w, w, ids, x), ValueError), (lambda: wq.lora_gemm(x.T.contiguous().T, w, w, ids, x), ValueError),
            (lambda: wq.lora_gemm(x, w, w, ids, x, scale=torch.ones(3, device="cuda")), ValueError),
            (lambda: wq.lora_gemm(x, rows((2, 12, 16), 3), rows((2, 16, 12), 4), ids, x), wq.WQError),
            (lambda: wq.lora_gemm(rows((3, 20), 1)[:, :16], w, w, ids, x), wq.WQError),
            (lambda: wq.lora_gemm(x, w, w, ids, x, ws=torch.empty(16, dtype=torch.uint8, device="cuda")), wq.WQError)]:
        with pytest.raises(err):
            call()


def test_beside_a_quantized_layer():
    """A decode step's projection with adapters: wna16_gemm, then the adapters in place on a slice of its columns."""
    N, K, bits, M, n, r = 768, 1024, 6, 12, 4, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    codes = torch.randint(0, 64, (N, K), generator=g, device="cuda", dtype=torch.uint8)
    scales = ((torch.rand((N, K // 128), generator=g, device="cuda") + 0.5) / (32 * K ** 0.5)).bfloat16()
    packed, s_dev = wq.wna16_repack(codes, scales, bits)
    x, ids = rows((M, K), 2), ids_of(M, n, 3)
    A, B = rows((n, r, K), 4, K ** -0.5), rows((n, 256, r), 5, r ** -0.5)
    y = wq.wna16_gemm(x, packed, s_dev, N, K, bits)
    plain = y.clone()
    wq.lora_gemm(x, A, B, dev(ids), y[:, 512:], y=y[:, 512:])
    want, first, second = R.lora(f64(x), f64(A), f64(B), ids, f64(plain[:, 512:]))
    assert torch.equal(y[:, :512], plain[:, :512])
    assert np.all(np.abs(f64(y[:, 512:]) - want) <= tolerance(want, first, second, f64(plain[:, 512:]), K, r))


def test_same_bits_captured_on_another_stream_and_from_threads():
    jobs = []
    for i, (M, K, N, r, n) in enumerate([(1, 2048, 640, 16, 8), (64, 1024, 512, 32, 40), (900, 256, 384, 64, 3)]):
        x, A, B = rows((M, K), i), rows((n, r, K), i + 1, K ** -0.5), rows((n, N, r), i + 2, r ** -0.5)
        ids, base = dev(ids_of(M, n, i)), rows((M, N), i + 3)
        jobs.append(lambda x=x, A=A, B=B, ids=ids, base=base: wq.lora_gemm(x, A, B, ids, base))
    want = [job() for job in jobs]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for _ in range(10):
            for job, w in zip(jobs, want):
                assert torch.equal(job(), w)
    s.synchronize()
    graphs = []
    for job in jobs:  # two graphs of a job, replayed in turn with the others
        for _ in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                out = job()
            graphs.append((graph, out))
    for _ in range(3):
        for graph, out in graphs:
            out.zero_()
            graph.replay()
        for i, (graph, out) in enumerate(graphs):
            assert torch.equal(out, want[i // 2])
    wrong, errors = [0] * len(jobs), []
    start = threading.Barrier(len(jobs))

    def work(i):
        try:
            start.wait()
            wrong[i] = sum(not torch.equal(jobs[i](), want[i]) for _ in range(40))
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors and wrong == [0] * len(jobs), (errors, wrong)


@pytest.mark.parametrize("M,r", [(48, 16), (48, 32), (200, 16), (700, 16), (700, 64), (1500, 16)])
def test_inputs_changed_between_calls(M, r):
    """Every input is written anew before each call and each replay: what a call reads before the kernel in front of it
    ends is what was there when the call began."""
    K, N, n = 512, 264, 12
    made = lambda seed: [rows((M, K), seed), rows((n, r, K), seed + 1, K ** -0.5), rows((n, N, r), seed + 2, r ** -0.5),  # noqa: E731
                         dev(ids_of(M, n, seed + 3, none=0.2)), rows((M, N), seed + 4),
                         torch.rand(n, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")]
    use = made(0)
    call = lambda t, **kw: wq.lora_gemm(t[0], t[1], t[2], t[3], t[4], scale=t[5], **kw)  # noqa: E731
    call(use)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = call(use)
    sets = [made(10 * (i + 1)) for i in range(4)]
    want = [call(t) for t in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        for new, w in zip(sets, want):
            for a, b in zip(use, new):
                a.copy_(b)
            got = call(use)
            graph.replay()
            again = y.clone()
            in_place = call(use, y=use[4])
            assert torch.equal(got, w) and torch.equal(again, w) and torch.equal(in_place, w)


@pytest.mark.parametrize("r", [40, 64, 96, 128])
@pytest.mark.parametrize("M,K,N,n,base_wide,y_wide", [
    (512, 64, 8, 1, 0, 0), (513, 128, 1000, 3, 0, 16), (700, 256, 333, 5, 3, 0), (900, 136, 72, 700, 8, 7), (2100, 72, 1416, 4, 64, 0)])
def test_larger_ranks_of_many_rows(M, K, N, n, base_wide, y_wide, r):
    check(M, K, N, r, n, ids_of(M, n, M + r, each=1 + M // 100), base_wide=base_wide, y_wide=y_wide, seed=M + r)


@pytest.mark.parametrize("N", [200, 201])
@pytest.mark.parametrize("r", [64, 128])
def test_larger_ranks_of_out_of_range_infinite_and_other_inputs(N, r):
    M, K, n = 700, 128, 3
    ids = ids_of(M, n, M)
    ids[::4] = np.resize(np.array([3, 1024, 2 ** 31 - 1, -2 ** 31, -2], np.int32), ids[::4].size)
    check(M, K, N, r, n, ids, seed=N)
    check(M, K, N, r, n, np.full(M, -1, np.int32), seed=N)
    x, A, B = rows((M, K), 1), rows((n, r, K), 2).abs() + 0.1, rows((n, N, r), 3).abs() + 0.1
    x[0], x[1, 5], x[2], x[3] = float("inf"), float("nan"), 1e38, float("nan")
    base, ids = rows((M, N), 4), torch.zeros(M, dtype=torch.int32, device="cuda")
    ids[3] = -1
    y = wq.lora_gemm(x, A, B, ids, base)
    assert bool((y[0] == float("inf")).all() and y[1].isnan().all() and (y[2] == float("inf")).all())
    assert torch.equal(y[3], base[3]) and bool(y[4:].isfinite().all())
    # the same bits again, on two streams at once
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        got = []
        for s in (one, two):
            with torch.cuda.stream(s):
                got.append(wq.lora_gemm(x, A, B, ids, base))
        torch.cuda.synchronize()
        assert all(torch.equal(v.view(torch.int16), y.view(torch.int16)) for v in got)


@pytest.mark.parametrize("r", [64, 128])
def test_larger_ranks_beside_a_quantized_layer_of_many_rows(r):
    """A prompt's projection and its adapters, one after another in a stream, on two streams at once: both kinds of
    kernel hold tensor memory."""
    N, K, bits, M, n = 768, 1024, 6, 900, 4
    g = torch.Generator(device="cuda").manual_seed(1)
    codes = torch.randint(0, 64, (N, K), generator=g, device="cuda", dtype=torch.uint8)
    scales = ((torch.rand((N, K // 128), generator=g, device="cuda") + 0.5) / (32 * K ** 0.5)).bfloat16()
    packed, s_dev = wq.wna16_repack(codes, scales, bits)
    x, ids = rows((M, K), 2), ids_of(M, n, 3, each=50)
    A, B, at = rows((n, r, K), 4, K ** -0.5), rows((n, 256, r), 5, r ** -0.5), dev(ids)
    plain = wq.wna16_gemm(x, packed, s_dev, N, K, bits)

    def layer():
        y = wq.wna16_gemm(x, packed, s_dev, N, K, bits)
        wq.lora_gemm(x, A, B, at, y[:, 512:], y=y[:, 512:])
        return y

    first_y = layer()
    want, first, second = R.lora(f64(x), f64(A), f64(B), ids, f64(plain[:, 512:]))
    assert torch.equal(first_y[:, :512], plain[:, :512])
    assert np.all(np.abs(f64(first_y[:, 512:]) - want) <= tolerance(want, first, second, f64(plain[:, 512:]), K, r))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(layer())
    torch.cuda.synchronize()
    assert all(torch.equal(y, first_y) for y in got)
