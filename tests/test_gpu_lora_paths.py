"""GPU checks of the adapters' paths one by one, against their definition in float64 on
the GPU: the rings of the tensor cores in steady state (more stages a share and units a
block than a ring holds), 129 to 511 rows, and adapters rewritten between calls.

The tolerance is derived as in tests/test_gpu_lora.py; the two bf16 numbers of x A^T, the first
below it and the second the rest rounded, leave 2^-16 of it."""

import numpy as np
import pytest
import torch

from tests.helpers import Guarded
from tests.test_gpu_lora import check, dev, ids_of, rows

import weight_only_int2_gb300 as wq

pytestmark = pytest.mark.gpu


def definition(x, A, B, ids, base, scale):
    """(y, the sums of sizes of the first product's terms carried through the second, of the second's), float64."""
    y = base.double()
    first, second = torch.zeros_like(y), torch.zeros_like(y)
    for a in torch.unique(ids[(ids >= 0) & (ids < A.shape[0])]).tolist():
        at = (ids == a).nonzero().view(-1)
        xa, Aa, Ba, s = x[at].double(), A[a].double(), B[a].double(), scale[a].double()
        h = xa @ Aa.T
        y[at] += s * (h @ Ba.T)
        first[at] = s.abs() * (xa.abs() @ Aa.abs().T @ Ba.abs().T)
        second[at] = s.abs() * (h.abs() @ Ba.abs().T)
    return y, first, second


def near(y, x, A, B, ids, base, scale):
    want, first, second = definition(x, A, B, ids, base, scale)
    K, r = x.shape[1], A.shape[1]
    tol = (2.0 ** -8 * want.abs() + (K / 16 + 40) * 2.0 ** -23 * first + 2.0 ** -16 * second
           + (r / 8 + 4) * 2.0 ** -23 * (base.double().abs() + second))
    over = (y.double() - want).abs() - tol
    assert bool((over <= 0).all()), (float(over.max()), (over > 0).nonzero()[:4].tolist())


def made(M, K, N, r, n, seed, each, base_wide=0, none=0.1):
    x, A, B = rows((M, K), seed), rows((n, r, K), seed + 1, K ** -0.5), rows((n, N, r), seed + 2, r ** -0.5)
    scale = torch.rand(n, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda") + 0.5
    return x, A, B, dev(ids_of(M, n, seed, none=none, each=each)), rows((M, N + base_wide), seed + 3)[:, base_wide:], scale


@pytest.mark.parametrize("r", [16, 32, 64, 128])
@pytest.mark.parametrize("M,K,N,n,each,base_wide", [
    (512, 1024, 72, 400, 1, 0),       # a share is all of K: 16 stages a tile, many tiles a block
    (520, 11272, 40, 2, 100, 0),      # more than six stages a share, the last one of 8 values
    (2049, 17408, 136, 9, 111, 0),    # about 30 stages a share
    (2100, 72, 8192, 4, 60, 0),       # 15 units a block
    (2100, 72, 8193, 4, 60, 0),       # the same at any address
    (2100, 72, 8192, 4, 60, 5)])
def test_rings_of_many_rows(M, K, N, n, each, base_wide, r):
    x, A, B, ids, base, scale = made(M, K, N, r, n, M + r, each, base_wide)
    g = Guarded((M, N), torch.bfloat16)
    y = wq.lora_gemm(x, A, B, ids, base, scale=scale, y=g.t)
    g.check("y")
    near(y, x, A, B, ids, base, scale)
    wq.check_status()
    again = wq.lora_gemm(x, A, B, ids, base, scale=scale)
    in_place = wq.lora_gemm(x, A, B, ids, base, scale=scale, y=base)
    assert torch.equal(again, y) and torch.equal(in_place, y)


@pytest.mark.parametrize("N,base_wide,y_wide", [(96, 0, 0), (129, 0, 0), (96, 3, 0), (104, 0, 7)])
@pytest.mark.parametrize("r", [8, 16, 24, 32, 64, 72, 128])
@pytest.mark.parametrize("M,n", [(129, 3), (300, 40), (511, 2)])
def test_129_to_511_rows(M, n, r, N, base_wide, y_wide):
    check(M, 264, N, r, n, ids_of(M, n, M + r, each=1 + n % 5), base_wide=base_wide, y_wide=y_wide, seed=M + r)


@pytest.mark.parametrize("r", [16, 128])
@pytest.mark.parametrize("M", [5, 300])
def test_rings_of_few_rows(M, r):
    x, A, B, ids, base, scale = made(M, 17408, 8200, r, 3, M + r, 2)
    y = wq.lora_gemm(x, A, B, ids, base, scale=scale)
    near(y, x, A, B, ids, base, scale)
    odd = rows((M, 8201), M)[:, 1:]
    near(wq.lora_gemm(x, A, B, ids, odd, scale=scale), x, A, B, ids, odd, scale)


@pytest.mark.parametrize("M,r", [(200, 8), (200, 64), (200, 128), (130, 24)])
def test_inputs_changed_between_calls_of_129_to_511_rows(M, r):
    use = list(made(M, 512, 264, r, 12, 0, 1, none=0.2))
    sets = [made(M, 512, 264, r, 12, 10 * (i + 1), 1, none=0.2) for i in range(4)]
    call = lambda t, **kw: wq.lora_gemm(*t[:5], scale=t[5], **kw)  # noqa: E731
    call(use)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = call(use)
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


@pytest.mark.parametrize("early", [False, True])
@pytest.mark.parametrize("M,N,r,n", [(1, 17408, 16, 1), (1, 17408, 8, 1), (64, 17408, 16, 5), (64, 17408, 8, 41), (200, 4096, 16, 3),
                                     (1, 1024, 32, 1), (64, 17408, 64, 2)])
def test_only_B_changed_between_calls(M, N, r, n, early):
    """The place of an adapter's B gets another one between two calls, by torch's copy or by a kernel of the library's
    own, which lets the call's kernels start before it ends."""
    K = 256
    x, A, _, ids, base, scale = made(M, K, N, r, n, 1, 1, none=0.0)
    sets = [rows((n, N, r), 50 + i, r ** -0.5) for i in range(3)]
    want = [wq.lora_gemm(x, A, b, ids, base, scale=scale) for b in sets]
    B = torch.zeros_like(sets[0])
    flat = B.view(-1, 1024)
    slots = torch.arange(flat.shape[0], dtype=torch.int32, device="cuda").view(-1, 1)
    for i in range(60):
        b = sets[i % 3]
        if early:
            wq.moe_combine(b.view(-1, 1024), slots, out=flat)
        else:
            B.copy_(b)
        got = [wq.lora_gemm(x, A, B, ids, base, scale=scale) for _ in range(2)]
        assert all(torch.equal(y, want[i % 3]) for y in got), i


def test_definition_is_the_oracle():
    from oracle import choice as R
    x, A, B, ids, base, scale = made(30, 64, 24, 16, 3, 9, 2)
    got = definition(x, A, B, ids, base, scale)
    n = lambda t: t.double().cpu().numpy()  # noqa: E731
    for a, b in zip(got, R.lora(n(x), n(A), n(B), ids.cpu().numpy(), n(base), n(scale))):
        assert np.allclose(a.cpu().numpy(), b, rtol=1e-12, atol=1e-14)
