"""GPU checks of adapters with infinite values in B and of numbers beside the largest: the
results are infinite, NaN or finite where their definition is."""

import pytest
import torch

from tests.test_gpu_lora import rows

import weight_only_int2_gb300 as wq

pytestmark = pytest.mark.gpu

INF = float("inf")
# few rows, rows grouped by a launch, tiles of 64; any address and 16 bytes
PATHS = [(M, N, r) for M in (6, 200, 600) for N in (64, 33) for r in (8, 16, 32, 64, 128)]


def kind(t):
    """-1, 0, 1 for -inf, finite, inf; 2 for NaN."""
    return torch.where(t.isnan(), 2, torch.where(t.isinf(), t.sign(), 0)).int()


@pytest.mark.parametrize("M,N,r", PATHS)
def test_infinite_values_of_B(M, N, r):
    """x A^T of +-1, +-1.001 and +-0.999: a bf16 number itself (the second number is 0), above and below one."""
    K, n = 64, 2
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    x[:, 0] = torch.where(torch.arange(M, device="cuda") % 2 == 0, 1.0, -1.0)
    x[:, 1] = (torch.arange(M, device="cuda") % 3 - 1).float() * 2.0 ** -10
    A = torch.zeros((n, r, K), dtype=torch.bfloat16, device="cuda")
    A[:, :, :2] = 1.0
    A[:, 1::2] *= -1.0
    B = rows((n, N, r), 3)
    B[:, 1, 0], B[:, 2, 0] = INF, -INF
    B[:, 3, 0], B[:, 3, r - 1] = INF, INF     # h of both signs: NaN
    B[:, 4, 0], B[:, 4, r - 1] = INF, -INF    # infinite
    B[:, 5] = INF
    B[:, 6, r // 2] = float("nan")
    B[:, N - 1, r - 1] = INF
    base = rows((M, N), 4)
    base[:, 7] = INF
    ids = (torch.arange(M, device="cuda") % 3 - 1).int()
    y = wq.lora_gemm(x, A, B, ids, base)
    want, size = base.double(), base.double().abs()
    for a in range(n):
        at = (ids == a).nonzero().view(-1)
        # (sums of products of whole axes: an infinite value meets no zeros but the definition's own)
        terms = (x[at].double() @ A[a].double().T)[:, None, :] * B[a].double()[None]
        want[at] += terms.sum(2)
        size[at] += terms.abs().sum(2)
    assert torch.equal(kind(y), kind(want))
    ok = want.isfinite()
    # y's rounding; two bf16 numbers for x A^T 2^-16, r / 8 + 4 steps of 2^-23
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -16 + (r / 8 + 4) * 2.0 ** -23) * size
    assert bool(((y.double() - want).abs() <= tol)[ok].all())


@pytest.mark.parametrize("M,N,r", PATHS)
def test_sums_beyond_the_largest_number(M, N, r):
    """x A^T = +-2^64 (1 - 2^-10), whose second number has the other sign, times 2^100: infinite, as the sum is in bf16."""
    K = 64
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    x[:, 0], x[:, 1] = 2.0 ** 64, -2.0 ** 54
    x[1::2] *= -1.0
    A = torch.ones((1, r, K), dtype=torch.bfloat16, device="cuda")
    B, base = rows((1, N, r), 3), rows((M, N), 4)
    B[0, 8, 1], B[0, 20, r - 1], B[0, N - 1, 0] = 2.0 ** 100, -2.0 ** 100, 2.0 ** 64
    ids = torch.zeros(M, dtype=torch.int32, device="cuda")
    y = wq.lora_gemm(x, A, B, ids, base)
    want = base.double() + (x.double() @ A[0].double().T) @ B[0].double().T
    assert torch.equal(kind(y), kind(want.bfloat16())) and int((kind(y) != 0).sum()) == 3 * M


@pytest.mark.parametrize("M,N,r", PATHS)
def test_small_products_with_infinite_values(M, N, r):
    """x A^T down to 2^-126 times an infinite B is infinite, and exactly 0 times it NaN."""
    K = 64
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    power = -(torch.arange(M, device="cuda") % 125 + 2).double()
    x[:, 3] = torch.where(torch.arange(M, device="cuda") % 7 == 0, 0.0, 2.0 ** power)
    x[1::2] *= -1.0
    A = torch.ones((1, r, K), dtype=torch.bfloat16, device="cuda")
    B, base = torch.ones((1, N, r), dtype=torch.bfloat16, device="cuda"), torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    B[0, ::3, r // 2], B[0, 1::3, 1] = INF, -INF
    ids = torch.zeros(M, dtype=torch.int32, device="cuda")
    y = wq.lora_gemm(x, A, B, ids, base)
    sign = x[:, 3].float().sign()
    want = torch.zeros((M, N), device="cuda")
    want[:, ::3], want[:, 1::3] = (sign * INF)[:, None], (-sign * INF)[:, None]  # (0 * inf is NaN)
    want[:, 2::3] = r * x[:, 3, None].float()
    assert torch.equal(kind(y), kind(want))
    assert bool(((y - want)[:, 2::3].abs() <= (2.0 ** -8 + 2.0 ** -15) * want[:, 2::3].abs() + r * 2.0 ** -132).all())


@pytest.mark.parametrize("M,N,r", PATHS)
def test_x_A_beside_the_largest_number(M, N, r):
    """x A^T = 2^128 (1 - 2^-8 + 1.5 2^-9): a float32 number that bf16 rounds to infinity; times B it is ordinary."""
    K, n = 64, 1
    most = torch.finfo(torch.bfloat16).max
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    x[:, 3], x[:, 40] = most, 1.5 * 2.0 ** 119
    x[1::2] *= -1.0
    A = torch.ones((n, r, K), dtype=torch.bfloat16, device="cuda")
    B = rows((n, N, r), 5) * 2.0 ** -110
    base = rows((M, N), 6)
    ids = torch.zeros(M, dtype=torch.int32, device="cuda")
    y = wq.lora_gemm(x, A, B, ids, base)
    h = x.double().sum(1, keepdim=True)
    want = base.double() + h * B[0].double().sum(1)
    size = base.double().abs() + h.abs() * B[0].double().abs().sum(1)
    # y's rounding, two bf16 numbers for h 2^-16, r / 8 + 4 steps of 2^-23
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -16 + (r / 8 + 4) * 2.0 ** -23) * size
    assert bool(((y.double() - want).abs() <= tol).all())
    # an infinite x A^T stays one
    x[:, 5] = x[:, 3]
    y = wq.lora_gemm(x, A, B.abs() + 1, ids, base)
    assert torch.equal(kind(y), x[:, 3].sign().int()[:, None].expand(M, N))
