"""GPU check of adapters beside the widest projections (N next to 2^31): the last columns,
which end inside a unit of 64, against float64. B is followed by NaN."""

import pytest
import torch

from tests.test_gpu_lora import rows

import weight_only_int2_gb300 as wq

pytestmark = pytest.mark.gpu


def test_columns_next_to_two_to_the_31st():
    torch.cuda.empty_cache()
    K, r, most = 8, 16, 2 ** 31 - 1
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("B alone takes 69 GB")
    flat = torch.zeros((most + 65, r), dtype=torch.bfloat16, device="cuda")
    x, A, last = rows((1, K), 1), rows((1, r, K), 2, K ** -0.5), rows((200, r), 3)
    ids = torch.zeros(1, dtype=torch.int32, device="cuda")
    h = A[0].double() @ x[0].double()
    for N in (most, most // 8 * 8, most - 62, most - 63):  # at any address, by 16 bytes; one value in the last unit, none
        flat[-1000:] = 0
        flat[N - 200:N] = last
        flat[N:] = float("nan")
        base = torch.zeros((1, N), dtype=torch.bfloat16, device="cuda")
        base[0, -200:] = rows((200,), 4)
        y = wq.lora_gemm(x, A, flat[:N].unsqueeze(0), ids, base)
        want = base[0, -200:].double() + last.double() @ h
        size = base[0, -200:].double().abs() + last.double().abs() @ (A[0].double().abs() @ x[0].double().abs())
        # y's rounding; two bf16 numbers for h 2^-16; K / 16 + 40 and r / 8 + 4 steps of 2^-23
        assert bool(((y[0, -200:].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -15 * size).all()), N
        assert not bool(y[0, 5 * 10 ** 8:-200].any()) and not bool(y[0, :5 * 10 ** 8].any())
        del base, y
