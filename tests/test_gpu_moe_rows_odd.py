"""GPU checks of rows whose length or stride is no multiple of 8, on each way that they
take: sorted by one launch or by two, cut into parts, and the gradient's wide blocks.
The checks and tolerances are those of tests/test_gpu_moe_rows.py."""

import numpy as np
import pytest
import torch

from oracle import choice as R
from tests.helpers import Guarded
from tests.test_gpu_moe_rows import U, bits, choices, dev, f64, rows

import weight_only_int2_gb300 as wq

pytestmark = pytest.mark.gpu

# (above 2048 choices two launches; T below 2 blocks an SM and D above 2048: the gradient's blocks of 512)
SIZES = [(700, 4, 100, 0.1), (700, 4, 2049, 0.1), (5, 3, 4097, 0.3), (40, 8, 5121, 0.1), (3000, 1, 1033, 0.0), (300, 9, 1503, 0.2),
         (2, 1, 12345, 0.0), (4099, 2, 71, 0.5), (1, 1, 2055, 0.0)]


@pytest.mark.parametrize("wide", [0, 3])
@pytest.mark.parametrize("T,k,D,out_of", SIZES)
def test_sort(T, k, D, out_of, wide):
    ids = choices(T, k, 13, D + T, out_of)
    x = rows((T, D + wide), D)[:, :D]
    g = Guarded((T * k, D), torch.bfloat16)
    want = bits(g.t.clone())
    out, offsets, slots = wq.moe_sort(x, dev(ids), 13, out=g.t)
    g.check("out")
    want_offsets, want_slots, _ = R.sort(ids, 13)
    xb = bits(x)
    for t, j in np.argwhere(want_slots >= 0):
        want[want_slots[t, j]] = xb[t]
    assert np.array_equal(offsets.cpu().numpy(), want_offsets) and np.array_equal(slots.cpu().numpy(), want_slots)
    assert np.array_equal(bits(out), want)


@pytest.mark.parametrize("D,stride", [(64, 67), (2048, 2051), (5120, 5121)])
def test_sort_of_many_choices_with_an_odd_stride(D, stride):
    ids = choices(700, 4, 9, D, 0.1)
    x = rows((700, stride), D)[:, :D]
    out, _, slots = wq.moe_sort(x, dev(ids), 9)
    at = slots.view(-1) >= 0
    assert torch.equal(out[slots.view(-1)[at].long()], x.repeat_interleave(4, 0)[at])


@pytest.mark.parametrize("weighted,residual", [(True, True), (False, False)])
@pytest.mark.parametrize("T,k,D,out_of", SIZES)
def test_combine(T, k, D, out_of, weighted, residual):
    _, slots, _ = R.sort(choices(T, k, 13, D + T, out_of), 13)
    y = rows((T * k, D), 2)
    unused = np.setdiff1d(np.arange(T * k), slots[slots >= 0])
    y[dev(unused).long()] = float("nan")
    w = torch.rand((T, k), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda") - 0.3 if weighted else None
    res = rows((T, D), 4) if residual else None
    g = Guarded((T, D), torch.bfloat16)
    out = wq.moe_combine(y, dev(slots), w, residual=res, out=g.t)
    g.check("out")
    want, size = R.combine(f64(y), slots, None if w is None else f64(w), None if res is None else f64(res))
    assert np.all(np.abs(f64(out) - want) <= 2.0 ** -8 * np.abs(want) + (k + 2) * U * size)
    if residual:
        again = wq.moe_combine(y, dev(slots), w, residual=res, out=res)
        assert again is res and torch.equal(res, out)


@pytest.mark.parametrize("T,k,D,out_of", SIZES)
def test_combine_gradient(T, k, D, out_of):
    _, slots, _ = R.sort(choices(T, k, 13, D + T, out_of), 13)
    y, dout = rows((T * k, D), 2), rows((T, D), 3)
    w = torch.rand((T, k), generator=torch.Generator(device="cuda").manual_seed(4), device="cuda") - 0.3
    gy, gw = Guarded((T * k, D), torch.bfloat16), Guarded((T, k), torch.float32)
    before = gy.t.clone()
    dy, dw = wq.moe_combine_grad(dout, y, dev(slots), w, dy=gy.t, dweights=gw.t)
    gy.check("dy")
    gw.check("dweights")
    want_dy, want, size = R.combine_grad(f64(dout), f64(y), slots, f64(w), np.zeros((T * k, D)))
    named = np.zeros(T * k, bool)
    named[slots[slots >= 0]] = True
    # one float32 product, rounded to bf16
    err = np.abs(f64(dy) - want_dy)[named]
    assert np.all(err <= (2.0 ** -8 + 2 * U) * np.abs(want_dy)[named])
    rest = dev(~named)
    assert torch.equal(dy[rest].view(torch.int16), before[rest].view(torch.int16))
    assert np.all(np.abs(f64(dw) - want) <= (D / 128 + 32) * U * size)
