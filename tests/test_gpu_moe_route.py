"""GPU checks of the router and its gradient against the float64 oracle.

Tolerances. A weight is exp(x - m) over a sum, or 1 / (1 + exp(-x)), maybe over a
sum: with u = 2^-24 a rounding's share, the argument's rounding gives D u (D the
spread of the finite logits that count, at most 104, where exp ends), expf at most
2 ulp = 4 u, a lane's sum of at most 32 terms and the warp's of 32 lanes 37 u, the
quotient and the scale 2 u each, twice where the quotient's parts both have them:
(2 D + 64) u of the weight, and 2^-126 where the numbers have no full precision. A
gradient is p (g - sum g p) (times 1 - s): its terms' sizes p (|g| + sum |g| p)
carry that and the sum's 6 u more, and bf16 gradients the rounding 2^-8."""

import math

import numpy as np
import pytest
import torch

from oracle import choice as R
from tests.helpers import Guarded

import weight_only_int2_gb300 as wq

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def rel_of(x):
    spread = np.zeros(len(x))
    for t, row in enumerate(x):
        f = row[np.isfinite(row)]
        spread[t] = min(104.0, f.max() - f.min()) if f.size else 0.0
    return ((2 * spread + 64) * U)[:, None]


def logits(T, E, seed, masked=0.0, step=0.0):
    r = np.random.default_rng(seed)
    x = r.standard_normal((T, E)) * 2
    if step:
        x = np.round(x / step) * step  # many ties
    x[r.random((T, E)) < masked] = -np.inf
    return x.astype(np.float32)


def on_gpu(x, bf16):
    t = torch.from_numpy(x).cuda()
    return t.bfloat16() if bf16 else t


def close(got, want, tol):
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    assert np.all(np.abs(got - want)[ok] <= np.broadcast_to(tol, want.shape)[ok]), np.nanmax(np.abs(got - want) - tol)


def check(x, k, score, renorm, scale, bf16, seed, strided=False):
    t = on_gpu(x, bf16)
    if strided:
        wide = torch.full((x.shape[0], x.shape[1] + 3), math.nan, dtype=t.dtype, device="cuda")
        wide[:, :x.shape[1]] = t
        t = wide[:, :x.shape[1]]
    x = t.double().cpu().numpy()
    T, E = x.shape
    gi, gw = Guarded((T, k), torch.int32), Guarded((T, k), torch.float32)
    ids, w = wq.moe_route(t, k, score=score, renormalize=renorm, scale=scale, ids=gi.t, weights=gw.t)
    gi.check("ids")
    gw.check("weights")
    want_ids, want = R.route(x, k, score, renorm, scale)
    ids = ids.cpu().numpy()
    assert np.array_equal(ids, want_ids)
    rel = rel_of(x)
    close(w.double().cpu().numpy(), want, rel * np.abs(want) + 2.0 ** -126)

    dw = np.random.default_rng(seed).standard_normal((T, k)).astype(np.float32)
    gd = Guarded((T, E), t.dtype)
    d = wq.moe_route_grad(t, torch.from_numpy(ids).cuda(), torch.from_numpy(dw).cuda(), score=score, renormalize=renorm,
                          scale=scale, dlogits=gd.t)
    gd.check("dlogits")
    want_d = R.route_grad(x, ids, dw.astype(np.float64), score, renorm, scale)
    # the terms' sizes: p (|g| + sum |g| p) at every expert (a score is at most 1 of them)
    p = np.zeros((T, E))
    g = np.zeros((T, E))
    with np.errstate(invalid="ignore"):
        if score == "softmax" and not renorm:
            for i in range(T):
                p[i] = R._scores([float(v) for v in x[i]], score)
        for i, j in np.argwhere(ids >= 0):
            g[i, ids[i, j]] = abs(scale * dw[i, j])
            if not (score == "softmax" and not renorm):
                p[i, ids[i, j]] = want[i, j] / scale if scale else 0.0
        size = p * (g + (g * p).sum(1, keepdims=True))
        tol = (2 * rel + 8 * U) * size + 2.0 ** -120 + (2.0 ** -8 * np.abs(want_d) if bf16 else U * np.abs(want_d))
        if bf16:
            tol = tol + 2.0 ** -134  # half of bf16's smallest step
    close(d.double().cpu().numpy(), want_d, tol)


HOW = [("softmax", False, 1.0), ("softmax", True, 1.0), ("sigmoid", False, 2.5), ("sigmoid", True, 0.5)]


@pytest.mark.parametrize("score,renorm,scale", HOW)
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 4, 4), (17, 31, 2), (9, 32, 8), (50, 33, 6), (8, 64, 1), (40, 160, 8),
                                   (5, 257, 5), (7, 512, 32), (4, 1000, 3), (3, 1024, 32)])
def test_route_and_gradient(T, E, k, bf16, score, renorm, scale):
    check(logits(T, E, T + E + k), k, score, renorm, scale, bf16, 5)


@pytest.mark.parametrize("score,renorm,scale", HOW)
def test_masked_tied_and_strided(score, renorm, scale):
    check(logits(60, 70, 1, masked=0.97), 6, score, renorm, scale, False, 6)  # rows with a few, one, none left
    check(logits(60, 130, 2, step=1.0), 8, score, renorm, scale, False, 7)
    check(logits(60, 257, 3, masked=0.3, step=0.5), 8, score, renorm, scale, True, 8, strided=True)


@pytest.mark.parametrize("score,renorm,scale", HOW)
def test_extreme_logits(score, renorm, scale):
    low = np.finfo(np.float32).min
    x = logits(9, 40, 4)
    x[0] = low                  # a mask of the type's lowest value is an ordinary logit
    x[1] = -np.inf
    x[2] = -np.inf
    x[2, 7] = low
    x[3] *= 40                  # scores below the smallest number
    x[4] -= 500
    x[5] += 500
    x[6, ::2], x[6, 1::2] = 0.0, -0.0
    x[7, 3:] = low
    check(x, 5, score, renorm, scale, False, 9)


@pytest.mark.parametrize("bf16", [False, True])
def test_nan_and_infinity(bf16):
    x = logits(4, 50, 6)
    x[0, [5, 33]] = np.nan
    x[1, 40] = np.inf
    x[2, [2, 9]], x[2, 4] = np.inf, np.nan
    for score, renorm, scale in HOW:
        t = on_gpu(x, bf16)
        ids, w = wq.moe_route(t, 4, score=score, renormalize=renorm, scale=scale)
        want_ids, want = R.route(t.double().cpu().numpy(), 4, score, renorm, scale)
        assert np.array_equal(ids.cpu().numpy(), want_ids)
        w = w.double().cpu().numpy()
        assert np.array_equal(np.isnan(w), np.isnan(want)), (score, renorm)
        ok = ~np.isnan(want)
        assert np.allclose(w[ok], want[ok], rtol=1e-5)
        d = wq.moe_route_grad(t, ids, torch.ones_like(ids, dtype=torch.float32), score=score, renormalize=renorm, scale=scale)
        assert bool(d[3].isfinite().all())  # the ordinary row beside them


def test_every_nan_comes_first():
    """NaN of either sign and any payload, bf16 and float32."""
    pay = np.array([0x7FC00000, 0xFFC00000, 0x7F800001, 0xFF800001, 0xFFFFFFFF, 0x7FFFFFFF], np.uint32)
    x = logits(6, 64, 7)
    for t in range(6):
        x[t, 9 + t] = pay[t:t + 1].view(np.float32)[0]
        x[t, 50] = pay[5 - t:6 - t].view(np.float32)[0]
        x[t, 3] = np.inf
    for t in (torch.from_numpy(x).cuda(), torch.from_numpy((x.view(np.uint32) >> 16 | 1).astype(np.uint16).view(np.int16)).cuda().view(torch.bfloat16)):
        ids, _ = wq.moe_route(t, 3)
        first = 3 if t.dtype == torch.float32 else None  # (bf16's infinity became a NaN here)
        for i in range(6):
            want = [9 + i, 50, 3] if first else [3, 9 + i, 50]
            assert ids[i].tolist() == want, (t.dtype, i)


def test_keys_that_differ_in_their_lowest_bits():
    """Float32 logits that the expert's bits of a key cannot tell apart: among the chosen, at the border, and none."""
    r = np.random.default_rng(11)
    for E, k in ((20, 4), (64, 8), (256, 8), (1024, 32)):
        x = r.standard_normal((40, E)).astype(np.float32)
        x[::2] = (np.float32(1.0) + r.integers(0, 40, (20, E)).astype(np.float32) * np.float32(2.0 ** -23))
        x[1::4] = -x[::4]
        check(x, k, "softmax", True, 1.0, False, 3)


def test_gradient_of_ids_that_are_none_or_twice():
    x = logits(3, 20, 8)
    ids = np.array([[3, -1, 40], [2, 2, 5], [-7, 1 << 30, -1]], np.int32)
    dw = np.random.default_rng(1).standard_normal((3, 3)).astype(np.float32)
    for score, renorm, scale in HOW:
        d = wq.moe_route_grad(torch.from_numpy(x).cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(dw).cuda(),
                              score=score, renormalize=renorm, scale=scale).double().cpu().numpy()
        want = R.route_grad(x.astype(np.float64), ids, dw.astype(np.float64), score, renorm, scale)
        assert np.all(np.abs(d - want) <= 400 * U * np.abs(dw).max() * 3 * scale)


def test_many_tokens_and_empty():
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((40001, 96), generator=g, device="cuda")
    ids, w = wq.moe_route(x, 6, renormalize=True)
    top = torch.topk(x, 6, 1)
    assert torch.equal(ids, top.indices.int())
    assert torch.allclose(w, torch.softmax(top.values, 1), rtol=1e-5)
    for a in (torch.empty((0, 96), device="cuda"), x[:0]):
        ids, w = wq.moe_route(a, 6)
        assert ids.shape == (0, 6) and w.shape == (0, 6)
        assert wq.moe_route_grad(a, ids, w).shape == (0, 96)


def test_refusals():
    x = torch.zeros((4, 8), device="cuda")
    for call, err in [(lambda: wq.moe_route(x.half(), 2), TypeError), (lambda: wq.moe_route(x.T, 2), ValueError),
                      (lambda: wq.moe_route(x, 9), wq.WQError), (lambda: wq.moe_route(x, 0), wq.WQError),
                      (lambda: wq.moe_route(x, 2, score="max"), ValueError),
                      (lambda: wq.moe_route(x[0], 2), ValueError),
                      (lambda: wq.moe_route_grad(x, torch.zeros((3, 2), dtype=torch.int32, device="cuda"), x), ValueError)]:
        with pytest.raises(err):
            call()
