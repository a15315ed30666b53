"""CPU checks of the operators that pick weights by token: pins of their oracle
(closed forms, torch's autograd, differences), and the argument checks of the C
ABI and the binding, which come before any CUDA call."""

import math
import os

import numpy as np
import pytest
import torch

from oracle import choice as R


# ---------------------------------------------------------------- oracle pins

def _chosen(x, ids, score, renorm, scale):
    s = torch.softmax(x, 1) if score == "softmax" else torch.sigmoid(x)
    p = s.gather(1, ids)
    return scale * (p / p.sum(1, keepdim=True) if renorm else p)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_oracle_against_autograd(score, renorm):
    g = torch.Generator().manual_seed(3)
    x = torch.randn((7, 11), generator=g, dtype=torch.float64) * 2
    ids, w = R.route(x.numpy(), 4, score, renorm, 1.5)
    assert np.array_equal(ids, torch.topk(x, 4, 1).indices.numpy())
    x.requires_grad_()
    want = _chosen(x, torch.from_numpy(ids).long(), score, renorm, 1.5)
    assert np.allclose(w, want.detach().numpy(), rtol=1e-12)
    dw = torch.randn((7, 4), generator=g, dtype=torch.float64)
    (grad,) = torch.autograd.grad((want * dw).sum(), x)
    got = R.route_grad(x.detach().numpy(), ids, dw.numpy(), score, renorm, 1.5)
    assert np.allclose(got, grad.numpy(), rtol=1e-10, atol=1e-14)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_oracle_against_differences(score, renorm):
    r = np.random.default_rng(4)
    x, dw = r.standard_normal((2, 6)), r.standard_normal((2, 3))
    ids, _ = R.route(x, 3, score, renorm, 0.7)
    got = R.route_grad(x, ids, dw, score, renorm, 0.7)
    for t, e in np.ndindex(x.shape):
        up, down = x.copy(), x.copy()
        up[t, e] += 1e-6
        down[t, e] -= 1e-6
        f = [(R.route(v, 3, score, renorm, 0.7)[1] * dw).sum() for v in (up, down)]
        assert abs((f[0] - f[1]) / 2e-6 - got[t, e]) < 1e-8


def test_route_oracle_order_and_masks():
    inf, nan = math.inf, math.nan
    x = np.array([[1.0, 2.0, 2.0, -inf, 0.0], [-inf] * 5, [0.0, -0.0, 0.0, -0.0, -1.0], [3.0, nan, inf, 3.0, nan],
                  [-3e38, -inf, -inf, -inf, -inf]])
    ids, w = R.route(x, 3, "softmax", True, 1.0)
    assert ids.tolist() == [[1, 2, 0], [-1] * 3, [0, 1, 2], [1, 4, 2], [0, -1, -1]]
    assert np.allclose(w[2], 1 / 3) and not w[1].any() and np.isnan(w[3]).all() and w[4].tolist() == [1, 0, 0]
    _, w = R.route(np.full((1, 4), -500.0), 2, "sigmoid", True, 1.0)  # each score is below the smallest float32
    assert np.allclose(w, 0.5)
    _, w = R.route(x[:1], 3, "sigmoid", False, 2.0)
    assert np.allclose(w, 2 / (1 + np.exp([-2, -2, -1.0])))


def test_sort_and_combine_oracles_by_hand():
    ids = np.array([[2, 0], [0, 9], [2, 2], [-1, 1]], np.int32)
    offsets, slots, bad = R.sort(ids, 3)
    assert offsets.tolist() == [0, 2, 3, 6] and bad == 2
    assert slots.tolist() == [[3, 0], [1, -1], [4, 5], [-1, 2]]
    y = np.arange(12.0).reshape(6, 2)
    out, size = R.combine(y, slots, np.full((4, 2), 0.5), residual=-np.ones((4, 2)))
    assert out.tolist() == [[2, 3], [0, 0.5], [8, 9], [1, 1.5]] and size[0].tolist() == [4, 5]
    dy, dw, _ = R.combine_grad(np.ones((4, 2)), y, slots, np.array([[1, 2], [3, 4], [5, 6], [7, 8.0]]), np.zeros((6, 2)))
    assert dy[:, 0].tolist() == [2, 3, 8, 1, 5, 6] and dw.tolist() == [[13, 1], [5, 0], [17, 21], [0, 9]]


def test_lora_oracle_is_the_product():
    r = np.random.default_rng(5)
    A, B, x, base = (r.standard_normal(s) for s in ((2, 8, 16), (2, 5, 8), (3, 16), (3, 5)))
    y, _, _ = R.lora(x, A, B, [1, -1, 2], base, [1.0, 0.5])
    assert np.allclose(y[0], base[0] + 0.5 * x[0] @ A[1].T @ B[1].T) and np.array_equal(y[1:], base[1:])


# ---------------------------------------------------------------- refusals

@pytest.fixture(scope="module")
def lib():
    import weight_only_int2_gb300 as wq

    if not os.path.exists(wq.LIB_PATH):
        import __graft_entry__

        __graft_entry__.build()
    return wq.load()


@pytest.fixture(scope="module")
def p():
    """An address that no check below lets a kernel use; with a GPU a real buffer."""
    if torch.cuda.is_available():
        buf = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
        yield buf.data_ptr()
        torch.cuda.synchronize()
    else:
        yield 1 << 20


def refused(lib, name, ok, cases):
    for kw, status, word in cases:
        assert set(kw) <= set(ok)
        assert getattr(lib, name)(*{**ok, **kw}.values()) == status, (name, kw, lib.wq_last_error())
        assert word.encode() in lib.wq_last_error(), (kw, lib.wq_last_error())


ROUTE = [(dict(logits=None), 1, "logits is NULL"), (dict(logits=8), 1, "logits is not 16"), (dict(type=2), 1, "logits_type"),
         (dict(ld=15), 1, "ld must"), (dict(T=-1), 1, "T must"), (dict(E=0), 1, "E must"), (dict(E=1025, ld=1025), 1, "E must"),
         (dict(k=0), 1, "k must"), (dict(k=33), 1, "k must"), (dict(k=17), 1, "at most E"), (dict(T=1 << 30, k=4), 1, "T * k"),
         (dict(score=2), 1, "score must"), (dict(scale=math.inf), 1, "scale must"), (dict(scale=math.nan), 1, "scale must"),
         (dict(ids=None), 1, "ids is NULL"), (dict(ids=2), 1, "ids is not 4")]


def test_route_refusals(lib, p):
    ok = dict(logits=p, type=0, ld=16, T=2, E=16, k=2, score=0, renorm=0, scale=1.0, ids=p, weights=p, stream=None)
    refused(lib, "moe_route", ok, ROUTE + [(dict(weights=None), 1, "weights is NULL")])
    assert lib.moe_route(*{**ok, "T": 0, "logits": None, "ids": None}.values()) == 0
    ok = dict(logits=p, type=0, ld=16, T=2, E=16, k=2, score=0, renorm=0, scale=1.0, ids=p, dw=p, dlogits=p, stream=None)
    refused(lib, "moe_route_grad", ok, ROUTE + [(dict(dw=None), 1, "dweights is NULL"), (dict(dlogits=p + 4), 1, "dlogits is not 16")])
    assert lib.moe_route_grad(*{**ok, "T": 0, "logits": None, "ids": None}.values()) == 0


def test_sort_refusals(lib, p):
    ok = dict(x=p, xs=64, T=2, D=64, ids=p, k=2, E=4, out=p, offsets=p, slots=p, bad=None, stream=None)
    refused(lib, "moe_sort", ok, [
        (dict(x=None), 1, "x is NULL"), (dict(out=None), 1, "out is NULL"), (dict(x=p + 2), 1, "x is not 16"),
        (dict(xs=63), 1, "x_stride"), (dict(D=0), 1, "D must"), (dict(T=-1), 1, "T must"), (dict(k=0), 1, "k must"),
        (dict(k=33), 1, "k must"), (dict(E=0), 1, "E must"), (dict(E=1025), 1, "E must"), (dict(ids=None), 1, "ids is NULL"),
        (dict(offsets=None), 1, "offsets is NULL"), (dict(offsets=p + 2), 1, "offsets is not 4"),
        (dict(slots=None), 1, "slots is NULL"), (dict(bad=p + 1), 1, "bad_count"), (dict(T=1 << 30), 1, "T * k")])


def test_combine_refusals(lib, p):
    ok = dict(y=p, R=4, slots=p, weights=p, residual=p, T=2, D=64, k=2, out=p, stream=None)
    refused(lib, "moe_combine", ok, [
        (dict(y=None), 1, "y is NULL"), (dict(R=0), 1, "R must"), (dict(slots=None), 1, "slots is NULL"),
        (dict(weights=p + 2), 1, "weights is not 4"), (dict(residual=p + 2), 1, "residual is not 16"), (dict(T=-1), 1, "T must"),
        (dict(D=0), 1, "D must"), (dict(k=0), 1, "k must"), (dict(k=33), 1, "k must"), (dict(out=None), 1, "out is NULL")])
    assert lib.moe_combine(*{**ok, "T": 0, "y": None, "out": None}.values()) == 0
    ok = dict(dout=p, y=p, R=4, slots=p, weights=p, T=2, D=64, k=2, dy=p, dw=p, stream=None)
    refused(lib, "moe_combine_grad", ok, [
        (dict(dout=None), 1, "dout is NULL"), (dict(y=p + 8), 1, "y is not 16"), (dict(R=0), 1, "R must"),
        (dict(slots=None), 1, "slots is NULL"), (dict(weights=None), 1, "weights is NULL"), (dict(T=-1), 1, "T must"),
        (dict(D=0), 1, "D must"), (dict(k=33), 1, "k must"), (dict(dy=None), 1, "dy is NULL"),
        (dict(dw=None), 1, "dweights is NULL")])
    assert lib.moe_combine_grad(*{**ok, "T": 0, "y": None, "dy": None}.values()) == 0


def test_no_tokens_after_a_sort_of_none(lib, p):
    # what moe_sort gives for no tokens has no rows
    assert lib.moe_combine(None, 0, None, None, None, 0, 64, 2, None, None) == 0
    assert lib.moe_combine_grad(None, None, 0, None, None, 0, 64, 2, None, None, None) == 0
    for n in (-1, 1 << 31):
        assert lib.moe_combine(p, n, p, p, p, 0, 64, 2, p, None) == 1 and b"R must" in lib.wq_last_error()
        assert lib.moe_combine_grad(p, p, n, p, p, 0, 64, 2, p, p, None) == 1 and b"R must" in lib.wq_last_error()


def test_lora_refusals(lib, p):
    need = lib.lora_workspace_bytes(3, 2, 16)
    assert need > 0 and lib.lora_workspace_bytes(0, 2, 16) == 0 and lib.lora_workspace_bytes(3, 2, 256) == 0
    ok = dict(x=p + 16384, xs=64, M=3, K=64, A=p, B=p, n=2, r=16, N=40, adapter=p, scale=None, base=p, bs=40, y=p + 4096,
              ys=40, ws=p, wsb=need, stream=None)
    refused(lib, "lora_gemm", ok, [
        (dict(x=None), 1, "x is NULL"), (dict(x=p + 8), 1, "x is not 16"), (dict(xs=56), 1, "x_stride"), (dict(xs=68), 1, "x_stride"),
        (dict(M=-1), 1, "M must"), (dict(K=0), 1, "K must"), (dict(K=60), 1, "K must"), (dict(N=0), 1, "N must"),
        (dict(n=0), 1, "n must"), (dict(n=1025), 1, "n must"), (dict(r=0), 2, "r must"), (dict(r=12), 2, "r must"),
        (dict(r=136), 2, "r must"), (dict(A=None), 1, "A is NULL"), (dict(B=p + 2), 1, "B is not 16"),
        (dict(adapter=None), 1, "adapter is NULL"), (dict(adapter=p + 2), 1, "adapter is not 4"), (dict(scale=p + 2), 1, "scale is not 4"),
        (dict(base=None), 1, "base is NULL"), (dict(base=p + 1), 1, "base is not 2"), (dict(bs=39), 1, "base_stride"),
        (dict(y=None), 1, "y is NULL"), (dict(ys=39), 1, "y_stride"), (dict(y=p, ys=48), 1, "y is base"),
        (dict(y=p + 2), 1, "y must be base"), (dict(y=p + 80), 1, "y must be base"), (dict(y=p + 80, ys=48), 1, "y must be base"),
        (dict(bs=100, y=p + 78, ys=100), 1, "y must be base"), (dict(bs=100, y=p + 122, ys=100), 1, "y must be base"),
        (dict(base=p + 80, bs=100, y=p + 202, ys=100), 1, "y must be base"), (dict(y=p + 16384), 1, "y must not overlap x"),
        (dict(y=p + 16384 - 2), 1, "y must not overlap x"), (dict(y=p + 16384 + 2 * (2 * 64 + 63)), 1, "y must not overlap x"),
        (dict(ws=None), 1, "workspace is NULL"), (dict(wsb=need - 1), 1, "workspace too small"), (dict(ws=p + 8), 1, "workspace is not 16")])
    assert lib.lora_gemm(*{**ok, "M": 0, "x": None, "y": None}.values()) == 0
    # side by side in one buffer, or one behind the other: the next check is reached
    refused(lib, "lora_gemm", {**ok, "ws": None}, [
        (kw, 1, "workspace is NULL") for kw in (dict(y=p), dict(y=p + 240), dict(base=p + 240, y=p), dict(bs=100, y=p + 80, ys=100),
                                                dict(bs=100, y=p + 120, ys=100), dict(base=p + 80, bs=100, y=p, ys=100),
                                                dict(xs=128, y=p + 16384 + 128, ys=128), dict(y=p + 16384 - 240))])


def test_binding_refuses_cpu_tensors():
    import weight_only_int2_gb300 as wq

    i, f, h = torch.zeros((2, 2), dtype=torch.int32), torch.zeros((2, 2)), torch.zeros((4, 8), dtype=torch.bfloat16)
    w = torch.zeros((1, 8, 8), dtype=torch.bfloat16)
    for call in (lambda: wq.moe_route(f, 1), lambda: wq.moe_route_grad(f, i, f), lambda: wq.moe_sort(h, i, 2),
                 lambda: wq.moe_combine(h, i), lambda: wq.moe_combine_grad(h, h, i, f),
                 lambda: wq.lora_gemm(h, w, w, torch.zeros(4, dtype=torch.int32), h)):
        with pytest.raises(ValueError, match="must be a CUDA tensor"):
            call()


def test_the_workspace_holds_every_share_of_the_first_product():
    """The sizes behind lora_workspace_bytes, for any split of the rows into tiles: with G blocks, t tiles of at most
    tile rows and s = min(32, max(1, G // t)) shares, the s * rows partial sums lie inside, and with many rows two bf16
    numbers for each value of each tile."""
    import weight_only_int2_gb300 as wq

    for M in (1, 2, 15, 16, 17, 100, 511, 512, 513, 4000, 70000):
        tile = 8 if M < 512 else 64
        for n in (1, 3, 1024):
            for r in (8, 128):
                have = wq.lora_workspace_bytes(M, n, r)
                most = M // tile + min(M, n + 1)
                head = 16 * (1 + most) + -(-4 * M // 16) * 16
                if tile == 64 and r > 32:
                    head += most * 64 * 128 * 4
                for rows in {1, min(M, 7), M // 2 + 1, M}:
                    for groups in {1, min(n, rows)}:
                        per = -(-rows // groups)
                        tiles = sum(-(-min(per, rows - at) // tile) for at in range(0, rows, per))
                        assert tiles <= most
                        for G in (1, 152, 1024):
                            shares = min(32, max(1, G // tiles))
                            assert head + shares * rows * r * 4 <= have, (M, n, r, rows, groups, G)
