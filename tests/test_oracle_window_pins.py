"""Pins of the sliding-window, norm and page oracles (no GPU): torch's fp64 autograd, central differences, closed forms."""

import math

import numpy as np
import pytest
import torch

from oracle import cross as oc
from oracle import window as ow


def _inputs(B, Hq, Hkv, N, Nk, d, seed):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(B, Hq, N, d, generator=g, dtype=torch.float64)
    k, v = (torch.randn(B, Hkv, Nk, d, generator=g, dtype=torch.float64) for _ in range(2))
    return q, k, v, torch.randn(B, Hq, N, d, generator=g, dtype=torch.float64)


SHAPES = [(2, 4, 2, 7, 7, 3, 0), (1, 3, 1, 6, 9, 2, 2), (1, 2, 2, 1, 5, 1, 1), (1, 2, 2, 5, 5, 100, 0), (2, 2, 1, 8, 11, 1, 0)]


@pytest.mark.parametrize("B,Hq,Hkv,N,Nk,W,S", SHAPES)
def test_window_oracle_matches_torch_and_autograd(B, Hq, Hkv, N, Nk, W, S):
    q, k, v, do = _inputs(B, Hq, Hkv, N, Nk, 8, 3)
    o, lse, _, _ = ow.window_attention(q, k, v, 0.3, W, S)
    grads, _ = ow.window_backward(q, k, v, do, 0.3, W, S)
    see = torch.tensor([[j <= i + Nk - N and (i + Nk - N - j < W or j < S) for j in range(Nk)] for i in range(N)])
    x = [t.clone().requires_grad_() for t in (q, k, v)]
    kk, vv = (t.repeat_interleave(Hq // Hkv, 1) for t in x[1:])
    ref = torch.nn.functional.scaled_dot_product_attention(x[0], kk, vv, attn_mask=see, scale=0.3)
    np.testing.assert_allclose(o, ref.detach(), atol=1e-13)
    score = (0.3 * x[0] @ kk.transpose(-1, -2)).masked_fill(~see, -math.inf)
    np.testing.assert_allclose(lse, torch.logsumexp(score, -1).detach(), atol=1e-13)
    for name, g in zip(("dq", "dk", "dv"), torch.autograd.grad(ref, x, do)):
        np.testing.assert_allclose(grads[name], g, atol=1e-12)


def test_window_oracle_limits():
    q, k, v, _ = _inputs(1, 2, 2, 6, 6, 8, 1)
    o, lse, _, _ = ow.window_attention(q, k, v, 0.3, 1)
    np.testing.assert_allclose(o, v, atol=1e-13)  # its own key alone
    np.testing.assert_allclose(lse, 0.3 * (q * k).sum(-1), atol=1e-13)
    from oracle import attention
    causal, _ = attention(q, k, v, 0.3, True)
    for W, S in ((6, 0), (99, 3), (1, 6)):
        np.testing.assert_allclose(ow.window_attention(q, k, v, 0.3, W, S)[0], np.asarray(causal).reshape(o.shape), atol=1e-12)
    # what no query sees has no influence: keys 1 .. 3 of eight, for the last three queries
    q, k, v, do = _inputs(1, 1, 1, 3, 8, 8, 2)
    a, ga = ow.window_attention(q, k, v, 0.3, 2, 1), ow.window_backward(q, k, v, do, 0.3, 2, 1)[0]
    k[:, :, 1:4], v[:, :, 1:4] = math.nan, math.inf
    b, gb = ow.window_attention(q, k, v, 0.3, 2, 1), ow.window_backward(q, k, v, do, 0.3, 2, 1)[0]
    assert np.array_equal(a[0], b[0]) and all(np.array_equal(ga[n], gb[n]) for n in ga)
    assert (gb["dk"][:, :, 1:4] == 0).all() and (gb["dv"][:, :, 1:4] == 0).all()


def test_window_gradients_match_differences():
    q, k, v, do = _inputs(1, 4, 2, 5, 7, 8, 4)
    grads, _ = ow.window_backward(q, k, v, do, 0.4, 3, 1)
    loss = lambda: float((ow.window_attention(q, k, v, 0.4, 3, 1)[0] * do.numpy()).sum())  # noqa: E731
    h = 1e-5
    for name, x in (("dq", q), ("dk", k), ("dv", v)):
        flat = x.view(-1)
        for i in range(0, flat.numel(), 7):
            at = float(flat[i])
            flat[i] = at + h
            up = loss()
            flat[i] = at - h
            down = loss()
            flat[i] = at
            assert abs((up - down) / (2 * h) - grads[name].reshape(-1)[i]) < 1e-7


def test_decode_is_the_last_row():
    q, k, v, _ = _inputs(2, 4, 2, 1, 9, 8, 5)
    o, lse, _, _ = ow.window_decode(q[:, :, 0], k, v, [9, 0], 0.3, 4, 2)
    want, wl, _, _ = ow.window_attention(q[:1], k[:1], v[:1], 0.3, 4, 2)
    assert np.array_equal(o[0], want[0, :, 0]) and np.array_equal(lse[0], wl[0, :, 0])
    assert (o[1] == 0).all() and np.isneginf(lse[1]).all()


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("weight", [False, True])
def test_norm_rope_matches_complex_autograd_and_differences(inter, weight):
    g = torch.Generator().manual_seed(1)
    x, dy = (torch.randn(2, 3, 5, 8, generator=g, dtype=torch.float64) for _ in range(2))
    w = torch.randn(8, generator=g, dtype=torch.float64) if weight else None
    pos = torch.randint(-50, 50, (2, 2, 5), generator=g)
    axis, rates = oc.rope_rates(8, (1, 3), 100.0)
    ref = lambda x, w: _turned(x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-3) * (1 if w is None else w),  # noqa: E731
                               pos, axis, rates, inter)
    y, _ = ow.norm_rope(x, w, pos, axis, rates, inter, 1e-3)
    np.testing.assert_allclose(y, ref(x, w), atol=1e-13)
    dx, dw, _, _, _ = ow.norm_rope_backward(x, w, dy, pos, axis, rates, inter, 1e-3)
    xs, ws = x.clone().requires_grad_(), (torch.ones(8, dtype=torch.float64) if w is None else w).clone().requires_grad_()
    gx, gw = torch.autograd.grad(ref(xs, ws), (xs, ws), dy)
    np.testing.assert_allclose(dx, gx, atol=1e-12)
    np.testing.assert_allclose(dw, gw, atol=1e-12)
    h = 1e-6
    for i in range(0, x.numel(), 17):
        side = []
        for s in (h, -h):
            z = x.clone()
            z.view(-1)[i] += s
            side.append(float((ow.norm_rope(z, w, pos, axis, rates, inter, 1e-3)[0] * dy.numpy()).sum()))
        assert abs((side[0] - side[1]) / (2 * h) - dx.reshape(-1)[i]) < 1e-6


def _turned(x, pos, axis, rates, inter):
    n = x.shape[-1] // 2
    z = torch.view_as_complex(x.unflatten(-1, (n, 2)).contiguous() if inter else
                              x.unflatten(-1, (2, n)).transpose(-1, -2).contiguous())
    angle = torch.stack([pos[a].double() * float(r) for a, r in zip(axis, rates)], -1)[:, None]
    y = torch.view_as_real(z * torch.polar(torch.ones_like(angle), angle))
    return (y if inter else y.transpose(-1, -2)).flatten(-2)


def test_pages_by_hand():
    table, lens, stack = [[7, -1, -1], [-1, -1, -1], [3, 5, -1]], [64, 0, 70], [9, 8, 4, 2, 0, 0, 0, 0, 0, 0]
    t, n, s, f, granted, slots = ow.pages_extend(table, lens, [1, 64, -40], stack, 4, 64, 2)
    assert t == [[7, 2, -1], [4, -1, -1], [3, -1, -1]] and n == [65, 64, 30] and granted == [1, 64, -40]
    assert slots == [[128, -1], [256, 257], [-1, -1]]
    assert f == 3 and s[:3] == [9, 8, 5]
    # back again: the stack and the table's pages as they were
    t, n, s, f, granted, _ = ow.pages_extend(t, n, [-1, -64, 40], s, f, 64)
    assert n == lens and f == 4 and t == [[7, -1, -1], [-1, -1, -1], [3, 5, -1]] and s[:4] == [9, 8, 4, 2]
    # out of pages: none from the first that cannot be served on; room in the last page is; so is a table's end
    t, n, s, f, granted, _ = ow.pages_extend([[0, -1], [1, -1], [2, -1], [3, -1]], [64, 64, 63, 64], [64, 1, 1, 65],
                                             [6, 7, 0, 0, 0, 0, 0, 0], 1, 64)
    assert granted == [64, 0, 1, 0] and n == [128, 64, 64, 64] and t[0] == [0, 6] and f == 0
