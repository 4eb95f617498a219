"""Pins of the cross attention and rotary oracles (no GPU): torch's fp64 attention and autograd, central
differences, closed forms, complex rotation."""

import math

import numpy as np
import pytest
import torch

from oracle import cross as oc


def _inputs(B, Hq, Hkv, Nq, Nk, d, seed):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(B, Hq, Nq, d, generator=g, dtype=torch.float64)
    k, v = (torch.randn(B, Hkv, Nk, d, generator=g, dtype=torch.float64) for _ in range(2))
    return q, k, v, torch.randn(B, Hq, Nq, d, generator=g, dtype=torch.float64)


@pytest.mark.parametrize("B,Hq,Hkv,Nq,Nk,lens", [(2, 4, 2, 5, 7, None), (3, 3, 1, 4, 6, [6, 1, 0]),
                                                 (1, 2, 2, 1, 9, [5])])
def test_cross_oracle_matches_torch_and_autograd(B, Hq, Hkv, Nq, Nk, lens):
    q, k, v, do = _inputs(B, Hq, Hkv, Nq, Nk, 8, 3)
    o, lse, _, _ = oc.cross_attention(q, k, v, 0.3, lens)
    grads, _ = oc.cross_backward(q, k, v, do, 0.3, lens)
    for b, n in enumerate(lens or [Nk] * B):
        if n == 0:
            assert (o[b] == 0).all() and np.isneginf(lse[b]).all() and (grads["dq"][b] == 0).all()
            assert (grads["dk"][b] == 0).all() and (grads["dv"][b] == 0).all()
            continue
        x = [t[b:b + 1].clone().requires_grad_() for t in (q, k, v)]
        kk, vv = (t[:, :, :n].repeat_interleave(Hq // Hkv, 1) for t in x[1:])
        ref = torch.nn.functional.scaled_dot_product_attention(x[0], kk, vv, scale=0.3)
        np.testing.assert_allclose(o[b], ref[0].detach(), atol=1e-13)
        np.testing.assert_allclose(lse[b], torch.logsumexp(0.3 * x[0] @ kk.transpose(-1, -2), -1)[0].detach(), atol=1e-13)
        for name, g in zip(("dq", "dk", "dv"), torch.autograd.grad(ref, x, do[b:b + 1])):
            np.testing.assert_allclose(grads[name][b], g[0], atol=1e-12)


def test_cross_oracle_gradients_match_differences():
    q, k, v, do = _inputs(1, 4, 2, 3, 5, 8, 4)
    grads, _ = oc.cross_backward(q, k, v, do, 0.4, [4])
    loss = lambda: float((oc.cross_attention(q, k, v, 0.4, [4])[0] * do.numpy()).sum())  # noqa: E731
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
            assert abs((up - down) / (2 * h) - grads[name].reshape(-1)[i]) < 1e-8


def test_rope_oracle_is_a_rotation_by_complex_numbers():
    g = torch.Generator().manual_seed(5)
    x = torch.randn(2, 3, 7, 16, generator=g, dtype=torch.float64)
    pos = torch.randint(-50, 5000, (2, 2, 7), generator=g)
    for cyclic in (False, True):
        for per_axis in (False, True):
            axis, rates = oc.rope_rates(16, (3, 5), 100.0, per_axis, cyclic)
            assert axis == ([0, 1, 0, 1, 0, 1, 1, 1] if cyclic else [0] * 3 + [1] * 5)
            for inter in (False, True):
                y, _ = oc.rope(x, pos, axis, rates, inter)
                pair = (lambda t: t[..., 0::2] + 1j * t[..., 1::2]) if inter else (lambda t: t[..., :8] + 1j * t[..., 8:])
                ang = np.stack([pos[a].numpy() * float(r) for a, r in zip(axis, rates)], -1)[:, None]
                np.testing.assert_allclose(pair(y), pair(x.numpy()) * np.exp(1j * ang), atol=1e-11)
                back, _ = oc.rope(y, pos, axis, rates, inter, inverse=True)
                np.testing.assert_allclose(back, x, atol=1e-13)
    _, rates = oc.rope_rates(16, (8,))
    np.testing.assert_allclose(np.float64(rates), 10000.0 ** (-np.arange(8) / 8.0), rtol=1e-15)
    _, rates = oc.rope_rates(16, (4, 4), 100.0, per_axis=True)
    np.testing.assert_allclose(np.float64(rates), [100.0 ** (-j / 4) for j in range(4)] * 2, rtol=1e-15)


def test_cross_bounds_cover_a_rounded_evaluation():
    """The bound of cross_backward is one: an evaluation with P and dS rounded to bf16 stays inside it."""
    q, k, v, do = (t.to(torch.bfloat16).double() for t in _inputs(1, 2, 1, 40, 30, 64, 6))
    scale = 1 / math.sqrt(64)
    rel = torch.finfo(torch.bfloat16).eps / 2
    grads, bound = oc.cross_backward(q, k, v, do, scale, None, rel=rel)
    kk, vv = k.repeat_interleave(2, 1), v.repeat_interleave(2, 1)
    p = torch.softmax(scale * q @ kk.transpose(-1, -2), -1)
    o = p @ vv
    ds = p * (do @ vv.transpose(-1, -2) - (o * do).sum(-1, keepdim=True))
    p, ds = p.to(torch.bfloat16).double(), ds.to(torch.bfloat16).double()
    dq, dk, dv = scale * ds @ kk, scale * (ds.transpose(-1, -2) @ q).sum(1), (p.transpose(-1, -2) @ do).sum(1)
    for name, got in (("dq", dq), ("dk", dk[:, None]), ("dv", dv[:, None])):
        assert (np.abs(got.numpy() - grads[name]) <= bound[name] + 1e-14).all(), name
        assert (bound[name] <= 0.2 * np.abs(grads[name]).mean() * 10).mean() > 0.9  # and not an empty one
