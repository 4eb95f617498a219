"""The weights' gradients of fa_norm_rope_axes_bwd over many rows: blocks that walk several groups of rows, every partial sum.

Bound.  A term g n of dw has g off by far = 2^-21 + |pos| 2^-48 of its pair's |a| + |b| (tests/test_gpu_norm_rope.py), and n = x r
by r's 2^-20 and the products' 2 2^-24: below rel = 2^-19 of |g n|.  The terms are added in fp32 in chains: a thread's over its
groups of rows and heads, a block's over the threads that hold the same columns, a lane's over every 128th partial sum; each
addition is off by 2^-24 of at most the terms' absolute sum.  The lanes are joined in fp64 and rounded once (2^-24 of dw).
With L the chains' lengths together, |dw - ref| <= sum |g n| (rel + L 2^-24 (1 + 2^-10)) + far sum (|a| + |b|) |n| +
2^-24 |ref| (1 + 2^-10)."""

import numpy as np
import pytest
import torch

from _util import ensure_built
from exact_attention_06_gb300 import fattn, inputs
from oracle import cross as oc
from oracle import window as ow

pytestmark = pytest.mark.gpu
DEV = "cuda"
LANES = 128  # of a column of the last sums


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _rows_of_a_block(d):
    return 128 // (d // 16)


def _chains(B, Hq, Hk, N, d):
    """The longest chains together, and the fewest groups of rows that a block walks, over every way in which heads can be
    shared out to the partial sums that the workspace holds."""
    rows = _rows_of_a_block(d)
    groups = -(-B * N // rows)
    partials = fattn.fa_norm_rope_axes_bwd_workspace_bytes(B, Hq, Hk, N, d) // (4 * d)
    found = []
    for heads in range(1, 17):
        y = -(-Hq // heads) + -(-Hk // heads)
        if partials % y == 0 and partials // y <= groups:
            walks = -(-groups // (partials // y))
            found.append((walks * heads + rows + -(-partials // LANES), walks))
    return max(f[0] for f in found), min(f[1] for f in found)


# (walks: groups of rows that a block takes at least)
@pytest.mark.parametrize("B,Hq,Hk,N,d,walks", [(3, 3, 1, 10001, 128, 4), (3, 3, 1, 25001, 64, 4), (1, 16, 2, 12001, 128, 2),
                                               (1, 2, 0, 60001, 64, 2), (7, 1, 1, 4099, 128, 3), (2, 16, 4, 3001, 128, 1)])
def test_every_partial_sum_counts(B, Hq, Hk, N, d, walks):
    eps, R = 1e-6, _rows_of_a_block(d)
    length, least = _chains(B, Hq, Hk, N, d)
    assert least >= walks
    q, gq = inputs.normal_bf16((B, Hq, N, d), 1, DEV), inputs.normal_bf16((B, Hq, N, d), 5, DEV)
    k, gk = (inputs.normal_bf16((B, Hk, N, d), s, DEV) if Hk else None for s in (2, 6))
    w = [(1 + 0.3 * torch.randn(d, generator=torch.Generator().manual_seed(s))).to(DEV) for s in (3, 4)]
    pos = torch.randint(-4096, 4096, (1, B, N), generator=torch.Generator().manual_seed(7), dtype=torch.int32)
    plan = fattn.fa_rope_axes_plan(d, (d // 2,), 10000.0)
    axis, rates = oc.rope_rates(d, (d // 2,), 10000.0)
    dw = [torch.full((d,), float("nan"), device=DEV) for _ in range(2)]
    dq, dk = torch.empty_like(q), torch.empty_like(k) if Hk else None
    fattn.fa_norm_rope_axes_bwd(q, k, w[0], w[1], pos.to(DEV), plan, gq, gk, dq, dk, dw[0], dw[1] if Hk else None, eps=eps)
    assert fattn.fa_get_status() == fattn.FA_OK
    far = 2.0 ** -21 + float(pos.abs().max()) * 2.0 ** -48
    for what, x, g, wt, got in (("q", q, gq, w[0], dw[0]), ("k", k, gk, w[1], dw[1]))[:2 if Hk else 1]:
        ref = np.zeros(d)
        err, size = np.zeros(d), np.zeros(d)
        for h in range(x.shape[1]):  # (a head at a time: the oracle holds many fp64 copies)
            _, rw, _, ew, abs_w = ow.norm_rope_backward(x[:, h:h + 1], wt, g[:, h:h + 1], pos, axis, rates, False, eps, far=far,
                                                        rel=2.0 ** -19)
            ref, err, size = ref + rw, err + ew, size + abs_w
        bound = err + (1 + 2.0 ** -10) * 2.0 ** -24 * (length * size + np.abs(ref))
        off = np.abs(got.cpu().double().numpy() - ref)
        assert (off <= bound).all(), f"{what}: {float((off / bound).max()):.2f} of the bound"
        # the bound notices the rows that a block takes at one time, of one head, if they are left out
        for n0 in (0, N // 2, N - R):
            one = slice(n0, n0 + R)
            rw = ow.norm_rope_backward(x[:1, :1, one], wt, g[:1, :1, one], pos[:, :1, one], axis, rates, False, eps)[1]
            assert (np.abs(rw) > 2 * bound).any(), "the bound is too wide"
