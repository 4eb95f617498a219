"""Rotary positions with several axes on the GPU, against the fp64 definition.

Bound of an output: half a bf16 step of the value, plus the fp32 arithmetic before it.  The half turns
are an integer's top 32 bits rounded to fp32: off by at most 2^-25 (of values up to 1) and 2^-32, so the
angle by pi times that, < 2^-23.  cos and sin are within 2 fp32 ulps (2^-23 of at most 1), products and
sum within 2^-24 each of at most |a| + |b|: together < 2^-21 (|a| + |b|).  The plan's rate is within
(4 + ln base) 2^-53 and 2^-65 turns, times the position: for |pos| < 2^24 below 2^-24, else
|pos| * 2^-48 at most (base <= 1e6)."""

import itertools

import numpy as np
import pytest
import torch

from _util import ensure_built
from exact_attention_06_gb300 import fattn, inputs
from oracle import cross as oc

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _pos(axes, B, N, seed, high=4096):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-high, high, (axes, B, N), generator=g, dtype=torch.int64).to(torch.int32)


def _check(y, x, pos, d, sections, base, inter, per_axis, cyclic, inverse=False, what=""):
    axis, rates = oc.rope_rates(d, sections, base, per_axis, cyclic)
    ref, size = oc.rope(x, pos, axis, rates, inter, inverse)
    far = 2.0 ** -21 + float(np.abs(pos.numpy().astype(np.float64)).max()) * 2.0 ** -48
    tol = np.abs(ref) * 2.0 ** -8 + size * far * (1 + 2.0 ** -8) + 1e-38
    err = np.abs(y.cpu().double().numpy() - ref)
    assert np.isfinite(err).all() and (err <= tol).all(), f"{what}: {float((err / tol).max()):.2f} of the bound"


SECTIONS = {64: [(32,), (16, 16), (8, 12, 12), (1, 2, 3, 26)], 128: [(64,), (32, 32), (16, 24, 24), (5, 7, 11, 41)]}


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n_axes", [1, 2, 3, 4])
@pytest.mark.parametrize("inter,per_axis,cyclic", list(itertools.product([False, True], repeat=3)))
def test_every_form_and_its_gradient(d, n_axes, inter, per_axis, cyclic):
    sections = SECTIONS[d][n_axes - 1]
    B, Hq, Hk, N = 2, 5, 2, 37
    q, k = inputs.normal_bf16((B, Hq, N, d), 1, DEV), inputs.normal_bf16((B, Hk, N, d), 2, DEV)
    pos = _pos(n_axes, B, N, 3)
    plan = fattn.fa_rope_axes_plan(d, sections, 10000.0, inter, per_axis, cyclic)
    qo, ko = torch.full_like(q, float("nan")), torch.full_like(k, float("nan"))
    fattn.fa_rope_axes(q, k, pos.to(DEV), plan, qo, ko)
    args = (pos, d, sections, 10000.0, inter, per_axis, cyclic)
    _check(qo, q, *args, what="q")
    _check(ko, k, *args, what="k")
    # the gradients of q and k are the outputs' turned back (in place here)
    gq, gk = inputs.normal_bf16((B, Hq, N, d), 4, DEV), inputs.normal_bf16((B, Hk, N, d), 5, DEV)
    gq0, gk0 = gq.clone(), gk.clone()
    fattn.fa_rope_axes(gq, gk, pos.to(DEV), plan, inverse=True)
    _check(gq, gq0, *args, inverse=True, what="dq")
    _check(gk, gk0, *args, inverse=True, what="dk")
    # by differences: the map is linear, so <R x, g> - <0, g> = <x, R^T g> up to both sides' rounding
    left, right = (qo.double() * gq0.double()).sum(), (q.double() * gq.double()).sum()
    bound = 2.0 ** -7 * ((qo.double() * gq0.double()).abs().sum() + (q.double() * gq.double()).abs().sum())
    assert abs(left - right) <= bound


@pytest.mark.parametrize("B,Hq,Hk,N", [(1, 1, 0, 1), (1, 1, 1, 1), (3, 4, 1, 2), (1, 9, 3, 31), (2, 33, 17, 65),
                                       (1, 3, 3, 1025), (5, 2, 0, 257), (1, 64, 8, 16)])
@pytest.mark.parametrize("d", [64, 128])
def test_sizes(B, Hq, Hk, N, d):
    q = inputs.normal_bf16((B, Hq, N, d), 1, DEV)
    k = inputs.normal_bf16((B, Hk, N, d), 2, DEV) if Hk else None
    pos = _pos(3, B, N, 3)
    sections = SECTIONS[d][2]
    plan = fattn.fa_rope_axes_plan(d, sections, 500000.0)
    guard = [torch.full((t.numel() + 512,), 7.0, dtype=torch.bfloat16, device=DEV) for t in (q, k) if t is not None]
    outs = [g[256:-256].view(t.shape) for g, t in zip(guard, (q, k))]
    fattn.fa_rope_axes(q, k, pos.to(DEV), plan, *outs)
    for y, x, g in zip(outs, (q, k), guard):
        _check(y, x, pos, d, sections, 500000.0, False, False, False)
        assert (g[:256] == 7).all() and (g[-256:] == 7).all()


def test_far_positions_keep_their_angles():
    d, N = 128, 64
    q = inputs.normal_bf16((1, 2, N, d), 1, DEV)
    for high in (2 ** 24, 2 ** 31 - 1):
        pos = _pos(2, 1, N, 3, high=high)
        pos[0, 0, :4] = torch.tensor([-2 ** 31, 2 ** 31 - 1, 0, -1]) if high > 2 ** 24 else torch.tensor([2 ** 24, 0, -1, 1])
        plan = fattn.fa_rope_axes_plan(d, (32, 32), 1e6)
        y = torch.empty_like(q)
        fattn.fa_rope_axes(q, None, pos.to(DEV), plan, y)
        _check(y, q, pos, d, (32, 32), 1e6, False, False, False, what=f"positions to {high}")
    zero = torch.zeros(2, 1, N, dtype=torch.int32, device=DEV)
    fattn.fa_rope_axes(q, None, zero, plan, y)
    assert torch.equal(y, q)  # position 0 turns nothing


def test_infinities_and_nan_stay_in_their_pair():
    d, N = 64, 8
    q = inputs.normal_bf16((1, 1, N, d), 1, DEV)
    bad = q.clone()
    bad[0, 0, 3, 5], bad[0, 0, 4, 40] = float("inf"), float("nan")
    pos = _pos(1, 1, N, 3).to(DEV)
    plan = fattn.fa_rope_axes_plan(d, (32,))
    good, y = torch.empty_like(q), torch.empty_like(q)
    fattn.fa_rope_axes(q, None, pos, plan, good)
    fattn.fa_rope_axes(bad, None, pos, plan, y)
    same = y == good
    same[0, 0, 3, [5, 37]] = True
    same[0, 0, 4, [8, 40]] = True
    assert same.all() and not torch.isfinite(y[0, 0, 3, [5, 37]]).any() and torch.isnan(y[0, 0, 4, [8, 40]]).all()


def test_an_offset_past_32_bits():
    # 2^31 elements of q and then some: the last rows and heads
    B, H, N, d = 1, 33, 2 ** 19, 128
    q = torch.zeros(B, H, N, d, dtype=torch.bfloat16, device=DEV)
    q[:, -1, -5:] = inputs.normal_bf16((5, d), 1, DEV)
    x = q[:, -1:, -5:].cpu()
    pos = torch.arange(N, dtype=torch.int32, device=DEV).view(1, 1, N)
    plan = fattn.fa_rope_axes_plan(d, (64,))
    fattn.fa_rope_axes(q, None, pos, plan)
    _check(q[:, -1:, -5:], x, pos[:, :, -5:].cpu(), d, (64,), 10000.0, False, False, False)


@pytest.mark.parametrize("d,ps,N,inter", [(64, 64, 1, False), (128, 64, 1, True), (128, 128, 70, False),
                                          (64, 192, 333, True)])
@pytest.mark.parametrize("ragged", [False, True])
def test_paged_append(d, ps, N, inter, ragged):
    B, Hq, Hk, mp = 4, 6, 3, 9
    q = inputs.normal_bf16((B, Hq, N, d), 1, DEV)
    k, v = inputs.normal_bf16((B, Hk, N, d), 2, DEV), inputs.normal_bf16((B, Hk, N, d), 3, DEV)
    P = B * mp
    kp, vp = inputs.normal_bf16((P, Hk, ps, d), 4, DEV), inputs.normal_bf16((P, Hk, ps, d), 5, DEV)
    kp0, vp0 = kp.clone(), vp.clone()
    table = torch.randperm(P, generator=torch.Generator().manual_seed(6)).to(torch.int32).view(B, mp)
    # a page boundary inside the chunk; from nothing; the table's last rows; past the table's end
    lens = torch.tensor([ps - 1, 0, mp * ps - N, mp * ps - N // 2], dtype=torch.int32)
    table[1, 0] = -1          # no page
    table[2, mp - 1] = P      # outside the pool
    new = torch.tensor([N, max(N // 2, 1), N, 0], dtype=torch.int32) if ragged else None
    pos = _pos(2, B, N, 7)
    sections = SECTIONS[d][1]
    plan = fattn.fa_rope_axes_plan(d, sections, interleaved=inter)
    qo = torch.full_like(q, 9.0)
    fattn.fa_rope_axes_paged(q, k, v, pos.to(DEV), plan, qo, kp, vp, table.to(DEV), lens.to(DEV),
                             new.to(DEV) if ragged else None)
    turned = torch.empty_like(k)
    want_q = torch.empty_like(q)
    fattn.fa_rope_axes(q, k, pos.to(DEV), plan, want_q, turned)  # (checked above)
    for b in range(B):
        n = int(new[b]) if ragged else N
        assert torch.equal(qo[b, :, :n], want_q[b, :, :n]) and (qo[b, :, n:] == 9).all()
        for t in range(n):
            key = int(lens[b]) + t
            page = int(table[b, key // ps]) if key // ps < mp else -1
            if 0 <= page < P:
                kp0[page, :, key % ps] = turned[b, :, t]
                vp0[page, :, key % ps] = v[b, :, t]
    assert torch.equal(kp, kp0) and torch.equal(vp, vp0)


def test_paged_append_drops_negative_lengths():
    d, ps = 64, 64
    q, k = inputs.normal_bf16((2, 1, 3, d), 1, DEV), inputs.normal_bf16((2, 1, 3, d), 2, DEV)
    kp = torch.zeros(2, 1, ps, d, dtype=torch.bfloat16, device=DEV)
    vp, table = kp.clone(), torch.tensor([[0], [1]], dtype=torch.int32, device=DEV)
    plan = fattn.fa_rope_axes_plan(d, (32,))
    pos = torch.zeros(1, 2, 3, dtype=torch.int32, device=DEV)
    fattn.fa_rope_axes_paged(q, k, k, pos, plan, torch.empty_like(q), kp, vp, table,
                             torch.tensor([-2, -2 ** 31], dtype=torch.int32, device=DEV))
    assert torch.equal(kp[0, :, 0], k[0, :, 2]) and (kp[0, :, 1:] == 0).all() and (kp[1] == 0).all()
    assert torch.equal(vp, kp)
