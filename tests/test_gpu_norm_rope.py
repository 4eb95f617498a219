"""RMS norms of queries and keys with rotary positions on the GPU, forward, backward and paged, against the fp64 definition.

Forward.  The row's squares are added in fp32 (16 fused multiply-adds and up to 3 additions of positive terms, each within
2^-24), scaled and shifted (2^-23), and rsqrtf is within 2 ulps (2^-22): r is off by less than 10 2^-24 + 2^-24 +
2^-22 < 2^-20 of itself, and the two products with it and the weight by 2^-23 more.  The turn adds what
tests/test_gpu_rope_axes.py derives: (2^-21 + |pos| 2^-48) of |a| + |b|.  Together below (2^-19 + |pos| 2^-48) (|a| + |b|)
of the normed pair; then half a bf16 step.

Backward.  The incoming gradient turned back, g, is off by far = 2^-21 + |pos| 2^-48 of its pair's |a| + |b|; every
other factor is r (2^-20, up to three times in a product), a product or a sum over the row (19 additions): below rel =
2^-17 of the terms' absolute values.  The weights' gradients add R rows' terms in fp32: R 2^-24 of the absolute sum more."""

import numpy as np
import pytest
import torch

from _util import ensure_built
from exact_attention_06_gb300 import fattn, inputs
from oracle import cross as oc
from oracle import window as ow

pytestmark = pytest.mark.gpu
DEV = "cuda"
SECTIONS = {64: [(32,), (16, 16), (8, 12, 12), (1, 2, 3, 26)], 128: [(64,), (32, 32), (16, 24, 24), (5, 7, 11, 41)]}


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _pos(axes, B, N, seed, high=4096):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-high, high, (axes, B, N), generator=g, dtype=torch.int64).to(torch.int32)


def _weight(d, seed, dtype):
    return None if dtype is None else (1 + 0.3 * torch.randn(d, generator=torch.Generator().manual_seed(seed))).to(dtype).to(DEV)


def _far(pos):
    return float(np.abs(pos.numpy().astype(np.float64)).max()) * 2.0 ** -48


def _inside(x, ref, tol, what):
    x = x.detach().cpu().double().numpy()
    assert np.isfinite(x).all(), f"{what}: not finite"
    err = np.abs(x - ref)
    assert (err <= tol).all(), f"{what}: {float((err / np.maximum(tol, 1e-300)).max()):.2f} of the bound"


def _check(y, x, w, pos, axis, rates, inter, eps, what=""):
    ref, size = ow.norm_rope(x, w, pos, axis, rates, inter, eps)
    tol = np.abs(ref) * 2.0 ** -8 + size * (2.0 ** -19 + _far(pos)) * (1 + 2.0 ** -8) + 1e-38
    _inside(y, ref, tol, what)


def _check_bwd(dx, dw, x, w, dy, pos, axis, rates, inter, eps, what=""):
    rows = x.shape[0] * x.shape[1] * x.shape[2]
    rx, rw, ex, ew, abs_w = ow.norm_rope_backward(x, w, dy, pos, axis, rates, inter, eps, far=2.0 ** -21 + _far(pos),
                                                  rel=2.0 ** -17)
    _inside(dx, rx, np.abs(rx) * 2.0 ** -8 + ex * (1 + 2.0 ** -7) + 1e-38, what + " dx")
    if dw is not None:
        _inside(dw, rw, ew + rows * 2.0 ** -24 * abs_w + 2.0 ** -23 * np.abs(rw) + 1e-38, what + " dw")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n_axes", [1, 2, 3, 4])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("wtype", [None, torch.bfloat16, torch.float32])
def test_every_form_and_its_gradient(d, n_axes, inter, wtype):
    B, Hq, Hk, N, eps = 2, 5, 2, 37, 1e-5
    sections = SECTIONS[d][n_axes - 1]
    q, k = inputs.normal_bf16((B, Hq, N, d), 1, DEV) * 3, inputs.normal_bf16((B, Hk, N, d), 2, DEV)
    wq, wk = _weight(d, 3, wtype), _weight(d, 4, wtype)
    pos = _pos(n_axes, B, N, 3)
    plan = fattn.fa_rope_axes_plan(d, sections, 10000.0, inter)
    axis, rates = oc.rope_rates(d, sections, 10000.0)
    qo, ko = torch.full_like(q, float("nan")), torch.full_like(k, float("nan"))
    fattn.fa_norm_rope_axes(q, k, wq, wk, pos.to(DEV), plan, qo, ko, eps=eps)
    _check(qo, q, wq, pos, axis, rates, inter, eps, "q")
    _check(ko, k, wk, pos, axis, rates, inter, eps, "k")
    q2, k2 = q.clone(), k.clone()  # in place
    fattn.fa_norm_rope_axes(q2, k2, wq, wk, pos.to(DEV), plan, eps=eps)
    assert torch.equal(q2, qo) and torch.equal(k2, ko)
    gq, gk = inputs.normal_bf16((B, Hq, N, d), 4, DEV), inputs.normal_bf16((B, Hk, N, d), 5, DEV)
    dq, dk = torch.full_like(q, float("nan")), torch.full_like(k, float("nan"))
    dwq, dwk = (torch.full((d,), float("nan"), device=DEV) for _ in range(2))
    fattn.fa_norm_rope_axes_bwd(q, k, wq, wk, pos.to(DEV), plan, gq, gk, dq, dk, dwq, dwk, eps=eps)
    _check_bwd(dq, dwq, q, wq, gq, pos, axis, rates, inter, eps, "q")
    _check_bwd(dk, dwk, k, wk, gk, pos, axis, rates, inter, eps, "k")
    one = torch.full((d,), 7.0, device=DEV)  # only one weight's gradient, or none; in the gradients' place, or the inputs'
    g2, k2 = gq.clone(), k.clone()
    fattn.fa_norm_rope_axes_bwd(q, k2, wq, wk, pos.to(DEV), plan, g2, gk, None, k2, None, one, eps=eps)
    assert torch.equal(g2, dq) and torch.equal(k2, dk) and torch.equal(one, dwk)
    dq2 = torch.empty_like(q)
    fattn.fa_norm_rope_axes_bwd(q, None, wq, None, pos.to(DEV), plan, gq, None, dq2, eps=eps)
    assert torch.equal(dq2, dq)


SIZES = [(1, 1, 0, 1), (1, 1, 1, 1), (3, 4, 1, 2), (1, 9, 3, 31), (2, 33, 17, 65), (1, 3, 3, 1025), (5, 2, 0, 257),
         (1, 64, 8, 16), (2, 16, 4, 3001)]


@pytest.mark.parametrize("B,Hq,Hk,N", SIZES)
@pytest.mark.parametrize("d", [64, 128])
def test_sizes(B, Hq, Hk, N, d):
    """Sentinels around every written buffer; the gradients repeat bit for bit."""
    eps = 1e-6
    q = inputs.normal_bf16((B, Hq, N, d), 1, DEV)
    k = inputs.normal_bf16((B, Hk, N, d), 2, DEV) if Hk else None
    wq, wk = _weight(d, 3, torch.float32), _weight(d, 4, torch.float32)
    gq, gk = inputs.normal_bf16((B, Hq, N, d), 5, DEV), inputs.normal_bf16((B, Hk, N, d), 6, DEV) if Hk else None
    pos = _pos(3, B, N, 3)
    plan = fattn.fa_rope_axes_plan(d, SECTIONS[d][2], 500000.0)
    axis, rates = oc.rope_rates(d, SECTIONS[d][2], 500000.0)

    def guarded(n, dtype):
        t = torch.full((n + 512,), 7, dtype=dtype, device=DEV)
        return t, t[256:256 + n]
    ws = fattn.fa_norm_rope_axes_bwd_workspace_bytes(B, Hq, Hk, N, d)
    assert ws > 0
    want = None
    for _ in range(2):
        bufs = {"ws": guarded(ws, torch.uint8)}
        for x, t in (("q", q), ("k", k)):
            if t is not None:
                bufs["o" + x], bufs["d" + x] = guarded(t.numel(), torch.bfloat16), guarded(t.numel(), torch.bfloat16)
                bufs["w" + x] = guarded(d, torch.float32)
        at = lambda n, like: bufs[n][1].view(like.shape) if n in bufs else None  # noqa: E731
        fattn.fa_norm_rope_axes(q, k, wq, wk, pos.to(DEV), plan, at("oq", q), at("ok", k), eps=eps)
        fattn.fa_norm_rope_axes_bwd(q, k, wq, wk, pos.to(DEV), plan, gq, gk, at("dq", q), at("dk", k), bufs["wq"][1],
                                    bufs["wk"][1] if Hk else None, eps=eps, workspace=bufs["ws"][1])
        assert fattn.fa_get_status() == fattn.FA_OK
        for whole, part in bufs.values():
            assert (whole[:256] == 7).all() and (whole[256 + part.numel():] == 7).all()
        got = {n: b[1].clone() for n, b in bufs.items() if n != "ws"}
        want = want or got
        assert all(torch.equal(got[n], want[n]) for n in got)
    _check(at("oq", q), q, wq, pos, axis, rates, False, eps, "q")
    _check_bwd(at("dq", q), bufs["wq"][1], q, wq, gq, pos, axis, rates, False, eps, "q")
    if Hk:
        _check(at("ok", k), k, wk, pos, axis, rates, False, eps, "k")
        _check_bwd(at("dk", k), bufs["wk"][1], k, wk, gk, pos, axis, rates, False, eps, "k")
    with pytest.raises(fattn.FattnError) as e:
        fattn.fa_norm_rope_axes_bwd(q, k, wq, wk, pos.to(DEV), plan, gq, gk, at("dq", q), at("dk", k), bufs["wq"][1], None,
                                    workspace=bufs["ws"][1][:-1])
    assert e.value.status == fattn.FA_ERR_WORKSPACE


def test_small_and_large_rows():
    """eps decides where a row is all zeros or tiny; large rows keep their direction."""
    d, N = 128, 8
    x = inputs.normal_bf16((1, 1, N, d), 1, DEV)
    x[0, 0, 0], x[0, 0, 1], x[0, 0, 2], x[0, 0, 3] = 0, x[0, 0, 1] * 2.0 ** -60, x[0, 0, 2] * 2.0 ** 40, x[0, 0, 3] * 2.0 ** -14
    pos, w = _pos(1, 1, N, 3), _weight(d, 1, torch.float32)
    plan = fattn.fa_rope_axes_plan(d, (64,))
    axis, rates = oc.rope_rates(d, (64,))
    y = torch.empty_like(x)
    fattn.fa_norm_rope_axes(x, None, w, None, pos.to(DEV), plan, y)
    _check(y, x, w, pos, axis, rates, False, 1e-6)
    assert (y[0, 0, 0] == 0).all()
    g, dx, dw = inputs.normal_bf16(x.shape, 2, DEV), torch.empty_like(x), torch.empty(d, device=DEV)
    fattn.fa_norm_rope_axes_bwd(x, None, w, None, pos.to(DEV), plan, g, None, dx, None, dw)
    _check_bwd(dx, dw, x, w, g, pos, axis, rates, False, 1e-6)


def test_nan_and_infinities_stay_in_their_row():
    d, N = 64, 8
    x = inputs.normal_bf16((1, 2, N, d), 1, DEV)
    bad = x.clone()
    bad[0, 0, 3, 5], bad[0, 1, 4, 40] = float("inf"), float("nan")
    pos, plan = _pos(1, 1, N, 3).to(DEV), fattn.fa_rope_axes_plan(d, (32,))
    good, y = torch.empty_like(x), torch.empty_like(x)
    fattn.fa_norm_rope_axes(x, None, None, None, pos, plan, good)
    fattn.fa_norm_rope_axes(bad, None, None, None, pos, plan, y)
    same = (y == good).all(-1)
    same[0, 0, 3] = same[0, 1, 4] = True
    assert same.all() and torch.isnan(y[0, 1, 4]).all()


def test_an_offset_past_32_bits():
    B, H, N, d = 1, 33, 2 ** 19, 128
    q, g = (torch.zeros(B, H, N, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    q[:, -1, -5:], g[:, -1, -5:] = inputs.normal_bf16((5, d), 1, DEV), inputs.normal_bf16((5, d), 2, DEV)
    x, gx = q[:, -1:, -5:].cpu(), g[:, -1:, -5:].cpu()
    pos = torch.arange(N, dtype=torch.int32, device=DEV).view(1, 1, N)
    plan = fattn.fa_rope_axes_plan(d, (64,))
    axis, rates = oc.rope_rates(d, (64,))
    dx, dw = torch.empty_like(q), torch.empty(d, device=DEV)
    fattn.fa_norm_rope_axes_bwd(q, None, None, None, pos, plan, g, None, dx, None, dw)
    _check_bwd(dx[:, -1:, -5:], dw, x, None, gx, pos[:, :, -5:].cpu(), axis, rates, False, 1e-6)
    fattn.fa_norm_rope_axes(q, None, None, None, pos, plan)
    _check(q[:, -1:, -5:], x, None, pos[:, :, -5:].cpu(), axis, rates, False, 1e-6)


@pytest.mark.parametrize("d,ps,N,inter", [(64, 64, 1, False), (128, 64, 1, True), (128, 128, 70, False), (64, 192, 333, True)])
@pytest.mark.parametrize("ragged", [False, True])
def test_paged_append(d, ps, N, inter, ragged):
    B, Hq, Hk, P = 4, 6, 3, 40
    q = inputs.normal_bf16((B, Hq, N, d), 1, DEV)
    k, v = inputs.normal_bf16((B, Hk, N, d), 2, DEV), inputs.normal_bf16((B, Hk, N, d), 3, DEV)
    kp, vp = inputs.normal_bf16((P, Hk, ps, d), 4, DEV), inputs.normal_bf16((P, Hk, ps, d), 5, DEV)
    kp0, vp0 = kp.clone(), vp.clone()
    slots = torch.randperm(P * ps, generator=torch.Generator().manual_seed(6))[:B * N].view(B, N).contiguous()
    slots[1, 0], slots[2, -1], slots[3, 0] = -1, P * ps, 2 ** 62  # no places
    new = torch.tensor([N, max(N // 2, 1), N, 0], dtype=torch.int32) if ragged else None
    pos, wq, wk = _pos(2, B, N, 7), _weight(d, 1, torch.bfloat16), _weight(d, 2, torch.bfloat16)
    plan = fattn.fa_rope_axes_plan(d, SECTIONS[d][1], interleaved=inter)
    qo = torch.full_like(q, 9.0)
    fattn.fa_norm_rope_axes_paged(q, k, v, wq, wk, pos.to(DEV), plan, qo, kp, vp, slots.to(DEV), new.to(DEV) if ragged else None)
    want_q, want_k = torch.empty_like(q), torch.empty_like(k)
    fattn.fa_norm_rope_axes(q, k, wq, wk, pos.to(DEV), plan, want_q, want_k)  # (checked above)
    for b in range(B):
        n = int(new[b]) if ragged else N
        assert torch.equal(qo[b, :, :n], want_q[b, :, :n]) and (qo[b, :, n:] == 9).all()
        for t in range(n):
            s = int(slots[b, t])
            if 0 <= s < P * ps:
                kp0[s // ps, :, s % ps], vp0[s // ps, :, s % ps] = want_k[b, :, t], v[b, :, t]
    assert torch.equal(kp, kp0) and torch.equal(vp, vp0)


def test_paged_append_into_a_pool_past_32_bits():
    ps, d, Hk = 128, 128, 8
    P = 2 ** 31 // (ps * d * Hk) + 4
    kp, vp = (torch.zeros(P, Hk, ps, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    q, k, v = (inputs.normal_bf16((1, Hk, 3, d), s, DEV) for s in range(3))
    slots = torch.tensor([[(P - 1) * ps + 5, (P - 2) * ps, 7]], device=DEV)
    pos, plan = _pos(1, 1, 3, 1).to(DEV), fattn.fa_rope_axes_plan(d, (64,))
    qo, want = torch.empty_like(q), torch.empty_like(k)
    fattn.fa_norm_rope_axes_paged(q, k, v, None, None, pos, plan, qo, kp, vp, slots)
    fattn.fa_norm_rope_axes(k, None, None, None, pos, plan, want)
    for t, (page, row) in enumerate(((P - 1, 5), (P - 2, 0), (0, 7))):
        assert torch.equal(kp[page, :, row], want[0, :, t]) and torch.equal(vp[page, :, row], v[0, :, t])
    assert int((kp != 0).any(-1).sum()) == 3 * Hk


def test_gradients_match_differences():
    """<y(x + s) - y(x - s), g> along each gradient's own signs, against fp64 differences at the same points."""
    d, eps = 64, 1e-3
    x, g = inputs.normal_bf16((2, 3, 40, d), 1, DEV), inputs.normal_bf16((2, 3, 40, d), 2, DEV)
    w = _weight(d, 3, torch.float32)
    pos, plan = _pos(2, 2, 40, 4), fattn.fa_rope_axes_plan(d, SECTIONS[d][1])
    axis, rates = oc.rope_rates(d, SECTIONS[d][1])
    dx, dw = torch.empty_like(x), torch.empty(d, device=DEV)
    fattn.fa_norm_rope_axes_bwd(x, None, w, None, pos.to(DEV), plan, g, None, dx, None, dw, eps=eps)
    gn = g.cpu().double().numpy()
    for name in ("x", "w"):
        sides, slack, exact, at = [], 0.0, [], []
        for s in (1, -1):
            xx = (x.float() + s * torch.sign(dx.float()) * 2.0 ** -4).to(torch.bfloat16) if name == "x" else x
            ww = w + s * torch.sign(dw) * 2.0 ** -4 if name == "w" else w
            y = torch.empty_like(x)
            fattn.fa_norm_rope_axes(xx, None, ww, None, pos.to(DEV), plan, y, eps=eps)
            ref, size = ow.norm_rope(xx, ww, pos, axis, rates, False, eps)
            sides.append(float((y.cpu().double().numpy() * gn).sum()))
            exact.append(float((ref * gn).sum()))
            slack += float((np.abs(gn) * (np.abs(ref) * 2.0 ** -8 + size * 2.0 ** -18)).sum())
            at.append((xx if name == "x" else ww).double())
        moved, grad = at[0] - at[1], (dx if name == "x" else dw).double()
        rx, rw, ex, ew, _ = ow.norm_rope_backward(x, w, g, pos, axis, rates, False, eps, far=2.0 ** -20, rel=2.0 ** -17)
        ref = torch.from_numpy(rx if name == "x" else rw).to(DEV)
        curve = abs((exact[0] - exact[1]) - float((ref * moved).sum()))
        own = float(((grad.abs() * 2.0 ** -8 + torch.from_numpy(ex if name == "x" else ew).to(DEV)) * moved.abs()).sum())
        assert abs((sides[0] - sides[1]) - float((grad * moved).sum())) <= slack + curve + own, name
