"""Sliding-window attention with sinks on the GPU, forward and backward, against the fp64 definition.

The bounds are those of tests/test_gpu_cross.py, whose products, exponents and roundings these kernels share: u = 2^-8
is bf16's half step, eps = d 2^-24 big + 2^-18 the relative error of exp(s - m), |O - O_ref| <= (u + 2 eps +
2 Nk 2^-24) sum p |v| and u |O| more for a bf16 output, lse within eps + Nk 2^-24 and 2^-22 of its value, gradients
within window_backward's bounds with rel = u + 4 eps + 2^-10."""

import math

import numpy as np
import pytest
import torch

from _util import ensure_built
from exact_attention_06_gb300 import fattn, inputs
from oracle import window as ow

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _inputs(B, Hq, Hkv, N, Nk, d, W=None, S=0, seed=0):
    """Inputs; what keys hold that no query sees may be anything."""
    q = inputs.normal_bf16((B, Hq, N, d), seed, DEV)
    k, v = inputs.normal_bf16((B, Hkv, Nk, d), seed + 1, DEV), inputs.normal_bf16((B, Hkv, Nk, d), seed + 2, DEV)
    do = inputs.normal_bf16((B, Hq, N, d), seed + 3, DEV)
    hidden = slice(S, max(S, Nk - N - (Nk if W is None else W) + 1))
    k[:, :, hidden][:, :, ::2], v[:, :, hidden][:, :, ::2] = float("nan"), float("inf")
    k[:, :, hidden][:, :, 1::2], v[:, :, hidden][:, :, 1::2] = float("-inf"), float("nan")
    return q, k, v, do


def _fwd(q, k, v, scale, W, S, o_fp32=False, **kw):
    o = torch.full(q.shape, float("nan"), dtype=torch.float32 if o_fp32 else torch.bfloat16, device=DEV)
    lse = torch.full(q.shape[:3], float("nan"), device=DEV)
    fattn.fa_window_fwd(q, k, v, o, lse, scale, W, S, **kw)
    assert fattn.fa_get_status() == fattn.FA_OK
    return o, lse


def _bounds(q, k, v, scale, W, S):
    Nk, d = k.shape[2], q.shape[3]
    ref, lse, pv, big = ow.window_attention(q, k, v, scale, W, S)
    eps = d * 2.0 ** -24 * big + 2.0 ** -18
    return ref, lse, (U + 2 * eps + 2 * Nk * 2.0 ** -24) * pv, eps + Nk * 2.0 ** -24, eps


def _inside(x, ref, tol, what):
    x = x.detach().cpu().double().numpy()
    assert np.isfinite(x).all(), f"{what}: not finite"
    err = np.abs(x - ref)
    at = np.unravel_index(np.argmax(err - tol), err.shape)
    assert (err <= tol).all(), f"{what}: off by {err[at]:.3e}, bound {tol[at]:.3e} at {at}"


def _check_fwd(o, lse, q, k, v, scale, W, S, what="", bounds=None):
    ref, lref, tol, ltol, _ = bounds or _bounds(q, k, v, scale, W, S)
    if o.dtype == torch.bfloat16:
        tol = tol + U * (np.abs(ref) + tol)
    _inside(o, ref, tol + 1e-30, what + " o")
    _inside(lse, lref, ltol + 2.0 ** -22 * np.abs(lref), what + " lse")


def _check_bwd(q, k, v, do, W, S, types=(torch.float32, torch.bfloat16)):
    scale = q.shape[3] ** -0.5
    o, lse = _fwd(q, k, v, scale, W, S)
    bounds = _bounds(q, k, v, scale, W, S)
    _check_fwd(o, lse, q, k, v, scale, W, S, bounds=bounds)
    ref, _, otol, _, eps = bounds
    # (rows of at most 32 keys have rowsum(O dO) from P and dP: the rounding of O is not in it)
    few = min(W + S, k.shape[2]) <= 32
    want, bound = ow.window_backward(q, k, v, do, scale, W, S, rel=U + 4 * eps + 2.0 ** -10,
                                     o_err=None if few else otol + U * (np.abs(ref) + otol))
    for t in types:
        got = {n: torch.full(x.shape, float("nan"), dtype=t, device=DEV) for n, x in (("dq", q), ("dk", k), ("dv", v))}
        fattn.fa_window_bwd(q, k, v, o, do, lse, *got.values(), scale, W, S)
        assert fattn.fa_get_status() == fattn.FA_OK
        for n, g in got.items():
            tol = bound[n] * (1 + 2.0 ** -6) + 1e-30
            _inside(g, want[n], tol + (U * (np.abs(want[n]) + tol) if t == torch.bfloat16 else 0), f"{n} {t}")
        hidden = slice(S, max(S, k.shape[2] - q.shape[2] - W + 1))  # keys that no query sees: zeros, whatever they hold
        assert (got["dk"][:, :, hidden] == 0).all() and (got["dv"][:, :, hidden] == 0).all()


CASES = [  # B, Hq, Hkv, N, Nk, window, sinks
    (1, 1, 1, 1, 1, 1, 0), (1, 2, 1, 1, 5, 1, 3), (2, 2, 1, 2, 2, 1, 0), (1, 2, 2, 127, 127, 64, 0),
    (1, 2, 1, 128, 128, 128, 4), (2, 3, 3, 129, 129, 127, 1), (1, 4, 2, 256, 256, 129, 128), (1, 2, 2, 257, 300, 1, 0),
    (1, 2, 2, 300, 300, 1, 100), (2, 4, 1, 385, 640, 128, 16), (1, 8, 2, 513, 513, 200, 0), (1, 5, 5, 333, 1000, 333, 5),
    (1, 6, 2, 700, 700, 5000, 7), (2, 2, 2, 1, 700, 100, 3), (1, 16, 1, 77, 1500, 256, 128), (1, 2, 1, 1000, 1000, 257, 65),
    (1, 1, 1, 2000, 2000, 600, 64), (1, 2, 2, 640, 640, 639, 2), (1, 2, 2, 640, 640, 640, 2), (1, 2, 2, 640, 640, 641, 2),
    (1, 2, 1, 400, 450, 2 ** 31 - 1, 128), (3, 1, 1, 130, 131, 2, 1), (1, 2, 2, 600, 600, 3, 63), (1, 3, 1, 70, 4000, 900, 50),
    (1, 2, 1, 260, 388, 129, 128), (1, 1, 1, 900, 900, 255, 128), (1, 2, 1, 512, 513, 256, 0),
    (2, 4, 2, 333, 333, 7, 9), (1, 2, 1, 700, 720, 16, 16), (1, 3, 3, 31, 31, 40, 0), (2, 2, 1, 500, 900, 8, 24),
    (1, 2, 1, 3000, 3000, 40, 9),
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Hq,Hkv,N,Nk,W,S", CASES)
def test_forward(B, Hq, Hkv, N, Nk, W, S, d):
    q, k, v, _ = _inputs(B, Hq, Hkv, N, Nk, d, W, S)
    for o_fp32 in (False, True):
        o, lse = _fwd(q, k, v, d ** -0.5, W, S, o_fp32)
        _check_fwd(o, lse, q, k, v, d ** -0.5, W, S, f"fp32={o_fp32}")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Hq,Hkv,N,Nk,W,S", CASES)
def test_backward(B, Hq, Hkv, N, Nk, W, S, d):
    _check_bwd(*_inputs(B, Hq, Hkv, N, Nk, d, W, S), W, S)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Hq,Hkv,N,Nk,W,S", [(8, 40, 40, 300, 300, 100, 3), (6, 64, 16, 260, 330, 33, 0),
                                               (7, 32, 32, 650, 650, 65, 17), (5, 48, 24, 900, 900, 300, 128)])
def test_more_blocks_than_multiprocessors(B, Hq, Hkv, N, Nk, W, S, d):
    """No key tile's list is cut but the sinks', and a block of the dQ kernel takes several query tiles."""
    _check_bwd(*_inputs(B, Hq, Hkv, N, Nk, d, W, S), W, S, types=(torch.bfloat16,))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Hq,Hkv,N,Nk,W,S", [(2, 32, 32, 300, 300, 30, 17), (2, 32, 16, 300, 300, 65, 0),
                                               (2, 40, 40, 200, 277, 65, 17), (2, 96, 48, 200, 277, 30, 3)])
def test_blocks_of_several_items(B, Hq, Hkv, N, Nk, W, S, d):
    """Of one head (the first two), or of all heads' list, so that a block's items are of two heads (the others)."""
    _check_bwd(*_inputs(B, Hq, Hkv, N, Nk, d, W, S), W, S)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [2, 3, 5, 7, 8, 12, 16, 31, 32, 40, 64, 100, 128, 130])
def test_heads_that_share_a_key_head(G, d):
    """The heads of a tile's rows, rows that no head takes, tiles of one position."""
    for B, Hkv, N, Nk, W, S in ((1, 2, 97, 140, 45, 3), (2, 1, 3, 200, 130, 70), (1, 1, 200, 200, 3, 0)):
        _check_bwd(*_inputs(B, Hkv * G, Hkv, N, Nk, d, W, S), W, S, types=(torch.bfloat16,))
    q, k, v, _ = _inputs(1, G, 1, 133, 300, d, 129, 17)
    o, lse = _fwd(q, k, v, 0.1, 129, 17, True)
    _check_fwd(o, lse, q, k, v, 0.1, 129, 17)


@pytest.mark.parametrize("d", [64, 128])
def test_a_window_of_everything_is_causal_attention(d):
    B, H, N = 2, 3, 700
    q, k, v, do = _inputs(B, H, H, N, N, d)
    scale = d ** -0.5
    for W, S in ((N, 0), (2 ** 31 - 1, 9), (N - 100, 128)):  # (the last: sinks cover what the window leaves out)
        o, lse = _fwd(q, k, v, scale, W, S, True)
        ref, lref, tol, ltol, _ = _bounds(q, k, v, scale, N, 0)
        _inside(o, ref, tol + 1e-30, "o")
        _inside(lse, lref, ltol + 2.0 ** -22 * np.abs(lref), "lse")
    want, wl = torch.empty_like(q), torch.empty(B, H, N, device=DEV)
    fattn.fa_fwd(q, k, v, want, wl, scale, True)
    o, lse = _fwd(q, k, v, scale, N, 0)
    assert (lse - wl).abs().max() < 1e-4 and (o.float() - want.float()).abs().max() < 2 * U * want.float().abs().max()


def test_a_peaked_softmax():
    """Keys x8 (scores far apart): the running maximum moves, most probabilities vanish."""
    q, k, v, _ = _inputs(1, 2, 2, 900, 900, 128)
    inputs.spike_every_64th_key(k)
    for W, S in ((300, 0), (300, 70), (64, 1)):
        o, lse = _fwd(q, k, v, 128 ** -0.5, W, S, True)
        _check_fwd(o, lse, q, k, v, 128 ** -0.5, W, S, f"{W} {S}")


@pytest.mark.parametrize("d", [64, 128])
def test_gradients_match_differences(d):
    """Along each gradient's own signs, with the forward's bound on each side and the curvature by fp64 differences at the
    same points."""
    W, S = 70, 5
    q, k, v, do = _inputs(1, 4, 2, 200, 230, d, W, S)
    k, v = torch.nan_to_num(k, 0, 0, 0), torch.nan_to_num(v, 0, 0, 0)
    scale = d ** -0.5
    o, lse = _fwd(q, k, v, scale, W, S)
    g = {n: torch.empty(x.shape, device=DEV) for n, x in (("dq", q), ("dk", k), ("dv", v))}
    fattn.fa_window_bwd(q, k, v, o, do, lse, *g.values(), scale, W, S)
    w = do.cpu().double().numpy()
    for i, n in enumerate(("dq", "dk", "dv")):
        step = torch.sign(g[n]) * 2.0 ** -3
        sides, slack, exact = [], 0.0, []
        for s in (1, -1):
            x = [q, k, v]
            x[i] = (x[i].float() + s * step).to(torch.bfloat16)
            oo, _ = _fwd(*x, scale, W, S, o_fp32=True)
            sides.append((float((oo.double().cpu().numpy() * w).sum()), x[i].double()))
            ref, _, tol, _, _ = _bounds(*x, scale, W, S)
            slack += float((np.abs(w) * tol).sum())
            exact.append(float((ref * w).sum()))
        moved = sides[0][1] - sides[1][1]  # (what the bf16 inputs really moved by)
        along = float((g[n].double() * moved).sum())
        curve = abs((exact[0] - exact[1]) - float((torch.from_numpy(
            ow.window_backward(q, k, v, do, scale, W, S)[0][n]).to(DEV) * moved).sum()))
        got = sides[0][0] - sides[1][0]
        assert abs(got - along) <= slack + curve + 2 * U * float((g[n].double() * moved).abs().sum()), n


@pytest.mark.parametrize("d", [64, 128])
def test_repeats_bitwise_on_any_stream(d):
    q, k, v, do = _inputs(2, 8, 2, 700, 800, d, 200, 9)
    want = None
    for s in (None, torch.cuda.Stream(), torch.cuda.current_stream().cuda_stream):
        torch.cuda.synchronize()
        out = [torch.empty_like(q), torch.empty(q.shape[:3], device=DEV), *(torch.empty_like(x) for x in (q, k, v))]
        fattn.fa_window_fwd(q, k, v, *out[:2], 0.1, 200, 9, stream=s)
        fattn.fa_window_bwd(q, k, v, out[0], do, out[1], *out[2:], 0.1, 200, 9, stream=s)
        torch.cuda.synchronize()
        assert fattn.fa_get_status() == fattn.FA_OK
        want = want or out
        assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Hq,Hkv,N,Nk,W,S", [(2, 6, 2, 333, 400, 90, 16), (1, 2, 2, 1500, 1500, 300, 1),
                                               (1, 4, 4, 100, 100, 7, 0)])
def test_outputs_and_workspaces_keep_their_bounds(B, Hq, Hkv, N, Nk, W, S, d):
    """Sentinels around every written buffer, workspaces of exactly the stated size."""
    q, k, v, do = _inputs(B, Hq, Hkv, N, Nk, d, W, S)

    def guarded(shape, dtype):
        n = math.prod(shape)
        t = torch.full((n + 512,), 7 if dtype == torch.uint8 else 7.0, dtype=dtype, device=DEV)
        return t, t[256:256 + n].view(shape)
    ws_bytes = fattn.fa_window_bwd_workspace_bytes(B, Hq, Hkv, N, Nk, d, W, S)
    for t in (torch.bfloat16, torch.float32):
        bufs = [guarded(s, x) for s, x in ((q.shape, torch.bfloat16), (q.shape[:3], torch.float32), ((ws_bytes,), torch.uint8),
                                           (q.shape, t), (k.shape, t), (k.shape, t))]
        o, lse, ws, dq, dk, dv = (b[1] for b in bufs)
        fattn.fa_window_fwd(q, k, v, o, lse, 0.1, W, S)
        fattn.fa_window_bwd(q, k, v, o, do, lse, dq, dk, dv, 0.1, W, S, workspace=ws)
        assert fattn.fa_get_status() == fattn.FA_OK
        for whole, part in bufs:
            assert (whole[:256] == 7).all() and (whole[256 + part.numel():] == 7).all()
        _check_fwd(o, lse, q, k, v, 0.1, W, S)
    with pytest.raises(fattn.FattnError) as e:
        fattn.fa_window_bwd(q, k, v, o, do, lse, dq, dk, dv, 0.1, W, S, workspace=ws[:-1])
    assert e.value.status == fattn.FA_ERR_WORKSPACE


@pytest.mark.parametrize("d", [64, 128])
def test_a_wait_that_runs_out_is_reported(d):
    W, S = 300, 20
    q, k, v, do = _inputs(2, 4, 2, 1000, 1000, d, W, S)
    o, lse = torch.empty_like(q), torch.empty(2, 4, 1000, device=DEV)
    for _ in range(2):
        fattn.fa_window_fwd(q, k, v, o, lse, 0.1, W, S, wait_budget_cycles=1)
        with pytest.raises(fattn.FattnError) as e:
            fattn.fa_get_status()
        assert e.value.status == fattn.FA_ERR_TIMEOUT and fattn.fa_get_status() == fattn.FA_OK
        o, lse = _fwd(q, k, v, 0.1, W, S)
        _check_fwd(o, lse, q, k, v, 0.1, W, S, "after a timeout")
        g = [torch.zeros_like(x) for x in (q, k, v)]
        fattn.fa_window_bwd(q, k, v, o, do, lse, *g, 0.1, W, S, wait_budget_cycles=1)
        with pytest.raises(fattn.FattnError) as e:
            fattn.fa_get_status()
        assert e.value.status == fattn.FA_ERR_TIMEOUT and fattn.fa_get_status() == fattn.FA_OK


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("S", [0, 3])
def test_outputs_aligned_to_16_bytes_only(S, d):
    """The same values as in outputs of torch's own alignment, and nothing before or behind them."""
    q, k, v, do = _inputs(2, 6, 2, 333, 333, d, 70, S)

    def step(shift):
        def out(x):
            buf = torch.full((x.numel() + 64,), 7.0, dtype=torch.bfloat16, device=DEV)
            return buf, buf[shift:shift + x.numel()].view(x.shape)
        bufs, outs = zip(*(out(x) for x in (q, q, k, v)))
        lse = torch.empty(q.shape[:3], device=DEV)
        fattn.fa_window_fwd(q, k, v, outs[0], lse, 0.1, 70, S)
        fattn.fa_window_bwd(q, k, v, outs[0], do, lse, *outs[1:], 0.1, 70, S)
        assert fattn.fa_get_status() == fattn.FA_OK
        for b, o in zip(bufs, outs):
            assert (b[:shift] == 7).all() and (b[shift + o.numel():] == 7).all()
        return outs
    assert all(torch.equal(x, y) for x, y in zip(step(0), step(8)))


def test_offsets_past_32_bits():
    """The last head lies behind 2^31 elements: what a call of its own gives."""
    B, Hq, Hkv, N, d, W, S = 1, 66, 66, 2 ** 18, 128, 130, 3
    q, k, v, do = (torch.zeros(B, H, N, d, dtype=torch.bfloat16, device=DEV) for H in (Hq, Hkv, Hkv, Hq))
    last = [inputs.normal_bf16((1, 1, N, d), s, DEV) for s in range(4)]
    for x, y in zip((q, k, v, do), last):
        x[:, -1:] = y

    def step(q, k, v, do):
        o, lse = torch.empty_like(q), torch.empty(q.shape[:3], device=DEV)
        fattn.fa_window_fwd(q, k, v, o, lse, 0.1, W, S)
        g = [torch.empty_like(x) for x in (q, k, v)]
        fattn.fa_window_bwd(q, k, v, o, do, lse, *g, 0.1, W, S)
        assert fattn.fa_get_status() == fattn.FA_OK
        return o, lse, *g
    got, want = step(q, k, v, do), step(*last)
    # the same ranges of queries for the sinks' tile (their length is the window's), so the same sums
    assert all(torch.equal(x[:, -1:], y) for x, y in zip(got, want))


@pytest.mark.parametrize("d", [64, 128])
def test_more_tiles_than_a_grid_has_rows(d):
    """65600 tiles of one head; its ends against the definition on the tokens that reach them."""
    N, W, T = 65600 * 128 + 77, 100, 500
    q, k, v, do = (inputs.normal_bf16((1, 1, N, d), s, DEV) for s in range(4))
    scale = d ** -0.5
    o, lse = _fwd(q, k, v, scale, W, 0)
    got = [torch.full_like(x, float("nan")) for x in (q, k, v)]
    fattn.fa_window_bwd(q, k, v, o, do, lse, *got, scale, W, 0)
    assert fattn.fa_get_status() == fattn.FA_OK
    for rows, keys, dk_from, dk_to in ((slice(N - T, N), slice(N - T - W, N), W, T + W), (slice(0, T), slice(0, T), 0, T - W)):
        qs, dos = q[:, :, rows], do[:, :, rows]
        ks, vs = k[:, :, keys], v[:, :, keys]
        bounds = _bounds(qs, ks, vs, scale, W, 0)
        _check_fwd(o[:, :, rows], lse[:, :, rows], qs, ks, vs, scale, W, 0, bounds=bounds)
        ref, _, otol, _, eps = bounds
        want, bound = ow.window_backward(qs, ks, vs, dos, scale, W, 0, rel=U + 4 * eps + 2.0 ** -10,
                                         o_err=otol + U * (np.abs(ref) + otol))
        for n, g in zip(("dq", "dk", "dv"), got):
            part = slice(0, T) if n == "dq" else slice(dk_from, dk_to)  # (the keys all of whose queries are here)
            tol = bound[n] * (1 + 2.0 ** -6) + 1e-30
            tol = tol + U * (np.abs(want[n]) + tol)
            _inside(g[:, :, rows if n == "dq" else keys][:, :, part], want[n][:, :, part], tol[:, :, part], n)
