"""Cross attention on the GPU, forward and backward, against the fp64 definition.

The bounds count what the kernels round.  u = 2^-8 is bf16's half step.
* Scores: products of bf16 are exact in fp32, their sum of d terms is off by at most d 2^-24 of the sum
  of their absolute values, which is at most ``big``; the exponent's fused multiply-add and ex2.approx
  add < 2^-18 for |scores| < 64.  eps = d 2^-24 big + 2^-18 bounds the relative error of exp(s - m).
* O = sum p v / sum p: p rounded to bf16 in the numerator (u), both sums off by eps and by fp32
  sums of up to Nk terms (Nk 2^-24): |O - O_ref| <= (u + 2 eps + 2 Nk 2^-24) sum p |v|, and u |O| more
  for a bf16 output.
* lse: eps + Nk 2^-24 absolutely, 2^-22 of its value.
* Gradients: P and dS rounded to bf16 (u each); P off by 2 eps more, dP and D by 2^-24 d of their terms'
  absolute sums, O by the bound above: the bounds cross_backward computes with rel = u + 4 eps + 2^-10
  (the 2^-10 for the fp32 accumulations of up to 2^14 terms), and u of the value for bf16 gradients."""

import ctypes
import math

import numpy as np
import pytest
import torch

from _util import ensure_built
from exact_attention_06_gb300 import fattn, inputs
from oracle import cross as oc

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _inputs(B, Hq, Hkv, Nq, Nk, d, lens, seed=0, junk=True):
    q = inputs.normal_bf16((B, Hq, Nq, d), seed, DEV)
    k, v = inputs.normal_bf16((B, Hkv, Nk, d), seed + 1, DEV), inputs.normal_bf16((B, Hkv, Nk, d), seed + 2, DEV)
    do = inputs.normal_bf16((B, Hq, Nq, d), seed + 3, DEV)
    if lens is not None and junk:  # what padding may hold
        for b, n in enumerate(lens):
            n = min(max(n, 0), Nk)
            k[b, :, n::3], v[b, :, n::3] = float("nan"), float("inf")
            k[b, :, n + 1::3], v[b, :, n + 1::3] = float("-inf"), float("nan")
    return q, k, v, do, None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV)


def _fwd(q, k, v, kl, scale, o_fp32=False, cut=True, **kw):
    o = torch.full(q.shape, float("nan"), dtype=torch.float32 if o_fp32 else torch.bfloat16, device=DEV)
    lse = torch.full(q.shape[:3], float("nan"), device=DEV)
    if cut:
        fattn.fa_cross_fwd(q, k, v, o, lse, scale, kv_lens=kl, **kw)
    else:  # a NULL workspace: one kernel
        B, Hq, Nq, d = q.shape
        opts = fattn.FaCrossOpts(int(o_fp32), 0)
        p = lambda t: ctypes.c_void_p(0 if t is None else t.data_ptr())  # noqa: E731
        st = fattn.lib().fa_cross_fwd(p(q), p(k), p(v), p(kl), p(o), p(lse), B, Hq, k.shape[1], Nq, k.shape[2], d,
                                      ctypes.c_float(scale), p(None), 0,
                                      ctypes.c_void_p(torch.cuda.current_stream().cuda_stream), ctypes.byref(opts))
        assert st == fattn.FA_OK, fattn.fa_last_error()
    assert fattn.fa_get_status() == fattn.FA_OK
    return o, lse


def _bounds(q, k, v, scale, lens):
    Nk, d = k.shape[2], q.shape[3]
    ref, lse, pv, big = oc.cross_attention(q, k, v, scale, lens)
    eps = d * 2.0 ** -24 * big + 2.0 ** -18
    return ref, lse, (U + 2 * eps + 2 * Nk * 2.0 ** -24) * pv, eps + Nk * 2.0 ** -24, eps


def _inside(x, ref, tol, what):
    x = x.detach().cpu().double().numpy()
    assert np.isfinite(x).all(), f"{what}: not finite"
    err = np.abs(x - ref)
    at = np.unravel_index(np.argmax(err - tol), err.shape)
    assert (err <= tol).all(), f"{what}: off by {err[at]:.3e}, bound {tol[at]:.3e} at {at}"


def _check_fwd(o, lse, q, k, v, scale, lens, what=""):
    ref, lref, tol, ltol, _ = _bounds(q, k, v, scale, lens)
    if o.dtype == torch.bfloat16:
        tol = tol + U * (np.abs(ref) + tol)
    _inside(o, ref, tol + 1e-30, what + " o")
    got = lse.cpu().double().numpy()
    empty = np.isneginf(lref)
    assert np.isneginf(got[empty]).all() and (o.cpu().double().numpy()[empty] == 0).all(), what + ": empty rows"
    err = np.abs(got[~empty] - lref[~empty])
    assert (err <= ltol + 2.0 ** -22 * np.abs(lref[~empty])).all(), f"{what} lse: {err.max() if err.size else 0:.3e}"


CASES = [  # B, Hq, Hkv, Nq, Nk, lens
    (1, 1, 1, 1, 1, None), (2, 2, 1, 1, 2, [1, 2]), (1, 1, 1, 127, 63, None), (2, 3, 3, 128, 127, None),
    (1, 2, 2, 129, 128, None), (3, 4, 2, 1, 129, [129, 0, 128]), (2, 8, 1, 16, 257, [256, 255]),
    (1, 6, 2, 85, 300, None), (4, 4, 4, 33, 640, [640, 1, 0, 513]), (2, 5, 5, 300, 1000, [1000, 999]),
    (1, 8, 8, 1, 4099, None), (3, 12, 4, 43, 641, [641, 428, 0]), (1, 1, 1, 1000, 5, None),
    (2, 2, 2, 257, 129, [-5, 400]), (1, 32, 8, 1, 2000, [1999]),
    # at most 32 rows a key head (the few-row kernel): one and two row blocks, clusters and partials
    (1, 1, 1, 32, 5000, None), (2, 32, 1, 1, 700, [700, 333]), (1, 24, 2, 2, 3000, [2500]), (1, 17, 1, 1, 64, None),
    (3, 16, 1, 1, 70, [70, 0, 64]), (4, 2, 2, 8, 65, [65, 63, 17, 1]), (1, 33, 1, 1, 1025, None),
    (2, 1, 1, 1, 20000, [19999, 0]),
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Hq,Hkv,Nq,Nk,lens", CASES)
def test_forward(B, Hq, Hkv, Nq, Nk, lens, d):
    q, k, v, _, kl = _inputs(B, Hq, Hkv, Nq, Nk, d, lens)
    scale = d ** -0.5
    for o_fp32 in (False, True):
        for cut in (False, True):
            o, lse = _fwd(q, k, v, kl, scale, o_fp32, cut)
            _check_fwd(o, lse, q, k, v, scale, lens, f"fp32={o_fp32} cut={cut}")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Hq,Hkv,Nq,Nk,lens", CASES)
def test_backward(B, Hq, Hkv, Nq, Nk, lens, d):
    q, k, v, do, kl = _inputs(B, Hq, Hkv, Nq, Nk, d, lens)
    scale = d ** -0.5
    o, lse = _fwd(q, k, v, kl, scale)
    ref, _, otol, _, eps = _bounds(q, k, v, scale, lens)
    want, bound = oc.cross_backward(q, k, v, do, scale, lens, rel=U + 4 * eps + 2.0 ** -10,
                                    o_err=otol + U * (np.abs(ref) + otol))
    for t in (torch.float32, torch.bfloat16):
        got = {n: torch.full(x.shape, float("nan"), dtype=t, device=DEV) for n, x in (("dq", q), ("dk", k), ("dv", v))}
        fattn.fa_cross_bwd(q, k, v, o, do, lse, *got.values(), scale, kv_lens=kl)
        assert fattn.fa_get_status() == fattn.FA_OK
        for n, g in got.items():
            tol = bound[n] * (1 + 2.0 ** -6) + 1e-30
            _inside(g, want[n], tol + (U * (np.abs(want[n]) + tol) if t == torch.bfloat16 else 0), f"{n} {t}")
        for b, n in enumerate(lens or []):  # padded keys: zeros, whatever they held
            n = min(max(n, 0), Nk)
            assert (got["dk"][b, :, n:] == 0).all() and (got["dv"][b, :, n:] == 0).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Hq,Hkv,Nq,Nk", [(64, 8, 8, 40, 100), (100, 6, 3, 70, 130), (30, 8, 8, 300, 257),
                                             (4, 16, 8, 1500, 77), (3, 8, 8, 3333, 64), (3, 4, 4, 7000, 1)])
def test_many_blocks_of_few_keys(B, Hq, Hkv, Nq, Nk, d):
    """More blocks than SMs, each with a tile or two of keys and padding (or nothing) behind them."""
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(-1, Nk + 2, (B,), generator=g).tolist()
    q, k, v, do, kl = _inputs(B, Hq, Hkv, Nq, Nk, d, lens)
    scale = d ** -0.5
    o, lse = _fwd(q, k, v, kl, scale)
    _check_fwd(o, lse, q, k, v, scale, lens)
    ref, _, otol, _, eps = _bounds(q, k, v, scale, lens)
    want, bound = oc.cross_backward(q, k, v, do, scale, lens, rel=U + 4 * eps + 2.0 ** -10,
                                    o_err=otol + U * (np.abs(ref) + otol))
    got = {n: torch.full(x.shape, float("nan"), device=DEV) for n, x in (("dq", q), ("dk", k), ("dv", v))}
    fattn.fa_cross_bwd(q, k, v, o, do, lse, *got.values(), scale, kv_lens=kl)
    assert fattn.fa_get_status() == fattn.FA_OK
    for n, x in got.items():
        _inside(x, want[n], bound[n] * (1 + 2.0 ** -6) + 1e-30, n)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nk,lens", [(64, None), (65, [65, 64]), (96, None), (97, [97, 96]), (128, [128, 33]),
                                     (77, [0, 77])])
def test_blocks_that_stream_many_query_tiles(Nk, lens, d):
    """The edges of the key tiles (64, 96, 128), with more query tiles in a block than its ring holds."""
    q, k, v, _, kl = _inputs(2, 8, 4, 9000, Nk, d, lens)
    for o_fp32 in (False, True):
        o, lse = _fwd(q, k, v, kl, d ** -0.5, o_fp32)
        _check_fwd(o, lse, q, k, v, d ** -0.5, lens, f"fp32={o_fp32}")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nk,lens", [(1, None), (64, [64, 0]), (65, [65, 64]), (96, None), (97, [97, 96]),
                                     (128, [128, 33]), (77, [0, 77]), (31, [32, 5]),
                                     # more than one key tile: the dQ kernel's blocks take several query tiles
                                     (129, None), (130, [130, 1]), (200, [65, 129]), (256, [256, 64]), (300, [193, 0]),
                                     (600, [599, 300])])
def test_gradients_of_many_query_tiles_over_few_keys(Nk, lens, d):
    B, Hq, Hkv, Nq = 2, 8, 4, 7001  # some twenty query tiles a block, or ranges of them
    q, k, v, do, kl = _inputs(B, Hq, Hkv, Nq, Nk, d, lens)
    scale = d ** -0.5
    o, lse = _fwd(q, k, v, kl, scale)
    ref, _, otol, _, eps = _bounds(q, k, v, scale, lens)
    want, bound = oc.cross_backward(q, k, v, do, scale, lens, rel=U + 4 * eps + 2.0 ** -10,
                                    o_err=otol + U * (np.abs(ref) + otol))
    for t in (torch.float32, torch.bfloat16):
        got = {n: torch.full(x.shape, float("nan"), dtype=t, device=DEV) for n, x in (("dq", q), ("dk", k), ("dv", v))}
        fattn.fa_cross_bwd(q, k, v, o, do, lse, *got.values(), scale, kv_lens=kl)
        assert fattn.fa_get_status() == fattn.FA_OK
        for n, g in got.items():
            tol = bound[n] * (1 + 2.0 ** -6) + 1e-30
            _inside(g, want[n], tol + (U * (np.abs(want[n]) + tol) if t == torch.bfloat16 else 0), f"{n} {t}")


def test_a_peaked_softmax():
    """Keys x8 (scores far apart): the running maximum moves, most probabilities vanish."""
    B, H, Nq, Nk, d, lens = 1, 2, 200, 700, 128, [650]
    q, k, v, _, kl = _inputs(B, H, H, Nq, Nk, d, lens, junk=False)
    inputs.spike_every_64th_key(k)
    for cut in (False, True):
        o, lse = _fwd(q, k, v, kl, d ** -0.5, True, cut)
        _check_fwd(o, lse, q, k, v, d ** -0.5, lens, f"cut={cut}")


@pytest.mark.parametrize("d", [64, 128])
def test_gradients_match_differences(d):
    """dV by the forward's linearity in V, dQ and dK along their own signs, with the forward's bound on
    each side and the curvature bound by a second, wider step in fp64."""
    B, Hq, Hkv, Nq, Nk, lens = 1, 4, 2, 60, 200, [170]
    q, k, v, do, kl = _inputs(B, Hq, Hkv, Nq, Nk, d, lens, junk=False)
    scale = d ** -0.5
    o, lse = _fwd(q, k, v, kl, scale)
    g = {n: torch.empty(x.shape, device=DEV) for n, x in (("dq", q), ("dk", k), ("dv", v))}
    fattn.fa_cross_bwd(q, k, v, o, do, lse, *g.values(), scale, kv_lens=kl)
    w = do.cpu().double().numpy()
    for i, n in enumerate(("dq", "dk", "dv")):
        step = torch.sign(g[n]) * 2.0 ** -3
        sides, slack, exact = [], 0.0, []
        for s in (1, -1):
            x = [q, k, v]
            x[i] = (x[i].float() + s * step).to(torch.bfloat16)
            oo, _ = _fwd(*x, kl, scale, o_fp32=True)
            sides.append((float((oo.double().cpu().numpy() * w).sum()), x[i].double()))
            ref, _, tol, _, _ = _bounds(*x, scale, lens)
            slack += float((np.abs(w) * tol).sum())
            exact.append(float((ref * w).sum()))
        moved = sides[0][1] - sides[1][1]  # (what the bf16 inputs really moved by)
        along = float((g[n].double() * moved).sum())
        # fp64 differences at the same points give the curvature's share
        curve = abs((exact[0] - exact[1]) - float((torch.from_numpy(
            oc.cross_backward(q, k, v, do, scale, lens)[0][n]).to(DEV) * moved).sum()))
        got = sides[0][0] - sides[1][0]
        assert abs(got - along) <= slack + curve + 2 * U * float((g[n].double() * moved).abs().sum()), n


def test_repeats_bitwise_and_matches_the_square_forward():
    B, H, N, d = 2, 3, 300, 128
    q, k, v, do, _ = _inputs(B, H, H, N, N, d, None)
    a, la = _fwd(q, k, v, None, 0.09)
    b, lb = _fwd(q, k, v, None, 0.09)
    assert torch.equal(a, b) and torch.equal(la, lb)
    o, lse = torch.empty_like(q), torch.empty(B, H, N, device=DEV)
    fattn.fa_fwd(q, k, v, o, lse, 0.09)
    c, lc = _fwd(q, k, v, None, 0.09, cut=False)
    assert torch.equal(o, c) and torch.equal(lse, lc)  # the same kernel, the same order
    grads = [[torch.empty_like(q) for _ in range(3)] for _ in range(2)]
    for g in grads:
        fattn.fa_cross_bwd(q, k, v, a, do, la, *g, 0.09)
    assert all(torch.equal(x, y) for x, y in zip(*grads))


@pytest.mark.parametrize("Nq,Nk", [(300, 700), (3, 700), (1, 20000), (5000, 77), (9000, 300)])
def test_a_wait_that_runs_out_is_reported(Nq, Nk):
    q, k, v, do, kl = _inputs(2, 4, 2, Nq, Nk, 128, [Nk, 650])
    o, lse = torch.empty_like(q), torch.empty(2, 4, Nq, device=DEV)
    fattn.fa_cross_fwd(q, k, v, o, lse, 0.1, kv_lens=kl, wait_budget_cycles=1)
    try:
        fattn.fa_get_status()
        # (a block of few rows has its few stages all in flight from the start: each can land within the
        # barrier instruction's own wait, and then no budget runs out and the result stands)
        assert Nq < 300
        _check_fwd(o, lse, q, k, v, 0.1, [Nk, 650], "within the budget")
    except fattn.FattnError as e:
        assert e.status == fattn.FA_ERR_TIMEOUT
    o, lse = _fwd(q, k, v, kl, 0.1)
    _check_fwd(o, lse, q, k, v, 0.1, [Nk, 650], "after a timeout")
    g = [torch.zeros_like(x) for x in (q, k, v)]
    fattn.fa_cross_bwd(q, k, v, o, do, lse, *g, 0.1, kv_lens=kl, wait_budget_cycles=1)
    with pytest.raises(fattn.FattnError) as e:
        fattn.fa_get_status()
    assert e.value.status == fattn.FA_ERR_TIMEOUT and fattn.fa_get_status() == fattn.FA_OK


def test_outputs_and_workspaces_keep_their_bounds():
    """Sentinels around every written buffer, workspaces of exactly the stated size."""
    for B, Hq, Hkv, Nq, Nk, d, lens in ((2, 6, 2, 43, 641, 64, [641, 200]), (1, 2, 2, 1, 1500, 128, [1400]),
                                        (1, 6, 2, 7, 20000, 128, [19000]),
                                        (1, 4, 4, 900, 70, 128, None), (1, 8, 4, 3001, 77, 64, [60]),
                                        (2, 4, 4, 700, 33, 128, [33, 0]), (1, 2, 2, 17, 97, 64, None)):
        q, k, v, do, kl = _inputs(B, Hq, Hkv, Nq, Nk, d, lens)

        def guarded(shape, dtype):
            n = math.prod(shape)
            t = torch.full((n + 512,), 7 if dtype == torch.uint8 else 7.0, dtype=dtype, device=DEV)
            return t, t[256:256 + n].view(shape)
        size = (B, Hq, Hkv, Nq, Nk, d)
        bufs = [guarded(s, t) for s, t in ((q.shape, torch.bfloat16), (q.shape[:3], torch.float32),
                                           ((fattn.fa_cross_workspace_bytes(*size),), torch.uint8),
                                           ((fattn.fa_cross_bwd_workspace_bytes(*size),), torch.uint8),
                                           (q.shape, torch.bfloat16), (k.shape, torch.bfloat16),
                                           (k.shape, torch.bfloat16))]
        o, lse, ws, wsb, dq, dk, dv = (b[1] for b in bufs)
        fattn.fa_cross_fwd(q, k, v, o, lse, 0.1, kv_lens=kl, workspace=ws if ws.numel() else None)
        fattn.fa_cross_bwd(q, k, v, o, do, lse, dq, dk, dv, 0.1, kv_lens=kl, workspace=wsb)
        assert fattn.fa_get_status() == fattn.FA_OK
        for whole, part in bufs:
            assert (whole[:256] == 7).all() and (whole[256 + part.numel():] == 7).all()
        _check_fwd(o, lse, q, k, v, 0.1, lens)


def test_workspaces_that_are_too_small_are_refused():
    q, k, v, do, _ = _inputs(1, 2, 2, 1, 20000, 128, None)
    o, lse = torch.empty_like(q), torch.empty(1, 2, 1, device=DEV)
    assert fattn.fa_cross_workspace_bytes(1, 2, 2, 1, 20000, 128) > 256
    small = torch.empty(256, dtype=torch.uint8, device=DEV)
    with pytest.raises(fattn.FattnError) as e:
        fattn.fa_cross_fwd(q, k, v, o, lse, 0.1, workspace=small)
    assert e.value.status == fattn.FA_ERR_WORKSPACE
    with pytest.raises(fattn.FattnError) as e:
        fattn.fa_cross_bwd(q, k, v, o, do, lse, torch.empty_like(q), torch.empty_like(k), torch.empty_like(v), 0.1,
                           workspace=small[:0])
    assert e.value.status == fattn.FA_ERR_WORKSPACE


def test_calls_on_two_streams_keep_apart():
    """Two streams, workspaces allocated inside the calls: neither call's partials reach the other."""
    assert fattn.fa_cross_workspace_bytes(1, 4, 2, 1, 9001, 128) > 0
    a = _inputs(1, 4, 2, 1, 9001, 128, [8900], seed=1)
    b = _inputs(1, 4, 2, 1, 9001, 128, [1777], seed=9)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for _ in range(10):
        for (q, k, v, _, kl), s in zip((a, b), streams):
            o, lse = torch.empty_like(q), torch.empty(1, 4, 1, device=DEV)
            fattn.fa_cross_fwd(q, k, v, o, lse, 0.09, kv_lens=kl, stream=s)
            outs.append((o, lse))
    torch.cuda.synchronize()
    assert fattn.fa_get_status() == fattn.FA_OK
    for i, (o, lse) in enumerate(outs):
        q, k, v, _, kl = (a, b)[i % 2]
        _check_fwd(o, lse, q, k, v, 0.09, kl.tolist(), f"call {i}")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nk", [50, 77, 128])
def test_few_keys_captured_and_repeated(Nk, d):
    """A training step over few keys, several blocks a key head: replayed with other inputs and lengths, on two streams
    with the workspaces of their graphs, and the same gradients bit for bit."""
    steps, size = [], (2, 8, 4, 4000, Nk, d)
    for seed, lens in ((1, [Nk, Nk // 2]), (5, [0, Nk - 1])):
        q, k, v, do, kl = _inputs(*size, lens, seed=seed)
        buf = [x.clone() for x in (q, k, v, do, kl)]
        out = [torch.empty_like(q), torch.empty(q.shape[:3], device=DEV), *(torch.empty_like(x) for x in (q, k, v))]
        steps.append(((q, k, v, do, kl), buf, out))

    def step(buf, out):
        (q, k, v, do, kl), (o, lse, *g) = buf, out
        fattn.fa_cross_fwd(q, k, v, o, lse, 0.1, kv_lens=kl)
        fattn.fa_cross_bwd(q, k, v, o, do, lse, *g, 0.1, kv_lens=kl)
    want = []
    for first, buf, out in steps:
        step(buf, out)
        want.append([x.clone() for x in out])
        step(buf, out)
        assert all(torch.equal(x, y) for x, y in zip(want[-1], out))
    streams, graphs = [torch.cuda.Stream(), torch.cuda.Stream()], []
    torch.cuda.synchronize()
    for s, (first, buf, out) in zip(streams, steps):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            step(buf, out)
    for turn in range(4):  # each graph's buffers get the other's inputs in turn
        for i, (_, buf, out) in enumerate(steps):
            for x, y in zip(buf, steps[(i + turn) % 2][0]):
                x.copy_(y)
            for x in out:
                x.fill_(float("nan"))
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for i, (_, _, out) in enumerate(steps):
            assert all(torch.equal(x, y) for x, y in zip(out, want[(i + turn) % 2])), f"graph {i}, turn {turn}"
    assert fattn.fa_get_status() == fattn.FA_OK


@pytest.mark.parametrize("fp32", [False, True])
def test_few_keys_past_32_bits(fp32):
    """The last sequence lies behind 2^31 elements: what a call of its own gives."""
    B, H, Nq, Nk, d = 66, 64, 8192, 77, 64
    t = torch.float32 if fp32 else torch.bfloat16
    q, do = (torch.zeros(B, H, Nq, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    k, v = (torch.zeros(B, H, Nk, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    last = _inputs(1, H, H, Nq, Nk, d, None)
    for x, y in zip((q, k, v, do), last):
        x[-1:] = y

    def step(q, k, v, do):
        o, lse = torch.empty_like(q), torch.empty(q.shape[:3], device=DEV)
        fattn.fa_cross_fwd(q, k, v, o, lse, 0.1)
        g = [torch.empty(x.shape, dtype=t, device=DEV) for x in (q, k, v)]
        fattn.fa_cross_bwd(q, k, v, o, do, lse, *g, 0.1)
        assert fattn.fa_get_status() == fattn.FA_OK
        return o, lse, *g
    got, want = step(q, k, v, do), step(*last[:4])
    for x, y in zip(got[:3], want[:3]):
        assert torch.equal(x[-1:], y)
    # dK and dV: other ranges of queries, so the same terms in another order, each side within Nq 2^-24 of their
    # absolute sum, and rounded to bf16.
    q, k, v, do = (x.double() for x in last[:4])
    p = (q @ k.mT * 0.1).softmax(-1)
    dp = do @ v.mT
    ds = p * (dp.abs() + (p * dp).sum(-1, keepdim=True).abs())
    for x, y, terms in zip(got[3:], want[3:], (0.1 * ds.mT @ q.abs(), p.mT @ do.abs())):
        slack = 2 * Nq * 2.0 ** -24 * (1 + 4 * U) * terms
        assert ((x[-1:].double() - y.double()).abs() <= slack + (0 if fp32 else 2 * U * (y.double().abs() + slack))).all()
