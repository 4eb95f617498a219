"""Cross attention and rotary positions: every refusal of the C ABI and of the binding comes before
anything is launched (no GPU), and the rotary plan is the definition's table."""

import ctypes

import numpy as np
import pytest
import torch

from _util import ensure_built
from oracle import cross as oc

vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def fattn():
    ensure_built()
    from exact_attention_06_gb300 import fattn
    fattn.lib()
    return fattn


def _cross(f, q=16, k=16, v=16, lens=0, o=16, lse=16, B=1, Hq=2, Hkv=1, Nq=4, Nk=8, d=64, scale=0.125, ws=0, wsb=0,
           opts=None):
    return f.lib().fa_cross_fwd(vp(q), vp(k), vp(v), vp(lens), vp(o), vp(lse), B, Hq, Hkv, Nq, Nk, d,
                                ctypes.c_float(scale), vp(ws), wsb, vp(0), ctypes.byref(opts) if opts else None)


def _cross_bwd(f, p=(16,) * 9, lens=0, B=1, Hq=2, Hkv=1, Nq=4, Nk=8, d=64, scale=0.125, fp32=0, ws=256, wsb=1 << 30):
    q, k, v, o, do, lse, dq, dk, dv = p
    return f.lib().fa_cross_bwd(vp(q), vp(k), vp(v), vp(lens), vp(o), vp(do), vp(lse), vp(dq), vp(dk), vp(dv), B, Hq,
                                Hkv, Nq, Nk, d, ctypes.c_float(scale), fp32, vp(ws), wsb, vp(0), None)


SIZES = [dict(B=0), dict(Hq=0), dict(Hkv=0), dict(Nq=0), dict(Nk=0), dict(Hq=3, Hkv=2), dict(Hq=1, Hkv=2),
         dict(scale=0.0), dict(scale=float("inf")), dict(lens=6)]
TOO_BIG = [dict(d=96), dict(B=1 << 16, Hq=1 << 16, Hkv=1 << 16), dict(Nq=65535 * 64 + 1), dict(Nk=65535 * 128 + 1),
           dict(Nk=2 ** 31 - 1)]


def test_cross_forward_refusals(fattn):
    for name in ("q", "k", "v", "o", "lse"):
        assert _cross(fattn, **{name: 0}) == fattn.FA_ERR_INVALID_ARG
    for name in ("q", "k", "v", "o"):
        assert _cross(fattn, **{name: 24}) == fattn.FA_ERR_INVALID_ARG
    assert _cross(fattn, lse=18) == fattn.FA_ERR_INVALID_ARG
    assert _cross(fattn, ws=128, wsb=1 << 30) == fattn.FA_ERR_INVALID_ARG
    assert _cross(fattn, opts=fattn.FaCrossOpts(2, 0)) == fattn.FA_ERR_INVALID_ARG
    for bad in SIZES:
        assert _cross(fattn, **bad) == fattn.FA_ERR_INVALID_ARG, bad
    for bad in TOO_BIG:
        assert _cross(fattn, **bad) == fattn.FA_ERR_UNSUPPORTED, bad
    assert fattn.lib().fa_cross_workspace_bytes(1, 3, 2, 4, 8, 64) == 0
    if not torch.cuda.is_available():  # a valid call gets as far as the device
        assert _cross(fattn) == fattn.FA_ERR_ARCH


def test_cross_backward_refusals(fattn):
    for i in range(9):
        assert _cross_bwd(fattn, p=tuple(0 if j == i else 16 for j in range(9))) == fattn.FA_ERR_INVALID_ARG
        odd = 18 if i == 5 else 24
        assert _cross_bwd(fattn, p=tuple(odd if j == i else 16 for j in range(9))) == fattn.FA_ERR_INVALID_ARG
    for bad in SIZES + [dict(fp32=2), dict(ws=128)]:
        assert _cross_bwd(fattn, **bad) == fattn.FA_ERR_INVALID_ARG, bad
    for bad in TOO_BIG:
        assert _cross_bwd(fattn, **bad) == fattn.FA_ERR_UNSUPPORTED, bad
    assert _cross_bwd(fattn, ws=0) == fattn.FA_ERR_WORKSPACE
    assert fattn.lib().fa_cross_bwd_workspace_bytes(1, 0, 1, 4, 8, 64) == 0


def test_plan_refusals(fattn):
    for kw in (dict(sections=(32, 1)), dict(sections=(31,)), dict(sections=(0, 32)), dict(sections=(-1, 33)),
               dict(sections=()), dict(sections=(8, 8, 8, 4, 4)), dict(base=0.5), dict(base=float("nan")),
               dict(base=float("inf"))):
        with pytest.raises(fattn.FattnError) as e:
            fattn.fa_rope_axes_plan(64, **{"sections": (16, 16), **kw})
        assert e.value.status == fattn.FA_ERR_INVALID_ARG, kw
    with pytest.raises(fattn.FattnError) as e:
        fattn.fa_rope_axes_plan(96, (24, 24))
    assert e.value.status == fattn.FA_ERR_UNSUPPORTED
    s = (ctypes.c_int * 1)(32)
    p = fattn.FaRopeAxesPlan()
    assert fattn.lib().fa_rope_axes_plan(None, 64, 1, s, 10.0, 0, 0, 0) == fattn.FA_ERR_INVALID_ARG
    assert fattn.lib().fa_rope_axes_plan(ctypes.byref(p), 64, 1, None, 10.0, 0, 0, 0) == fattn.FA_ERR_INVALID_ARG
    for flags in ((2, 0, 0), (0, -1, 0), (0, 0, 3)):
        assert fattn.lib().fa_rope_axes_plan(ctypes.byref(p), 64, 1, s, 10.0, *flags) == fattn.FA_ERR_INVALID_ARG


@pytest.mark.parametrize("d,sections", [(64, (32,)), (64, (8, 12, 12)), (128, (16, 24, 24)), (128, (1, 2, 3, 58)),
                                        (128, (32, 32))])
@pytest.mark.parametrize("per_axis", [False, True])
@pytest.mark.parametrize("cyclic", [False, True])
@pytest.mark.parametrize("base", [1.0, 10000.0, 1e6])
def test_plan_is_the_definition(fattn, d, sections, per_axis, cyclic, base):
    plan = fattn.fa_rope_axes_plan(d, sections, base, True, per_axis, cyclic)
    axis, rates = oc.rope_rates(d, sections, base, per_axis, cyclic)
    assert (plan.d, plan.n_axes, plan.interleaved) == (d, len(sections), 1)
    assert list(plan.axis)[:d // 2] == axis
    turns = np.array([np.longdouble(int(t)) for t in list(plan.turns)[:d // 2]]) / np.longdouble(2) ** 64
    want = rates / (2 * np.longdouble("3.14159265358979323846264338327950288"))
    # The entry is the nearest multiple of 2^-64: half of that, 2^-65, absolute.  Relative, in units of
    # u = 2^-53 (half a double's step): pow's result 2 u, the product and the constant 1 / (2 pi) u each,
    # and the exponent's own rounding (u of an exponent <= 1) changes base^-e by ln(base) u <= 14 u.
    assert np.all(np.abs(turns - want) <= 2.0 ** -65 + (4 + np.log(base)) * 2.0 ** -53 * want)


def _plan(f, d=64):
    return f.fa_rope_axes_plan(d, (d // 2,))


def _rope(f, q=16, k=16, pos=16, qo=16, ko=16, B=1, Hq=2, Hk=1, N=4, plan=0, inverse=0):
    p = _plan(f) if plan == 0 else plan
    return f.lib().fa_rope_axes(vp(q), vp(k), vp(pos), vp(qo), vp(ko), B, Hq, Hk, N,
                                ctypes.byref(p) if p else None, inverse, vp(0))


def _paged(f, p=(16,) * 9, new=0, B=1, Hq=2, Hk=1, N=1, ps=64, mp=2, npg=2, plan=0):
    q, k, v, pos, qo, kp, vpg, bt, sl = p
    pl = _plan(f) if plan == 0 else plan
    return f.lib().fa_rope_axes_paged(vp(q), vp(k), vp(v), vp(pos), vp(qo), vp(kp), vp(vpg), vp(bt), vp(sl), vp(new),
                                      B, Hq, Hk, N, ps, mp, npg, ctypes.byref(pl) if pl else None, vp(0))


def test_rope_refusals(fattn):
    for name in ("q", "k", "pos", "qo", "ko"):
        assert _rope(fattn, **{name: 0}) == fattn.FA_ERR_INVALID_ARG
        assert _rope(fattn, **{name: 18 if name == "pos" else 24}) == fattn.FA_ERR_INVALID_ARG
    bad_axis, blank = _plan(fattn), fattn.FaRopeAxesPlan()
    bad_axis.axis[5] = 1
    for bad in (dict(B=0), dict(Hq=0), dict(Hk=-1), dict(N=0), dict(inverse=2), dict(plan=None), dict(plan=blank),
                dict(plan=bad_axis)):
        assert _rope(fattn, **bad) == fattn.FA_ERR_INVALID_ARG, bad
    assert _rope(fattn, Hq=65536) == fattn.FA_ERR_UNSUPPORTED
    assert _rope(fattn, B=1 << 16, N=1 << 16) == fattn.FA_ERR_UNSUPPORTED
    if not torch.cuda.is_available():
        assert _rope(fattn, k=0, ko=0, Hk=0) == fattn.FA_ERR_ARCH  # q alone is a valid call


def test_rope_paged_refusals(fattn):
    for i in range(9):
        assert _paged(fattn, p=tuple(0 if j == i else 16 for j in range(9))) == fattn.FA_ERR_INVALID_ARG
        odd = 18 if i in (3, 7, 8) else 24
        assert _paged(fattn, p=tuple(odd if j == i else 16 for j in range(9))) == fattn.FA_ERR_INVALID_ARG
    for bad in (dict(new=18), dict(B=0), dict(Hk=0), dict(N=0), dict(mp=0), dict(npg=0), dict(plan=None)):
        assert _paged(fattn, **bad) == fattn.FA_ERR_INVALID_ARG, bad
    for bad in (dict(ps=96), dict(ps=0), dict(npg=1 << 30, Hk=4, Hq=4), dict(Hk=40000, Hq=40000)):
        assert _paged(fattn, **bad) == fattn.FA_ERR_UNSUPPORTED, bad


def test_binding_refuses_what_the_library_cannot_read(fattn):
    q = torch.zeros(1, 4, 8, 64, dtype=torch.bfloat16)
    k = torch.zeros(1, 2, 5, 64, dtype=torch.bfloat16)
    lse, plan = torch.zeros(1, 4, 8), _plan(fattn)
    pos = torch.zeros(1, 1, 8, dtype=torch.int32)

    def refused(fn, *args, what, **kw):
        with pytest.raises(fattn.FattnError) as e:
            fn(*args, **kw)
        assert e.value.status == fattn.FA_ERR_INVALID_ARG and what in str(e.value), str(e.value)

    refused(fattn.fa_cross_fwd, q, k, k, q, lse, 0.1, what="CUDA")
    refused(fattn.fa_cross_fwd, q[0], k, k, q, lse, 0.1, what="4-dimensional")
    refused(fattn.fa_cross_fwd, q.half(), k, k, q, lse, 0.1, what="dtype")
    refused(fattn.fa_cross_fwd, q.transpose(1, 2), k, k, q, lse, 0.1, what="contiguous")
    refused(fattn.fa_cross_bwd, q.float(), k, k, q, q, lse, q, k, k, 0.1, what="dtype")
    refused(fattn.fa_rope_axes, q.float(), None, pos, plan, what="dtype")
    refused(fattn.fa_rope_axes, None, None, pos, plan, what="4-dimensional")
    refused(fattn.fa_rope_axes_paged, q, k, k, pos, plan, q, k[0], k, pos[0], pos[0, 0], what="4-dimensional")
    refused(fattn.fa_rope_axes_paged, q, k, k, pos, plan, q, k, k, pos, pos[0, 0], what="2-dimensional")
