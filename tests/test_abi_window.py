"""Sliding windows, norms with rotary positions and the cache's pages: every refusal of the C ABI and of the binding comes
before anything is launched (no GPU)."""

import ctypes

import pytest
import torch

from _util import ensure_built

vp, cf = ctypes.c_void_p, ctypes.c_float
BIG = 2 ** 31 - 1


@pytest.fixture(scope="module")
def fattn():
    ensure_built()
    from exact_attention_06_gb300 import fattn
    fattn.lib()
    return fattn


def _ptrs(n):
    return tuple(1024 * (j + 1) for j in range(n))


def _at(n, i, value):
    return tuple(value if j == i else x for j, x in enumerate(_ptrs(n)))


def _fwd(f, p=_ptrs(5), B=1, Hq=2, Hkv=1, N=4, Nk=8, d=64, scale=0.125, W=3, S=1, opts=None):
    return f.lib().fa_window_fwd(*map(vp, p), B, Hq, Hkv, N, Nk, d, cf(scale), W, S, vp(0),
                                 ctypes.byref(opts) if opts else None)


def _bwd(f, p=_ptrs(9), B=1, Hq=2, Hkv=1, N=4, Nk=8, d=64, scale=0.125, W=3, S=1, fp32=0, ws=256, wsb=1 << 30):
    return f.lib().fa_window_bwd(*map(vp, p), B, Hq, Hkv, N, Nk, d, cf(scale), W, S, fp32, vp(ws), wsb, vp(0), None)


def _decode(f, p=_ptrs(7), B=1, Hq=2, Hkv=1, d=64, ps=64, mp=4, npg=8, L=200, scale=0.125, W=3, S=1, ws=0, wsb=0, opts=None):
    return f.lib().fa_window_decode_paged(*map(vp, p), B, Hq, Hkv, d, ps, mp, npg, L, cf(scale), W, S, vp(ws), wsb, vp(0),
                                          ctypes.byref(opts) if opts else None)


SIZES = [dict(B=0), dict(Hq=0), dict(Hkv=0), dict(Hq=3, Hkv=2), dict(Hq=1, Hkv=2), dict(scale=0.0), dict(scale=float("nan")),
         dict(W=0), dict(W=-1), dict(S=-1)]
SQUARE = SIZES + [dict(N=0), dict(Nk=0), dict(N=9)]
TOO_BIG = [dict(d=96), dict(B=1 << 16, Hq=1 << 16, Hkv=1 << 16), dict(S=129)]


def test_window_refusals(fattn):
    for i in range(5):
        assert _fwd(fattn, _at(5, i, 0)) == fattn.FA_ERR_INVALID_ARG
        assert _fwd(fattn, _at(5, i, 18 if i == 4 else 24)) == fattn.FA_ERR_INVALID_ARG
    for i in range(9):
        assert _bwd(fattn, _at(9, i, 0)) == fattn.FA_ERR_INVALID_ARG
        assert _bwd(fattn, _at(9, i, 18 if i == 5 else 24)) == fattn.FA_ERR_INVALID_ARG
    assert _fwd(fattn, opts=fattn.FaWindowOpts(2, 0)) == fattn.FA_ERR_INVALID_ARG
    for bad in SQUARE:
        assert _fwd(fattn, **bad) == fattn.FA_ERR_INVALID_ARG, bad
        assert _bwd(fattn, **bad) == fattn.FA_ERR_INVALID_ARG, bad
    for out in (6, 7, 8):  # outputs are tensors of their own
        for other in set(range(9)) - {5, out}:
            assert _bwd(fattn, _at(9, out, _ptrs(9)[other])) == fattn.FA_ERR_INVALID_ARG
    for other in range(3):
        assert _fwd(fattn, _at(5, 3, _ptrs(5)[other])) == fattn.FA_ERR_INVALID_ARG
    for bad in TOO_BIG + [dict(N=BIG, Nk=BIG, B=128), dict(Nk=2 ** 30 + 1)]:
        assert _fwd(fattn, **bad) == fattn.FA_ERR_UNSUPPORTED, bad
        assert _bwd(fattn, **bad) == fattn.FA_ERR_UNSUPPORTED, bad
    assert _bwd(fattn, fp32=2) == fattn.FA_ERR_INVALID_ARG and _bwd(fattn, ws=128) == fattn.FA_ERR_INVALID_ARG
    assert _bwd(fattn, ws=0) == fattn.FA_ERR_WORKSPACE
    assert fattn.lib().fa_window_bwd_workspace_bytes(1, 2, 1, 9, 8, 64, 3, 1) == 0
    if not torch.cuda.is_available():  # valid calls get as far as the device
        assert _fwd(fattn, W=BIG, S=128) == fattn.FA_ERR_ARCH and _bwd(fattn) == fattn.FA_ERR_ARCH


def test_window_decode_refusals(fattn):
    for i in range(7):
        assert _decode(fattn, _at(7, i, 0)) == fattn.FA_ERR_INVALID_ARG
        assert _decode(fattn, _at(7, i, 18 if i in (3, 4, 6) else 24)) == fattn.FA_ERR_INVALID_ARG
    for bad in SIZES + [dict(mp=0), dict(npg=0), dict(L=0), dict(L=257), dict(ws=128, wsb=1 << 30),
                        dict(opts=fattn.FaDecodeOpts(2, 0))]:
        assert _decode(fattn, **bad) == fattn.FA_ERR_INVALID_ARG, bad
    for bad in TOO_BIG[:1] + TOO_BIG[2:] + [dict(ps=96), dict(ps=0), dict(Hq=33), dict(npg=1 << 30, Hkv=4, Hq=4)]:
        assert _decode(fattn, **bad) == fattn.FA_ERR_UNSUPPORTED, bad
    assert fattn.lib().fa_window_decode_paged_workspace_bytes(1, 33, 1, 64, 64, 4, 200, 3, 1) == 0
    if not torch.cuda.is_available():
        assert _decode(fattn, W=BIG, S=128) == fattn.FA_ERR_ARCH


def _plan(f, d=64):
    return f.fa_rope_axes_plan(d, (d // 2,))


def _norm(f, p=_ptrs(7), B=1, Hq=2, Hk=1, N=4, eps=1e-6, w32=1, plan=0):
    q, k, qw, kw, pos, qo, ko = p
    pl = _plan(f) if plan == 0 else plan
    return f.lib().fa_norm_rope_axes(vp(q), vp(k), vp(qw), vp(kw), w32, vp(pos), vp(qo), vp(ko), B, Hq, Hk, N, cf(eps),
                                     ctypes.byref(pl) if pl else None, vp(0))


def _norm_bwd(f, p=(16,) * 11, B=1, Hq=2, Hk=1, N=4, eps=1e-6, w32=1, plan=0, ws=256, wsb=1 << 30):
    q, k, qw, kw, pos, gq, gk, dq, dk, dwq, dwk = p
    pl = _plan(f) if plan == 0 else plan
    return f.lib().fa_norm_rope_axes_bwd(vp(q), vp(k), vp(qw), vp(kw), w32, vp(pos), vp(gq), vp(gk), vp(dq), vp(dk), vp(dwq),
                                         vp(dwk), B, Hq, Hk, N, cf(eps), ctypes.byref(pl) if pl else None, vp(ws), wsb, vp(0))


def _norm_paged(f, p=(16,) * 10, new=0, B=1, Hq=2, Hk=1, N=1, ps=64, npg=2, eps=1e-6, w32=1, plan=0):
    q, k, v, qw, kw, pos, qo, kp, vpg, slots = p
    pl = _plan(f) if plan == 0 else plan
    return f.lib().fa_norm_rope_axes_paged(vp(q), vp(k), vp(v), vp(qw), vp(kw), w32, vp(pos), vp(qo), vp(kp), vp(vpg),
                                           vp(slots), vp(new), B, Hq, Hk, N, ps, npg, cf(eps),
                                           ctypes.byref(pl) if pl else None, vp(0))


def test_norm_refusals(fattn):
    blank = fattn.FaRopeAxesPlan()
    for call, n, optional, odd in ((_norm, 7, {2, 3}, {2: 18, 3: 18, 4: 18}),
                                   (_norm_bwd, 11, {2, 3, 9, 10}, {2: 18, 3: 18, 4: 18, 9: 18, 10: 18}),
                                   (_norm_paged, 10, {3, 4}, {3: 18, 4: 18, 5: 18, 9: 20})):
        for i in range(n):
            if i not in optional:
                assert call(fattn, _at(n, i, 0)) == fattn.FA_ERR_INVALID_ARG, (call, i)
            assert call(fattn, _at(n, i, odd.get(i, 24))) == fattn.FA_ERR_INVALID_ARG, (call, i)
        for bad in (dict(B=0), dict(Hq=0), dict(Hk=-1), dict(N=0), dict(eps=0.0), dict(eps=float("inf")), dict(w32=2),
                    dict(plan=None), dict(plan=blank)):
            assert call(fattn, **bad) == fattn.FA_ERR_INVALID_ARG, (call, bad)
        for bad in (dict(Hq=65536), dict(B=1 << 16, N=1 << 16)):
            assert call(fattn, **bad) == fattn.FA_ERR_UNSUPPORTED, (call, bad)
    for bad in (dict(new=18), dict(Hk=0), dict(npg=0)):
        assert _norm_paged(fattn, **bad) == fattn.FA_ERR_INVALID_ARG, bad
    for bad in (dict(ps=96), dict(npg=1 << 30, Hk=4, Hq=4)):
        assert _norm_paged(fattn, **bad) == fattn.FA_ERR_UNSUPPORTED, bad
    assert fattn.lib().fa_norm_rope_axes_bwd_workspace_bytes(1, 0, 1, 4, 64) == 0
    if not torch.cuda.is_available():
        assert _norm(fattn, (16, 0, 0, 0, 16, 16, 0), Hk=0) == fattn.FA_ERR_ARCH
        assert _norm(fattn, (16, 16, 18, 18, 16, 16, 16), w32=0) == fattn.FA_ERR_ARCH  # (bf16 weights)


def _pages(f, p=(16, 32, 48, 64, 80, 96), slots=0, B=2, N=1, ps=64, mp=4, npg=8):
    return f.lib().fa_pages_extend(*map(vp, p), vp(slots), B, N, ps, mp, npg, vp(0))


def test_pages_refusals(fattn):
    base = (16, 32, 48, 64, 80, 96)
    for i in range(6):
        for bad in (0, 18):
            assert _pages(fattn, tuple(bad if j == i else x for j, x in enumerate(base))) == fattn.FA_ERR_INVALID_ARG
    for i, j in ((1, 2), (1, 5), (2, 5)):  # lengths, changes and grants are arrays of their own
        p = list(base)
        p[i] = p[j]
        assert _pages(fattn, p) == fattn.FA_ERR_INVALID_ARG
    for bad in (dict(slots=20), dict(B=0), dict(mp=0), dict(npg=0), dict(slots=16, N=0)):
        assert _pages(fattn, **bad) == fattn.FA_ERR_INVALID_ARG, bad
    for bad in (dict(ps=0), dict(ps=96), dict(mp=1 << 25), dict(B=1 << 20, mp=1 << 12), dict(slots=16, B=1 << 20, N=1 << 22), dict(slots=16, N=BIG)):
        assert _pages(fattn, **bad) == fattn.FA_ERR_UNSUPPORTED, bad
    if not torch.cuda.is_available():
        assert _pages(fattn, N=0) == fattn.FA_ERR_ARCH and _pages(fattn, slots=16) == fattn.FA_ERR_ARCH


def test_binding_refuses_what_the_library_cannot_read(fattn):
    q = torch.zeros(1, 4, 8, 64, dtype=torch.bfloat16)
    k = torch.zeros(1, 2, 9, 64, dtype=torch.bfloat16)
    k8, q1 = k[:, :, :8].contiguous(), q[:, :, 0].contiguous()
    lse, plan, w = torch.zeros(1, 4, 8), _plan(fattn), torch.zeros(64)
    pos, table = torch.zeros(1, 1, 8, dtype=torch.int32), torch.zeros(1, 4, dtype=torch.int32)
    lens, slots = table[0, :1], torch.zeros(1, 8, dtype=torch.int64)

    def refused(fn, *args, what, **kw):
        with pytest.raises(fattn.FattnError) as e:
            fn(*args, **kw)
        assert e.value.status == fattn.FA_ERR_INVALID_ARG and what in str(e.value), str(e.value)

    refused(fattn.fa_window_fwd, q, k, k, q, lse, 0.1, 3, what="CUDA")
    refused(fattn.fa_window_fwd, q[0], k, k, q, lse, 0.1, 3, what="4-dimensional")
    refused(fattn.fa_window_fwd, q.transpose(1, 2), k, k, q, lse, 0.1, 3, what="contiguous")
    refused(fattn.fa_window_bwd, q.float(), k, k, q, q, lse, q, k, k, 0.1, 3, what="dtype")
    refused(fattn.fa_window_decode_paged, q, k, k, table, lens, q1, lse[:, :, 0], 0.1, 9, 3, what="3-dimensional")
    refused(fattn.fa_window_decode_paged, q1, k, k, lens, lens, q1, lse[:, :, 0], 0.1, 9, 3, what="2-dimensional")
    refused(fattn.fa_window_decode_paged, q1, k.half(), k, table, lens, q1, lse[:, :, 0], 0.1, 9, 3, what="q must be a CUDA")
    refused(fattn.fa_norm_rope_axes, q.float(), None, w, w, pos, plan, what="dtype")
    refused(fattn.fa_norm_rope_axes, None, None, w, w, pos, plan, what="4-dimensional")
    refused(fattn.fa_norm_rope_axes_bwd, q, k8[0], w, w, pos, plan, q, k8, what="CUDA")
    refused(fattn.fa_norm_rope_axes_paged, q, k8, k8, w, w, pos, plan, q, k[0], k, slots, what="4-dimensional")
    refused(fattn.fa_pages_extend, lens, lens, lens, lens, lens, lens, None, 64, what="2-dimensional")
    refused(fattn.fa_pages_extend, table, lens, lens, lens, lens, lens, lens, 64, what="2-dimensional")
    refused(fattn.fa_pages_extend, table, lens, lens, lens, lens, lens, None, 64, what="CUDA")
