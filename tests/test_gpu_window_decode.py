"""One token of each sequence over a paged cache with a sliding window and sinks, on the GPU, against the fp64 definition.

The bounds are those of tests/test_gpu_window.py with the longest sequence's keys in place of Nk."""

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


def _cache(B, Hkv, L, d, ps, lens, W, S, seed=0, spare=3):
    """Pools in which keys that no token sees may be anything, and pages of none are not in the table at all."""
    g = torch.Generator().manual_seed(seed)
    mp = -(-L // ps)
    P = B * mp + spare
    table = torch.randperm(P, generator=g)[:B * mp].to(torch.int32).view(B, mp)
    k, v = inputs.normal_bf16((B, Hkv, mp * ps, d), seed + 1, DEV), inputs.normal_bf16((B, Hkv, mp * ps, d), seed + 2, DEV)
    kp = torch.full((P, Hkv, ps, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    vp = torch.full((P, Hkv, ps, d), float("inf"), dtype=torch.bfloat16, device=DEV)
    key = torch.arange(mp * ps)
    for b, n in enumerate(min(max(x, 0), L) for x in lens):
        seen = (key < n) & ((key >= n - W) | (key < S))
        for i in range(mp):
            rows = seen[i * ps:(i + 1) * ps].to(DEV)
            if not rows.any():
                table[b, i] = (-1, P, 2 ** 31 - 1, -2 ** 31)[i % 4]  # given back: nothing reads it
                continue
            at = slice(i * ps, (i + 1) * ps)
            kp[table[b, i], :, rows] = k[b, :, at][:, rows]
            vp[table[b, i], :, rows] = v[b, :, at][:, rows]
    return k, v, kp, vp, table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)


def _run(q, kp, vp, table, lens, scale, L, W, S, o_fp32=False, **kw):
    o = torch.full(q.shape, float("nan"), dtype=torch.float32 if o_fp32 else torch.bfloat16, device=DEV)
    lse = torch.full(q.shape[:2], float("nan"), device=DEV)
    fattn.fa_window_decode_paged(q, kp, vp, table, lens, o, lse, scale, L, W, S, **kw)
    assert fattn.fa_get_status() == fattn.FA_OK
    return o, lse


def _check(o, lse, q, k, v, lens, scale, L, W, S, what=""):
    lens = [min(max(int(n), 0), L) for n in lens]
    ref, lref, pv, big = ow.window_decode(q, k, v, lens, scale, W, S)
    eps = q.shape[2] * 2.0 ** -24 * big + 2.0 ** -18
    tol = (U + 2 * eps + 2 * L * 2.0 ** -24) * pv
    if o.dtype == torch.bfloat16:
        tol = tol + U * (np.abs(ref) + tol)
    got, gl = o.cpu().double().numpy(), lse.cpu().double().numpy()
    empty = np.isneginf(lref)
    assert np.isneginf(gl[empty]).all() and (got[empty] == 0).all(), f"{what}: empty sequences"
    assert np.isfinite(got).all() and (np.abs(got - ref) <= tol + 1e-30).all(), f"{what} o: {np.abs(got - ref).max():.3e}"
    err, size = np.abs(gl[~empty] - lref[~empty]), np.abs(lref[~empty])
    assert (err <= eps + L * 2.0 ** -24 + 2.0 ** -22 * size).all(), f"{what} lse"


CASES = [  # B, Hq, Hkv, page size, longest, lens, window, sinks
    (1, 1, 1, 64, 1, [1], 1, 0), (2, 2, 1, 64, 64, [64, 0], 1, 1), (3, 4, 2, 64, 200, [200, 130, 3], 64, 4),
    (2, 8, 1, 128, 300, [300, 129], 2 ** 31 - 1, 128), (2, 6, 2, 192, 1000, [999, 640], 100, 128),
    (4, 4, 4, 64, 640, [640, -3, 641, 65], 63, 0), (1, 16, 1, 64, 3000, [2999], 65, 100), (1, 17, 1, 64, 700, [700], 130, 7),
    (2, 32, 1, 128, 700, [650, 64], 300, 64), (1, 32, 8, 64, 5000, [4999], 4096, 16), (2, 5, 5, 64, 20000, [20000, 777], 9000, 5),
    (2, 2, 2, 64, 130, [129, 128], 2, 65), (2, 2, 1, 64, 400, [320, 384], 128, 128), (1, 3, 1, 256, 500, [257], 1, 128),
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Hq,Hkv,ps,L,lens,W,S", CASES)
def test_decode(B, Hq, Hkv, ps, L, lens, W, S, d):
    q = inputs.normal_bf16((B, Hq, d), 9, DEV)
    k, v, kp, vp, table, kl = _cache(B, Hkv, L, d, ps, lens, W, S)
    for o_fp32 in (False, True):
        o, lse = _run(q, kp, vp, table, kl, d ** -0.5, L, W, S, o_fp32)
        _check(o, lse, q, k, v, lens, d ** -0.5, L, W, S, f"fp32={o_fp32}")


@pytest.mark.parametrize("d", [64, 128])
def test_one_kernel_and_partials_agree(d):
    """Few long sequences: ranges of keys that leave partials, and with no workspace a cluster alone."""
    import ctypes
    B, Hq, Hkv, ps, L, W, S = 1, 4, 2, 64, 30000, 29000, 4
    q = inputs.normal_bf16((B, Hq, d), 9, DEV)
    k, v, kp, vp, table, kl = _cache(B, Hkv, L, d, ps, [L - 5], W, S)
    need = fattn.fa_window_decode_paged_workspace_bytes(B, Hq, Hkv, d, ps, table.shape[1], L, W, S)
    assert need > 256
    whole = torch.full((need + 512,), 7, dtype=torch.uint8, device=DEV)
    o, lse = _run(q, kp, vp, table, kl, 0.1, L, W, S, workspace=whole[256:256 + need])
    assert (whole[:256] == 7).all() and (whole[-256:] == 7).all()
    _check(o, lse, q, k, v, [L - 5], 0.1, L, W, S)
    with pytest.raises(fattn.FattnError) as e:
        _run(q, kp, vp, table, kl, 0.1, L, W, S, workspace=whole[:need - 256])
    assert e.value.status == fattn.FA_ERR_WORKSPACE
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    st = fattn.lib().fa_window_decode_paged(p(q), p(kp), p(vp), p(table), p(kl), p(o2), p(lse2), B, Hq, Hkv, d, ps,
                                            table.shape[1], kp.shape[0], L, ctypes.c_float(0.1), W, S, None, 0,
                                            ctypes.c_void_p(torch.cuda.current_stream().cuda_stream), None)
    assert st == fattn.FA_OK and fattn.fa_get_status() == fattn.FA_OK
    _check(o2, lse2, q, k, v, [L - 5], 0.1, L, W, S)


def test_matches_the_paged_decode_of_every_key():
    B, H, ps, L, d = 3, 4, 64, 900, 128
    q = inputs.normal_bf16((B, H, d), 9, DEV)
    lens = [900, 333, 64]
    k, v, kp, vp, table, kl = _cache(B, H, L, d, ps, lens, L, 0)
    o, lse = _run(q, kp, vp, table, kl, 0.1, L, L, 0, True)
    want, wl = torch.empty_like(o), torch.empty_like(lse)
    fattn.fa_decode_paged(q, kp, vp, table, kl, want, wl, 0.1, L)
    _check(want, wl, q, k, v, lens, 0.1, L, L, 0)
    _check(o, lse, q, k, v, lens, 0.1, L, L, 0)


def test_pages_outside_the_pool_read_as_zeros():
    B, H, ps, L, d = 2, 2, 64, 300, 64
    q = inputs.normal_bf16((B, H, d), 9, DEV)
    k, v, kp, vp, table, kl = _cache(B, H, L, d, ps, [300, 200], 150, 10)
    table[0, 3], table[1, 0] = kp.shape[0], -7
    k[0, :, 192:256], v[0, :, 192:256], k[1, :, :64], v[1, :, :64] = 0, 0, 0, 0
    o, lse = _run(q, kp, vp, table, kl, 0.1, L, 150, 10)
    _check(o, lse, q, k, v, [300, 200], 0.1, L, 150, 10)


@pytest.mark.parametrize("d", [64, 128])
def test_many_sequences(d):
    B, Hq, Hkv, ps, L, W, S = 150, 8, 2, 64, 900, 333, 17
    lens = torch.randint(0, L + 1, (B,), generator=torch.Generator().manual_seed(3)).tolist()
    q = inputs.normal_bf16((B, Hq, d), 9, DEV)
    k, v, kp, vp, table, kl = _cache(B, Hkv, L, d, ps, lens, W, S)
    o, lse = _run(q, kp, vp, table, kl, d ** -0.5, L, W, S)
    _check(o, lse, q, k, v, lens, d ** -0.5, L, W, S)
    again = _run(q, kp, vp, table, kl, d ** -0.5, L, W, S, stream=torch.cuda.current_stream())
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


def test_a_pool_past_32_bits():
    """Pages behind 2^31 elements of the pools."""
    ps, d, Hkv = 128, 128, 8
    P = 2 ** 31 // (ps * d * Hkv) + 40
    kp, vp = (torch.zeros(P, Hkv, ps, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    k, v = inputs.normal_bf16((1, Hkv, 10 * ps, d), 1, DEV), inputs.normal_bf16((1, Hkv, 10 * ps, d), 2, DEV)
    table = torch.arange(P - 10, P, dtype=torch.int32, device=DEV).flip(0).view(1, 10).contiguous()
    for i in range(10):
        kp[table[0, i]], vp[table[0, i]] = k[0, :, i * ps:(i + 1) * ps], v[0, :, i * ps:(i + 1) * ps]
    q = inputs.normal_bf16((1, 32, d), 9, DEV)
    lens = torch.tensor([1200], dtype=torch.int32, device=DEV)
    o, lse = _run(q, kp, vp, table, lens, 0.1, 1280, 700, 20)
    _check(o, lse, q, k, v, [1200], 0.1, 1280, 700, 20)


def test_a_wait_that_runs_out_is_reported_or_unneeded():
    k, v, kp, vp, table, kl = _cache(2, 2, 4000, 128, 64, [4000, 3900], 3000, 4)
    q = inputs.normal_bf16((2, 4, 128), 9, DEV)
    o, lse = torch.empty_like(q), torch.empty(2, 4, device=DEV)
    fattn.fa_window_decode_paged(q, kp, vp, table, kl, o, lse, 0.1, 4000, 3000, 4, wait_budget_cycles=1)
    try:
        fattn.fa_get_status()
        _check(o, lse, q, k, v, [4000, 3900], 0.1, 4000, 3000, 4)  # (each stage landed within the instruction's own wait)
    except fattn.FattnError as e:
        assert e.status == fattn.FA_ERR_TIMEOUT
    o, lse = _run(q, kp, vp, table, kl, 0.1, 4000, 3000, 4)
    _check(o, lse, q, k, v, [4000, 3900], 0.1, 4000, 3000, 4)
