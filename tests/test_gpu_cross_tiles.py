"""Every tile of query rows reaches dK and dV, and only once: dO is zero but for one tile of 128 rows of each key head, and
that tile moves over the whole scan (its first tiles, the turns of the rings, the borders of the blocks' ranges, the last).

A bound on gradients that sum over thousands of rows grows with their number, the gradients themselves with its root, so a
lost tile can hide in it.  Of one tile alone the bound (cross_backward's, as in test_gpu_cross) is well below the gradients:
a part of a third, and tests without a GPU show that a lost tile, a doubled one and another tile's queries break it."""

import numpy as np
import pytest
import torch

from oracle import cross as oc

TILE = 128
U = 2.0 ** -8


def _expected(q, k, v, do, scale, lens):
    """The gradients of B sequences of one head and one tile of rows, and their bounds (fp32 outputs)."""
    Nk, d = k.shape[2], q.shape[3]
    ref, _, pv, big = oc.cross_attention(q, k, v, scale, lens)
    eps = d * 2.0 ** -24 * big + 2.0 ** -18
    o_tol = (U + 2 * eps + 2 * Nk * 2.0 ** -24) * pv
    want, bound = oc.cross_backward(q, k, v, do, scale, lens, rel=U + 4 * eps + 2.0 ** -10,
                                    o_err=o_tol + U * (np.abs(ref) + o_tol))
    return want, {n: b * (1 + 2.0 ** -6) + 1e-30 for n, b in bound.items()}


def _outside(got, want, bound):
    """The share of elements whose error is past the bound."""
    return float((~(np.abs(got - want) <= bound)).mean())


@pytest.mark.parametrize("Nk,d", [(77, 64), (64, 128), (300, 128), (600, 64), (1, 64)])
def test_a_lost_tile_breaks_the_bound(Nk, d):
    g = torch.Generator().manual_seed(Nk)
    q, do, q2 = (torch.randn(2, 1, TILE, d, generator=g).bfloat16() for _ in range(3))
    k, v = (torch.randn(2, 1, Nk, d, generator=g).bfloat16() for _ in range(2))
    scale, lens = d ** -0.5, [Nk, max(1, Nk - 5)]
    want, bound = _expected(q, k, v, do, scale, lens)
    # what the kernels round: P and dS as bf16
    rounded = {n: np.zeros_like(x) for n, x in want.items()}
    other = np.zeros_like(want["dk"])  # dS^T times another tile's queries
    for b, n in enumerate(lens):
        x, kk, vv, dd = (t[b, 0].double() for t in (q, k[:, :, :n], v[:, :, :n], do))
        p = torch.softmax(scale * x @ kk.T, -1)
        dp = dd @ vv.T
        ds = (p * (dp - (p * dp).sum(-1, keepdim=True))).bfloat16().double()
        p = p.bfloat16().double()
        rounded["dq"][b, 0], rounded["dk"][b, 0, :n] = scale * ds @ kk, scale * ds.T @ x
        rounded["dv"][b, 0, :n], other[b, 0, :n] = p.T @ dd, scale * ds.T @ q2[b, 0].double()
    assert all(_outside(rounded[n], want[n], bound[n]) == 0 for n in want)
    for n in ("dk", "dv"):
        if Nk == 1 and n == "dk":
            continue  # (of a single key there is no gradient)
        assert _outside(np.zeros_like(want[n]), want[n], bound[n]) > 0.5, n
        assert _outside(2 * want[n], want[n], bound[n]) > 0.5, n
    assert Nk == 1 or _outside(other, want["dk"], bound["dk"]) > 0.5


def _tiles(n):
    """Of n tiles: the first ten, the last four and every seventh between."""
    return sorted({*range(min(n, 10)), *range(9, n, 7), *range(max(0, n - 4), n)})


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hq,Hkv,Nq,Nk,d,lens", [
    (2, 8, 4, 7001, 77, 64, None), (2, 8, 4, 7001, 64, 64, [64, 33]), (2, 8, 4, 7001, 128, 64, [128, 97]),
    (2, 8, 4, 7001, 64, 128, None), (2, 8, 4, 7001, 96, 128, [96, 65]), (2, 8, 4, 7001, 128, 128, None),
    (3, 8, 8, 3333, 64, 128, None), (2, 8, 4, 7001, 300, 128, [193, 300]), (2, 8, 4, 7001, 300, 64, None),
    (2, 8, 4, 7001, 600, 64, [599, 300]), (2, 8, 4, 7001, 129, 64, None), (2, 8, 4, 2000, 1500, 128, [1500, 700]),
    (1, 2, 1, 40000, 200, 64, None)])
def test_each_tile_of_queries_reaches_the_gradients(B, Hq, Hkv, Nq, Nk, d, lens):
    from _util import ensure_built
    from exact_attention_06_gb300 import fattn
    from test_gpu_cross import _inputs
    ensure_built()
    q, k, v, do, kl = _inputs(B, Hq, Hkv, Nq, Nk, d, lens)
    scale, rows, heads = d ** -0.5, Hq // Hkv * Nq, B * Hkv
    o, lse = torch.empty_like(q), torch.empty(B, Hq, Nq, device="cuda")
    fattn.fa_cross_fwd(q, k, v, o, lse, scale, kv_lens=kl)
    got = {n: torch.empty(x.shape, device="cuda") for n, x in (("dq", q), ("dk", k), ("dv", v))}
    n_tiles = (rows + TILE - 1) // TILE
    per_head = lambda x, n: x.reshape(heads, 1, n, d)  # noqa: E731
    qh, doh = per_head(q, rows), per_head(do, rows)
    kh, vh = per_head(k, Nk).cpu(), per_head(v, Nk).cpu()
    head_lens = None if lens is None else [n for n in lens for _ in range(Hkv)]
    for t in _tiles(n_tiles):
        # another tile of each head: the blocks of a head are in other rounds
        at = [TILE * ((t + 3 * h) % n_tiles) for h in range(heads)]
        one = torch.zeros_like(doh)
        tile = [torch.zeros(heads, 1, TILE, d, dtype=q.dtype) for _ in range(2)]  # (rows past the last: zeros)
        for h, r in enumerate(at):
            m = min(TILE, rows - r)
            one[h, 0, r:r + m] = doh[h, 0, r:r + m]
            tile[0][h, 0, :m], tile[1][h, 0, :m] = qh[h, 0, r:r + m].cpu(), doh[h, 0, r:r + m].cpu()
        for x in got.values():
            x.fill_(float("nan"))
        fattn.fa_cross_bwd(q, k, v, o, one.view(do.shape), lse, *got.values(), scale, kv_lens=kl)
        assert fattn.fa_get_status() == fattn.FA_OK
        want, bound = _expected(tile[0], kh, vh, tile[1], scale, head_lens)
        for n in ("dk", "dv"):
            x = per_head(got[n], Nk).double().cpu().numpy()
            assert _outside(x, want[n], bound[n]) == 0, f"{n} of tile {t}"
            assert _outside(np.zeros_like(x), want[n], bound[n]) > 0.3, f"{n}: a bound that a lost tile would meet"
        dq = per_head(got["dq"], rows)
        for h, r in enumerate(at):
            m = min(TILE, rows - r)
            x = dq[h:h + 1, :, r:r + m].double().cpu().numpy()
            assert _outside(x, want["dq"][h:h + 1, :, :m], bound["dq"][h:h + 1, :, :m]) == 0, f"dq of tile {t}"
            dq[h, 0, r:r + m] = 0
        assert (dq == 0).all(), f"dq outside tile {t}"  # (NaN where nothing was written)
