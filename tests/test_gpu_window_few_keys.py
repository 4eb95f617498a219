"""fa_window_bwd where rows see about 48 keys, the most for which D = rowsum(O dO) comes from P and dP instead of the bf16 O:
by groups of 16 rows, whose first row, which sees the fewest keys, decides.

Values far from zero (64 plus a spread of 2) tell the two forms apart: the rounding of O, 2^-8 of 64, is then as large as the
differences dP - D themselves.  Rows of the first form are checked without any allowance for it; the bounds are otherwise those of
tests/test_gpu_window.py."""

import numpy as np
import pytest
import torch

from _util import ensure_built
from exact_attention_06_gb300 import fattn, inputs
from oracle import window as ow
from test_gpu_window import U, _bounds, _check_fwd, _fwd, _inside

pytestmark = pytest.mark.gpu
DEV = "cuda"
FEW = 48


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _few_rows(N, Nk, W, S):
    first = Nk - N + np.arange(N) // 16 * 16 + 1  # keys up to the first row of each row's group
    return np.minimum(first, W) + np.minimum(S, np.maximum(first - W, 0)) <= FEW


# W + S of 47, 48, 49 throughout, with and without sinks, N no multiple of 16; chunks; rows that see more and more
CASES = [(2, 4, 2, 205, 205, 47, 0), (1, 2, 2, 333, 333, 40, 7), (2, 4, 2, 205, 205, 48, 0), (1, 6, 2, 300, 300, 44, 4),
         (1, 2, 1, 170, 701, 32, 16), (2, 4, 2, 205, 205, 49, 0), (1, 6, 2, 300, 300, 45, 4), (1, 3, 1, 131, 150, 500, 0),
         (1, 2, 2, 100, 133, 64, 1), (1, 2, 1, 77, 77, 4096, 5)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Hq,Hkv,N,Nk,W,S", CASES)
def test_rows_about_the_limit(B, Hq, Hkv, N, Nk, W, S, d):
    q, k = inputs.normal_bf16((B, Hq, N, d), 1, DEV), inputs.normal_bf16((B, Hkv, Nk, d), 2, DEV)
    v = (64 + 2 * inputs.normal_bf16((B, Hkv, Nk, d), 3, DEV).float()).to(torch.bfloat16)
    do, scale = inputs.normal_bf16((B, Hq, N, d), 4, DEV), d ** -0.5
    few = _few_rows(N, Nk, W, S)
    assert few.all() == (min(W, Nk) + S <= FEW) and few.any() == (W + S <= FEW or Nk - N < FEW)
    o, lse = _fwd(q, k, v, scale, W, S)
    bounds = _bounds(q, k, v, scale, W, S)
    _check_fwd(o, lse, q, k, v, scale, W, S, bounds=bounds)
    ref, _, otol, _, eps = bounds
    o_err = otol + U * (np.abs(ref) + otol)
    o_err[:, :, few] = 0
    want, bound = ow.window_backward(q, k, v, do, scale, W, S, rel=U + 4 * eps + 2.0 ** -10, o_err=o_err)
    for t in (torch.float32, torch.bfloat16):
        got = {n: torch.full(x.shape, float("nan"), dtype=t, device=DEV) for n, x in (("dq", q), ("dk", k), ("dv", v))}
        fattn.fa_window_bwd(q, k, v, o, do, lse, *got.values(), scale, W, S)
        assert fattn.fa_get_status() == fattn.FA_OK
        for n, g in got.items():
            tol = bound[n] * (1 + 2.0 ** -6) + 1e-30
            _inside(g, want[n], tol + (U * (np.abs(want[n]) + tol) if t == torch.bfloat16 else 0), f"{n} {t}")


@pytest.mark.parametrize("d", [64, 128])
def test_the_bound_tells_the_forms_apart(d):
    """The definition's dQ with D from an O rounded to bf16 lies outside the bound of rows of few keys."""
    N, W = 205, 48
    q, k = inputs.normal_bf16((1, 1, N, d), 1, "cpu"), inputs.normal_bf16((1, 1, N, d), 2, "cpu")
    v = (64 + 2 * inputs.normal_bf16((1, 1, N, d), 3, "cpu").float()).to(torch.bfloat16)
    do, scale = inputs.normal_bf16((1, 1, N, d), 4, "cpu"), d ** -0.5
    _, _, _, _, eps = _bounds(q, k, v, scale, W, 0)
    want, bound = ow.window_backward(q, k, v, do, scale, W, 0, rel=U + 4 * eps + 2.0 ** -10)
    o = torch.from_numpy(ow.window_attention(q, k, v, scale, W)[0])
    s = torch.where(torch.from_numpy(ow.visible(N, N, W, 0)), scale * q[0, 0].double() @ k[0, 0].double().T, -float("inf"))
    D_off = ((o.bfloat16().double() - o)[0, 0] * do[0, 0].double()).sum(-1, keepdim=True)
    dq = want["dq"][0, 0] - (scale * (torch.softmax(s, -1) * D_off) @ k[0, 0].double()).numpy()
    assert (np.abs(dq - want["dq"][0, 0]) > bound["dq"][0, 0] * (1 + 2.0 ** -6)).any()
