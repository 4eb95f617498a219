"""Sliding windows at scores up to the stated 2^29: rows that are one visible key's alone, as in tests/test_gpu_score_range.py
(keys of signs, a query its key's signs), with that key in the window, among the sinks or the query's own; the other visible keys'
scores differ from it by at least 2^20, and hidden keys are larger: twice the query's own signs."""

import numpy as np
import pytest
import torch

from _util import ensure_built
from exact_attention_06_gb300 import fattn
from oracle import window as ow
from test_gpu_score_range import _check

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _inputs(H, N, Nk, d, W, S):
    """q, k, v, the rows' own v, their score.  A key hidden from every query holds signs of some query's key, twice as large."""
    g = torch.Generator().manual_seed(N + Nk + d + W)
    signs = torch.randint(0, 2, (1, H, Nk, d), generator=g) * 2.0 - 1
    see = torch.from_numpy(ow.visible(N, Nk, W, S))
    at = torch.multinomial(see.double(), H, replacement=True, generator=g).T[None]  # [1, H, N]: one of the row's visible keys
    v = torch.randn(1, H, Nk, d, generator=g).bfloat16()
    pick = lambda x: x.gather(2, at.unsqueeze(-1).expand(-1, -1, -1, d))  # noqa: E731
    other = (pick(signs) @ signs.mT).scatter(3, at.unsqueeze(-1), -d)
    assert other.max() <= d - d // 4
    q, want, k = (pick(signs) * 2.0 ** (13 if d == 64 else 12)).bfloat16(), pick(v), (signs * 2.0 ** 12).bfloat16()
    hidden = ~see.any(0)
    if hidden.any():
        k[:, :, hidden] = (pick(signs)[:, :, :1] * 2.0 ** 13).bfloat16()
    return q.to(DEV), k.to(DEV), v.to(DEV), want, d * 2.0 ** (25 if d == 64 else 24) * 0.125


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,Nk,W,S", [(640, 640, 200, 4), (640, 640, 640, 0), (300, 900, 130, 100), (77, 1500, 700, 0),
                                      (513, 513, 1, 33)])
def test_forward(N, Nk, W, S, d):
    q, k, v, want, score = _inputs(4, N, Nk, d, W, S)
    o, lse = torch.empty_like(q), torch.empty(q.shape[:3], device=DEV)
    fattn.fa_window_fwd(q, k, v, o, lse, 0.125, W, S)
    _check(o, lse, want, score)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("L,W,S", [(50, 50, 0), (700, 300, 70), (9000, 8000, 5), (3000, 64, 128)])
def test_one_token(L, W, S, d):
    H, ps = 3, 64
    q, k, v, want, score = _inputs(H, 1, L, d, W, S)
    pages = -(-L // ps)
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(1, pages).to(DEV)
    kp, vp = (torch.zeros(pages, H, ps, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    for i in range(pages):
        rows = slice(i * ps, min((i + 1) * ps, L))
        n = rows.stop - rows.start
        kp[table[0, i], :, :n], vp[table[0, i], :, :n] = k[0, :, rows], v[0, :, rows]
    o, lse = torch.empty(1, H, d, dtype=torch.bfloat16, device=DEV), torch.empty(1, H, device=DEV)
    lens = torch.tensor([L], dtype=torch.int32, device=DEV)
    fattn.fa_window_decode_paged(q[:, :, 0].contiguous(), kp, vp, table, lens, o, lse, 0.125, L, W, S)
    _check(o, lse, want[:, :, 0], score)
