"""Scores up to the stated 2^29: rows that are one key's alone.

Keys are vectors of signs times 2^12, a query is one key's signs times 2^13 (2^12 at d = 128): its score with that key is d 2^25 / 8 = 2^28
(d = 64), with the others smaller by at least 2^20, since no two of the few thousand sign vectors share all but d / 8 of their signs.
So O is that key's v.  p = 2^delta of the one key, |delta| <= 16 from the maximum's rounding, is rounded to bf16 in the
product but not in l: off by 2^-8 of v, as is bf16 O.  lse is within 2^-22 of its value."""

import numpy as np
import pytest
import torch

from _util import ensure_built
from exact_attention_06_gb300 import fattn

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _inputs(H, Nq, Nk, d):
    g = torch.Generator().manual_seed(Nq + Nk + d)
    signs = torch.randint(0, 2, (1, H, Nk, d), generator=g) * 2.0 - 1
    at = torch.randint(0, Nk, (1, H, Nq), generator=g)
    v = torch.randn(1, H, Nk, d, generator=g).bfloat16()
    pick = lambda x: x.gather(2, at.unsqueeze(-1).expand(-1, -1, -1, d))  # noqa: E731
    q = (pick(signs) * 2.0 ** (13 if d == 64 else 12)).bfloat16()
    other = (pick(signs) @ signs.mT).scatter(3, at.unsqueeze(-1), -d)
    assert other.max() <= d - d // 4  # (the gap)
    score = d * 2.0 ** (25 if d == 64 else 24) * 0.125
    return q.to(DEV), (signs * 2.0 ** 12).bfloat16().to(DEV), v.to(DEV), pick(v), score


def _check(o, lse, want, score):
    o, want = o.double().cpu().reshape(want.shape), want.double()
    assert ((o - want).abs() <= 2 * 2.0 ** -8 * want.abs()).all()
    assert np.allclose(lse.double().cpu().numpy(), score, rtol=2.0 ** -22, atol=0)
    assert fattn.fa_get_status() == fattn.FA_OK


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq,Nk", [(1, 50), (1, 700), (2, 9000), (20, 3000), (300, 60), (300, 90), (300, 128), (300, 700)])
def test_cross_attention(Nq, Nk, d):
    q, k, v, want, score = _inputs(2, Nq, Nk, d)
    for cut in (False, True):
        o, lse = torch.empty_like(q), torch.empty(q.shape[:3], device=DEV)
        ws = None if cut else torch.empty(0, dtype=torch.uint8, device=DEV)
        fattn.fa_cross_fwd(q, k, v, o, lse, 0.125, workspace=ws)
        _check(o, lse, want, score)


@pytest.mark.parametrize("d", [64, 128])
def test_prefill_and_decode(d):
    q, k, v, want, score = _inputs(2, 640, 640, d)
    o, lse = torch.empty_like(q), torch.empty(q.shape[:3], device=DEV)
    fattn.fa_fwd(q, k, v, o, lse, 0.125)
    _check(o, lse, want, score)
    q, k, v, want, score = _inputs(2, 1, 3000, d)
    q = q[:, :, 0].contiguous()
    for splits in (1, 5):
        o, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)
        ws = torch.empty(fattn.fa_decode_workspace_bytes(1, 2, 3000, d, 128, splits), dtype=torch.uint8, device=DEV)
        fattn.fa_decode_splitkv(q, k, v, o, lse, 0.125, ws, 128, splits)
        _check(o, lse.unsqueeze(-1), want, score)
