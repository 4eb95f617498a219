"""Cross attention at d = 64 over padded sequences that end inside a key tile, where a block's last items are single query
tiles: the tile whose threads clear V's rows behind the sequence changes from item to item, and may have had no rows
(and seen none of V's stages land) before.  Bounds as in test_gpu_cross."""

import pytest
import torch

from _util import ensure_built
from exact_attention_06_gb300 import fattn
from test_gpu_cross import _check_fwd, _fwd, _inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _lens(kind, B, first, Nk):
    """first: sequences whose blocks fill the SMs once; the rest are the single tiles of the last round."""
    g = torch.Generator().manual_seed(len(kind))
    n = torch.randint(Nk - 80, Nk + 1, (B,), generator=g)
    if kind == "short_last":  # one key tile each
        n[first:] = torch.randint(1, 128, (B - first,), generator=g)
    elif kind == "short":
        n = torch.randint(0, 128, (B,), generator=g)
    elif kind == "mixed":
        n = torch.randint(0, Nk + 1, (B,), generator=g)
    return n.tolist()


@pytest.mark.parametrize("kind", ["long", "short_last", "short", "mixed"])
@pytest.mark.parametrize("rows", [300, 100, 256, 129])
def test_single_tiles_behind_full_rounds(kind, rows):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    blocks, Nk, d = (rows + 255) // 256, 600, 64
    B = (sms + sms // 8) // blocks
    rem = B * blocks - sms
    assert 0 < 2 * rem <= sms and fattn.fa_cross_workspace_bytes(B, 1, 1, rows, Nk, d) == 0  # (the keys are not cut)
    lens = _lens(kind, B, sms // blocks, Nk)
    q, k, v, _, kl = _inputs(B, 1, 1, rows, Nk, d, lens)
    want = None
    for turn in range(6):
        o, lse = _fwd(q, k, v, kl, d ** -0.5)
        if want is None:
            want = o, lse
            _check_fwd(o, lse, q, k, v, d ** -0.5, lens, kind)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1]), turn


@pytest.mark.parametrize("lens", [[1], [100], [127, 0, 129], [599, 3]])
def test_single_tiles_alone(lens):
    """Fewer blocks than half the SMs: every item is a single tile, some of them empty."""
    for rows in (300, 100):
        q, k, v, _, kl = _inputs(len(lens), 2, 2, rows, 600, 64, lens)
        for cut in (False, True):
            o, lse = _fwd(q, k, v, kl, 0.125, cut=cut)
            _check_fwd(o, lse, q, k, v, 0.125, lens, f"rows={rows} cut={cut}")
