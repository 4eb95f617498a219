"""Waits that run out in the persistent forward kernels while their blocks have several items to go: the call ends, reports
FA_ERR_TIMEOUT (or has finished within the budget, with the right outputs), and the next call's outputs are what they were.

Budgets from one cycle (nothing arrives) to about the length of a call, so that waits run out at a block's first item, between
its items and at its last, and in only some of a tile's warps."""

import pytest
import torch

from _util import ensure_built
from exact_attention_06_gb300 import fattn, inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"
BUDGETS = (1, 300, 1000, 2000, 4000, 8000, 16000, 50000)


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _outputs(q, o_fp32):
    return (torch.full(q.shape, float("nan"), dtype=torch.float32 if o_fp32 else torch.bfloat16, device=DEV),
            torch.full(q.shape[:3], float("nan"), device=DEV))


def _check(call, q, o_fp32, items):
    assert items > 2 * torch.cuda.get_device_properties(0).multi_processor_count  # (blocks of several items)
    want = _outputs(q, o_fp32)
    call(*want, 0)
    assert fattn.fa_get_status() == fattn.FA_OK
    for budget in BUDGETS:
        for _ in range(3):
            got = _outputs(q, o_fp32)
            call(*got, budget)
            try:
                fattn.fa_get_status()
                assert budget > 1 and all(torch.equal(a, b) for a, b in zip(got, want)), f"budget {budget}"
            except fattn.FattnError as e:
                assert e.status == fattn.FA_ERR_TIMEOUT, f"budget {budget}"
        got = _outputs(q, o_fp32)
        call(*got, 0)
        assert fattn.fa_get_status() == fattn.FA_OK
        assert all(torch.equal(a, b) for a, b in zip(got, want)), f"after a budget of {budget}"


@pytest.mark.parametrize("o_fp32", [False, True])
@pytest.mark.parametrize("d,Hq,Hkv", [(64, 16, 16), (64, 16, 4), (128, 16, 16), (128, 16, 4)])
def test_window(d, Hq, Hkv, o_fp32):
    """Tiles of one head and of the heads that share a key head (d = 128: with half of O staged)."""
    B, N, W, S = 4, 2100, 256, 4
    q = inputs.normal_bf16((B, Hq, N, d), 1, DEV)
    k, v = inputs.normal_bf16((B, Hkv, N, d), 2, DEV), inputs.normal_bf16((B, Hkv, N, d), 3, DEV)
    _check(lambda o, lse, budget: fattn.fa_window_fwd(q, k, v, o, lse, 0.1, W, S, wait_budget_cycles=budget), q, o_fp32,
           B * Hq * N // 256)


@pytest.mark.parametrize("o_fp32", [False, True])
def test_prefill(o_fp32):
    B, H, N, d = 4, 16, 2100, 64
    q, k, v = (inputs.normal_bf16((B, H, N, d), s, DEV) for s in (1, 2, 3))
    _check(lambda o, lse, budget: fattn.fa_fwd_ex(q, k, v, o, lse, 0.1, False, wait_budget_cycles=budget), q, o_fp32,
           B * H * N // 256)


@pytest.mark.parametrize("o_fp32", [False, True])
def test_cross(o_fp32):
    """Sequences of their own lengths, one of them empty, whose last key tiles are cleared behind them."""
    B, Hq, Hkv, Nq, Nk, d = 4, 16, 8, 2100, 700, 64
    q = inputs.normal_bf16((B, Hq, Nq, d), 1, DEV)
    k, v = inputs.normal_bf16((B, Hkv, Nk, d), 2, DEV), inputs.normal_bf16((B, Hkv, Nk, d), 3, DEV)
    v[1, :, 333:] = float("nan")
    kv_lens = torch.tensor([Nk, 333, 0, 650], dtype=torch.int32, device=DEV)
    _check(lambda o, lse, budget: fattn.fa_cross_fwd(q, k, v, o, lse, 0.1, kv_lens, wait_budget_cycles=budget), q, o_fp32,
           B * Hq * Nq // 256)


@pytest.mark.parametrize("grads", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,B,H,N,W,S", [(64, 4, 16, 2100, 256, 4), (128, 2, 32, 4100, 128, 17), (64, 2, 96, 200, 30, 3)])
def test_window_backward(d, B, H, N, W, S, grads):
    """Blocks of several key tiles and several query tiles, of one head and of all heads' list."""
    q, k, v, do = (inputs.normal_bf16((B, H, N, d), s, DEV) for s in (1, 2, 3, 4))
    o, lse = torch.empty_like(q), torch.empty(B, H, N, device=DEV)
    fattn.fa_window_fwd(q, k, v, o, lse, 0.1, W, S)

    def step(budget):
        g = [torch.full(q.shape, float("nan"), dtype=grads, device=DEV) for _ in range(3)]
        fattn.fa_window_bwd(q, k, v, o, do, lse, *g, 0.1, W, S, wait_budget_cycles=budget)
        return g
    want = step(0)
    assert fattn.fa_get_status() == fattn.FA_OK
    for budget in BUDGETS:
        for _ in range(2):
            got = step(budget)
            try:
                fattn.fa_get_status()
                assert budget > 1 and all(torch.equal(a, b) for a, b in zip(got, want)), f"budget {budget}"
            except fattn.FattnError as e:
                assert e.status == fattn.FA_ERR_TIMEOUT, f"budget {budget}"
        got = step(0)
        assert fattn.fa_get_status() == fattn.FA_OK
        assert all(torch.equal(a, b) for a, b in zip(got, want)), f"after a budget of {budget}"
