"""Every tensor argument of the cross attention and rotary calls, replaced by one of another type, shape, layout
or place: refused by name before anything is launched, and the outputs are left as they were."""

import contextlib

import pytest
import torch

from _util import ensure_built
from exact_attention_06_gb300 import fattn, inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"
B, HQ, HK, NQ, NK, D, PAGE, P = 2, 4, 2, 70, 90, 64, 64, 6


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _bf16(*shape):
    return inputs.normal_bf16(shape, sum(shape), DEV)


def _int(*shape):
    return torch.ones(shape, dtype=torch.int32, device=DEV)


def _plan():
    return fattn.fa_rope_axes_plan(D, (16, 16))


def _calls():
    q, k, lse = (B, HQ, NQ, D), (B, HK, NK, D), torch.empty(B, HQ, NQ, device=DEV)
    kn, pool = (B, HK, NQ, D), (P, HK, PAGE, D)
    return {
        "fa_cross_fwd": (dict(q=_bf16(*q), k=_bf16(*k), v=_bf16(*k), o=_bf16(*q), lse=lse.clone()),
                         dict(kv_lens=_int(B)), dict(scale=0.1), ("o", "lse")),
        "fa_cross_bwd": (dict(q=_bf16(*q), k=_bf16(*k), v=_bf16(*k), o=_bf16(*q), dout=_bf16(*q), lse=lse.clone(),
                              dq=_bf16(*q), dk=_bf16(*k), dv=_bf16(*k)),
                         dict(kv_lens=_int(B)), dict(scale=0.1), ("dq", "dk", "dv")),
        "fa_rope_axes": (dict(q=_bf16(*q), k=_bf16(*kn), pos=_int(2, B, NQ), q_out=_bf16(*q), k_out=_bf16(*kn)), {},
                         dict(plan=_plan()), ("q_out", "k_out")),
        "fa_rope_axes_paged": (dict(q=_bf16(*q), k=_bf16(*kn), v=_bf16(*kn), pos=_int(2, B, NQ), q_out=_bf16(*q),
                                    k_pages=_bf16(*pool), v_pages=_bf16(*pool), block_table=torch.arange(P, dtype=torch.int32, device=DEV).view(B, 3),
                                    seq_lens=_int(B)), dict(new_lens=_int(B)), dict(plan=_plan()),
                               ("q_out", "k_pages", "v_pages")),
    }


def _wrong(t):
    other = torch.float16 if t.dtype == torch.bfloat16 else torch.float64 if t.dtype == torch.float32 else torch.int64
    yield "type", t.to(other)
    yield "shape", torch.cat((t, t[:1]))  # (one sequence, axis, page more; a block table's columns are free)
    yield "dimensions", t.unsqueeze(0)
    yield "place", t.cpu()
    if t.dim() > 1 and t.shape[-1] > 1 and t.shape[-2] > 1:
        yield "layout", t.transpose(-1, -2).contiguous().transpose(-1, -2)
    yield "nothing", "a text"


@pytest.mark.parametrize("name", ["fa_cross_fwd", "fa_cross_bwd", "fa_rope_axes", "fa_rope_axes_paged"])
def test_wrong_tensors_are_refused(name):
    tensors, optional, rest, written = _calls()[name]
    call = getattr(fattn, name)
    before = {n: tensors[n].clone() for n in written}
    for which in list(tensors) + list(optional):
        for what, bad in _wrong({**tensors, **optional}[which]):
            with pytest.raises(fattn.FattnError) as e:
                call(**{**tensors, **optional, which: bad}, **rest)
            assert e.value.status == fattn.FA_ERR_INVALID_ARG, (which, what)
    for stream in ("s", 1.5):
        with pytest.raises(fattn.FattnError):
            call(**tensors, **optional, **rest, stream=stream)
    torch.cuda.synchronize()
    for n in written:
        assert torch.equal(tensors[n], before[n]), n
    call(**tensors, **optional, **rest)  # and the right ones are taken
    assert fattn.fa_get_status() == fattn.FA_OK
    assert any(not torch.equal(tensors[n], before[n]) for n in written)


def test_wrong_plans_workspaces_and_numbers_are_refused():
    tensors, optional, rest, _ = _calls()["fa_rope_axes"]
    for plan in (None, fattn.fa_rope_axes_plan(128, (32, 32)), fattn.fa_rope_axes_plan(D, (32,)), b"plan"):
        with pytest.raises(fattn.FattnError):
            fattn.fa_rope_axes(**tensors, plan=plan)
    with pytest.raises(fattn.FattnError):
        fattn.fa_rope_axes(tensors["q"], None, tensors["pos"], _plan(), k_out=tensors["k_out"])
    for name in ("fa_cross_fwd", "fa_cross_bwd"):
        tensors, optional, rest, _ = _calls()[name]
        call = getattr(fattn, name)
        for bad in (dict(workspace=torch.zeros(4, dtype=torch.float32, device=DEV)),
                    dict(workspace=torch.zeros(4, dtype=torch.uint8)), dict(workspace=5), dict(wait_budget_cycles=-1),
                    dict(scale=0.0), dict(scale=float("nan")), dict(scale="much")):
            with pytest.raises(fattn.FattnError):
                call(**{**tensors, **optional, **rest, **bad})
        if name == "fa_cross_bwd":  # gradients of two types
            with pytest.raises(fattn.FattnError):
                call(**{**tensors, **optional, **rest, "dk": tensors["dk"].float()})


def test_a_scratch_allocation_that_fails_is_torchs_error():
    q, k = (32, 32, 2048, 64), (32, 4, 200, 64)  # 8 MB of scratch
    t = dict(zip(("q", "o", "dout", "dq"), (torch.zeros(q, dtype=torch.bfloat16, device=DEV) for _ in range(4))))
    t |= dict(zip(("k", "v", "dk", "dv"), (torch.zeros(k, dtype=torch.bfloat16, device=DEV) for _ in range(4))))
    t["lse"] = torch.zeros(q[:3], device=DEV)
    assert fattn.fa_cross_bwd_workspace_bytes(32, 32, 4, 2048, 200, 64) >= 8 << 20
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda.set_per_process_memory_fraction(1e-6)
    held = []
    try:
        with contextlib.suppress(torch.cuda.OutOfMemoryError):  # what the allocator still has in its segments
            while len(held) < 100000:
                held.append(torch.empty(2 << 20, dtype=torch.uint8, device=DEV))
        with pytest.raises(torch.cuda.OutOfMemoryError):
            fattn.fa_cross_bwd(**t, scale=0.1)
    finally:
        held.clear()
        torch.cuda.set_per_process_memory_fraction(1.0)
    fattn.fa_cross_bwd(**t, scale=0.1)
    assert fattn.fa_get_status() == fattn.FA_OK
