"""The operators as a model uses them together: rotary positions, self attention, cross attention; prompt,
decode steps through the paged cache (eagerly and replayed from a CUDA graph), and a training step."""

import numpy as np
import pytest
import torch

import oracle
from _util import assert_parity, ensure_built
from exact_attention_06_gb300 import fattn, inputs
from oracle import cross as oc

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _rand(shape, seed):
    return inputs.normal_bf16(shape, seed, DEV)


@pytest.mark.parametrize("graph", [False, True])
def test_decode_steps_through_the_paged_cache(graph):
    """Steps of one token: fa_rope_axes_paged, fa_decode_paged, fa_cross_fwd, against the oracles over the
    whole history; with ``graph``, captured once and replayed with new tokens and lengths."""
    ensure_built()
    B, H, d, ps, mp, Nk = 3, 4, 128, 64, 4, 333
    scale = d ** -0.5
    plan = fattn.fa_rope_axes_plan(d, (16, 24, 24))
    axis, rates = oc.rope_rates(d, (16, 24, 24))
    kp, vp = (torch.full((B * mp, H, ps, d), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    table = torch.randperm(B * mp, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(B, mp).to(DEV)
    enc_k, enc_v = _rand((B, 2, Nk, d), 2), _rand((B, 2, Nk, d), 3)
    enc_len = torch.tensor([333, 200, 0], dtype=torch.int32, device=DEV)
    before = torch.tensor([62, 0, 126], dtype=torch.int32, device=DEV)
    q, k, v = (torch.empty(B, H, 1, d, dtype=torch.bfloat16, device=DEV) for _ in range(3))
    pos = torch.empty(3, B, 1, dtype=torch.int32, device=DEV)
    qr, o, oc_ = torch.empty_like(q), torch.empty(B, H, d, device=DEV), torch.empty(B, H, 1, d, device=DEV)
    lse, lse_c = torch.empty(B, H, device=DEV), torch.empty(B, H, 1, device=DEV)

    def step():
        fattn.fa_rope_axes_paged(q, k, v, pos, plan, qr, kp, vp, table, before)
        fattn.fa_decode_paged(qr.view(B, H, d), kp, vp, table, before + 1, o, lse, scale, mp * ps)
        fattn.fa_cross_fwd(qr, enc_k, enc_v, oc_, lse_c, scale, kv_lens=enc_len)
        before.add_(1)

    # the history, written as a prompt chunk
    hist = before.tolist()
    T = max(hist)
    hk, hv, hpos = _rand((B, H, T, d), 4), _rand((B, H, T, d), 5), torch.arange(T, device=DEV, dtype=torch.int32)
    hpos = hpos.expand(3, B, T).contiguous()
    zero = torch.zeros_like(before)
    fattn.fa_rope_axes_paged(hk, hk, hv, hpos, plan, torch.empty_like(hk), kp, vp, table, zero, before.clone())
    turned = torch.empty_like(hk)
    fattn.fa_rope_axes(hk, None, hpos, plan, turned)
    keys = [[turned[b, :, :n].cpu(), hv[b, :, :n].cpu()] for b, n in enumerate(hist)]
    if graph:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):  # outside the capture once, and undone
            k.zero_(), v.zero_(), q.zero_(), pos.zero_()
            step()
            before.sub_(1)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
    for t in range(4):
        for i, x in enumerate((q, k, v)):
            x.copy_(_rand(x.shape, 10 + 3 * t + i))
        pos.copy_(torch.stack([before + 7, before // 3, before % 5]).unsqueeze(-1))
        g.replay() if graph else step()
        assert fattn.fa_get_status() == fattn.FA_OK
        kr, _ = oc.rope(k, pos.cpu(), axis, rates)
        kr = torch.from_numpy(kr).to(torch.bfloat16)
        for b in range(B):  # within a bf16 step of the oracle's rotation, read back from the cache
            n = keys[b][0].shape[1]
            at = kp[table[b, n // ps].long(), :, n % ps].cpu()
            assert (at.float() - kr[b, :, 0].float()).abs().max() <= 2.0 ** -6 * kr[b].abs().max().float()
            keys[b] = [torch.cat((keys[b][0], at[:, None]), 1), torch.cat((keys[b][1], v[b].cpu()), 1)]
            ref, lref = oracle.decode(qr[b:b + 1, :, 0].cpu(), keys[b][0][None], keys[b][1][None], scale)
            assert_parity(o[b], lse[b], ref, lref, f"self attention, step {t}, sequence {b}")
        ref, lref, _, _ = oc.cross_attention(qr, enc_k, enc_v, scale, enc_len.tolist())
        assert_parity(oc_, lse_c, ref, lref, f"cross attention, step {t}")


def test_a_training_step_of_a_layer():
    """x -> rotary -> causal self attention -> cross attention, and back to dq, dk, dv: each gradient
    against the fp64 chain, 2 % of the largest and 1 % of the mean magnitude as for fa_bwd."""
    ensure_built()
    B, H, N, Nk, d = 1, 3, 200, 140, 64
    scale = d ** -0.5
    plan = fattn.fa_rope_axes_plan(d, (16, 16), interleaved=True)
    axis, rates = oc.rope_rates(d, (16, 16))
    q, k, v, do = (_rand((B, H, N, d), 20 + i) for i in range(4))
    ek, ev = _rand((B, H, Nk, d), 30), _rand((B, H, Nk, d), 31)
    lens = [120]
    kl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    pos = torch.randint(0, 60, (2, B, N), generator=torch.Generator().manual_seed(3), dtype=torch.int32).to(DEV)
    qr, kr, o1, o2 = (torch.empty_like(q) for _ in range(4))
    l1, l2 = torch.empty(B, H, N, device=DEV), torch.empty(B, H, N, device=DEV)
    fattn.fa_rope_axes(q, k, pos, plan, qr, kr)
    fattn.fa_fwd(qr, kr, v, o1, l1, scale, True)
    fattn.fa_cross_fwd(o1, ek, ev, o2, l2, scale, kv_lens=kl)
    d1, dek, dev, dq, dk, dv = (torch.empty_like(x) for x in (q, ek, ev, q, k, v))
    fattn.fa_cross_bwd(o1, ek, ev, o2, do, l2, d1, dek, dev, scale, kv_lens=kl)
    fattn.fa_bwd(qr, kr, v, o1, d1, l1, dq, dk, dv, scale, True)
    fattn.fa_rope_axes(dq, dk, pos, plan, inverse=True)
    assert fattn.fa_get_status() == fattn.FA_OK
    # fp64 chain on what each operator really got
    want, _ = oc.cross_backward(o1, ek, ev, do, scale, lens)
    gq, gk, gv = oracle.attention_backward(qr.cpu(), kr.cpu(), v.cpu(), want["dq"], scale, True)
    gq, gk = (oc.rope(g, pos.cpu(), axis, rates, True, inverse=True)[0] for g in (gq, gk))
    for name, got, ref in (("dek", dek, want["dk"]), ("dev", dev, want["dv"]), ("dq", dq, gq), ("dk", dk, gk),
                           ("dv", dv, gv)):
        e = np.abs(got.cpu().double().numpy() - ref)
        assert e.max() <= 2e-2 * np.abs(ref).max() and e.mean() <= 1e-2 * np.abs(ref).mean(), name


def test_a_training_step_captured_and_replayed():
    """Forward and backward (with keys and queries cut into ranges) captured twice, in graphs with workspaces of
    their own, and replayed in turn on new values and lengths: bitwise what eager calls give."""
    ensure_built()
    B, Hq, Hkv, Nq, Nk, d = 2, 4, 2, 700, 900, 128
    scale = d ** -0.5
    size = (B, Hq, Hkv, Nq, Nk, d)
    plan = fattn.fa_rope_axes_plan(d, (16, 24, 24), cyclic=True)
    kl = torch.tensor([900, 900], dtype=torch.int32, device=DEV)
    pos = torch.randint(0, 500, (3, B, Nq), dtype=torch.int32, device=DEV)
    q, do = _rand((B, Hq, Nq, d), 1), _rand((B, Hq, Nq, d), 2)
    k, v = _rand((B, Hkv, Nk, d), 3), _rand((B, Hkv, Nk, d), 4)
    assert fattn.fa_cross_bwd_workspace_bytes(*size) > B * Hq * Nq * 4 + 256  # ranges of queries or keys

    def buffers():
        return [torch.empty_like(q), torch.empty_like(q), torch.empty(B, Hq, Nq, device=DEV), torch.empty_like(q),
                torch.empty_like(k), torch.empty_like(v),
                torch.empty(max(256, fattn.fa_cross_workspace_bytes(*size)), dtype=torch.uint8, device=DEV),
                torch.empty(fattn.fa_cross_bwd_workspace_bytes(*size), dtype=torch.uint8, device=DEV)]

    def step(b, stream=None):
        qr, o, lse, dq, dk, dv, w1, w2 = b
        fattn.fa_rope_axes(q, None, pos, plan, qr, stream=stream)
        fattn.fa_cross_fwd(qr, k, v, o, lse, scale, kv_lens=kl, workspace=w1, stream=stream)
        fattn.fa_cross_bwd(qr, k, v, o, do, lse, dq, dk, dv, scale, kv_lens=kl, workspace=w2, stream=stream)
        fattn.fa_rope_axes(dq, None, pos, plan, inverse=True, stream=stream)

    one, two, eager = buffers(), buffers(), buffers()
    step(eager)
    torch.cuda.synchronize()
    graphs = []
    for b in (one, two):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(b)
        graphs.append(g)
    for t, lens in enumerate(([900, 333], [0, 128], [901, 1])):
        for i, x in enumerate((q, k, v, do)):
            x.copy_(_rand(x.shape, 20 + 4 * t + i))
        kl.copy_(torch.tensor(lens, dtype=torch.int32))
        for b in (one, two, eager):
            for x in b[:6]:
                x.fill_(float("nan"))
        graphs[0].replay()
        graphs[1].replay()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        step(eager, stream=side.cuda_stream)  # a raw handle
        torch.cuda.synchronize()
        assert fattn.fa_get_status() == fattn.FA_OK
        for a, b, c in zip(one[:6], two[:6], eager[:6]):
            assert torch.equal(a, c) and torch.equal(b, c) and torch.isfinite(a).logical_or(a == -float("inf")).all()
