"""Calls one behind another without a pause: kernels that are launched before the one ahead has ended must neither read
what it has yet to write nor write what it still reads.  Bit for bit what the same calls give with a wait after each."""

import random
import threading

import pytest
import torch

from _util import ensure_built
from exact_attention_06_gb300 import fattn, inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


class _Chain:
    """Attention layers over a few encoder's states, each taking the last one's output as its queries: turned, attended,
    the gradients turned back and added to the inputs of the next.  What goes on to the next layer is clamped: dV alone
    sums a gradient over G Nq / Nk rows a key, up to 2000 times a layer where a sequence has one key, and as keys of the second attention
    dK and dV meet a dQ of the same size, so that unclamped the scores of the third layer reach 6e13, whose maximum rounds
    by 2^45 2^-24 = 2^21 in the exponent: far past the 2^29 that the library takes."""

    # B, Hq, Hkv, Nq, and the key counts of the layers: each kernel, its cut forms, none, lengths of 0
    SIZES = [(2, 4, 2, 300, (50, 77, 128, 129, 700)), (3, 8, 1, 4, (33, 640, 9000)), (2, 2, 2, 3000, (5, 200, 300)),
             (1, 1, 1, 1, (1, 20000, 64)), (4, 16, 4, 129, (96, 257))]

    def __init__(self, d, seed):
        rng = random.Random(seed)
        self.B, self.Hq, Hkv, self.Nq, keys = self.SIZES[seed % len(self.SIZES)]
        q = (self.B, self.Hq, self.Nq, d)
        self.x = inputs.normal_bf16(q, seed, DEV)
        self.plan = fattn.fa_rope_axes_plan(d, (d // 4, d // 4))
        self.pos = torch.randint(0, 999, (2, self.B, self.Nq), dtype=torch.int32, device=DEV)
        self.layers = []
        for i, n in enumerate(keys):
            lens = [rng.choice((0, 1, n // 2, n)) for _ in range(self.B)] if i % 3 else None
            if i % 3 == 2:
                lens = [0] * self.B
            self.layers.append((inputs.normal_bf16((self.B, Hkv, n, d), i, DEV), inputs.normal_bf16((self.B, Hkv, n, d), 9 + i, DEV),
                                None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV)))
        self.scale = d ** -0.5

    def run(self, steps, after=lambda: None, stream=None):
        """One set of buffers, used again by each layer."""
        on = torch.cuda.stream(stream or torch.cuda.current_stream())
        with on:
            x, r, o, dq, do = (self.x.clone() for _ in range(5))
            lse = torch.empty(x.shape[:3], device=DEV)
            grads = [(torch.empty_like(k), torch.empty_like(v)) for k, v, _ in self.layers]
            kept = []
            for step in range(steps):
                for (k, v, lens), (dk, dv) in zip(self.layers, grads):
                    for call in (
                            lambda: fattn.fa_rope_axes(x, None, self.pos, self.plan, r),
                            lambda: fattn.fa_cross_fwd(r, k, v, o, lse, self.scale, kv_lens=lens),
                            lambda: fattn.fa_cross_bwd(r, k, v, o, do, lse, dq, dk, dv, self.scale, kv_lens=lens),
                            lambda: fattn.fa_rope_axes(dq, None, self.pos, self.plan, inverse=True),
                            lambda: fattn.fa_cross_fwd(dq, dk, dv, do, lse, self.scale, kv_lens=lens),
                            lambda: x.add_(dq).add_(o).clamp_(-4, 4)):
                        call()
                        after()
                    do.add_(x).clamp_(-4, 4)
                    after()
            kept = [x.clone(), r.clone(), o.clone(), dq.clone(), lse.clone(), *(g.clone() for p in grads for g in p)]
        return kept


def _same(a, b):
    return all(torch.equal(x.nan_to_num(), y.nan_to_num()) and torch.equal(x.isnan(), y.isnan()) for x, y in zip(a, b))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("seed", range(5))
def test_a_chain_of_calls_is_the_calls_one_by_one(d, seed):
    chain = _Chain(d, seed)
    want = chain.run(3, after=torch.cuda.synchronize)
    assert torch.isfinite(want[0]).all()
    for _ in range(4):
        got = chain.run(3)
        torch.cuda.synchronize()
        assert _same(want, got)
    assert fattn.fa_get_status() == fattn.FA_OK


def test_threads_on_streams_of_their_own():
    """Four threads at once, each with its chain, its stream and the scratch that its calls allocate."""
    chains = [_Chain(64 if i % 2 else 128, i) for i in range(4)]
    want = [c.run(4, after=torch.cuda.synchronize) for c in chains]
    torch.cuda.synchronize()
    got, wrong, start = [None] * 4, [], threading.Barrier(4)

    def work(i):
        try:
            stream = torch.cuda.Stream()
            start.wait()
            for _ in range(3):
                got[i] = chains[i].run(4, stream=stream)
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            wrong.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong and fattn.fa_get_status() == fattn.FA_OK
    for w, g in zip(want, got):
        assert _same(w, g)


def test_threads_on_one_stream():
    """Their kernels interleave: between a backward's kernels come those of other calls."""
    chains = [_Chain(64 if i % 2 else 128, i) for i in range(4)]
    want = [c.run(4, after=torch.cuda.synchronize) for c in chains]
    got, wrong, start = [None] * 4, [], threading.Barrier(4)
    torch.cuda.synchronize()

    def work(i):
        try:
            start.wait()
            got[i] = chains[i].run(4)
        except Exception as e:  # noqa: BLE001
            wrong.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong and fattn.fa_get_status() == fattn.FA_OK
    for w, g in zip(want, got):
        assert _same(w, g)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq,Nk", [(1, 3), (1, 130), (40, 3), (20, 70), (40, 130)])
def test_more_key_heads_than_a_grid_dimension(Nq, Nk, d):
    """70000 sequences: each gives what it gives in a call of its own hundred."""
    B = 70000
    q = inputs.normal_bf16((100, 1, Nq, d), 1, DEV).repeat(B // 100, 1, 1, 1)
    k, v = (inputs.normal_bf16((100, 1, Nk, d), i, DEV).repeat(B // 100, 1, 1, 1) for i in (2, 3))
    lens = torch.randint(0, Nk + 1, (100,), generator=torch.Generator().manual_seed(4)).to(torch.int32).repeat(B // 100).to(DEV)

    def step(q, k, v, lens):
        o, lse = torch.empty_like(q), torch.empty(q.shape[:3], device=DEV)
        fattn.fa_cross_fwd(q, k, v, o, lse, 0.1, kv_lens=lens)
        g = [torch.empty_like(x) for x in (q, k, v)]
        fattn.fa_cross_bwd(q, k, v, o, q, lse, *g, 0.1, kv_lens=lens)
        assert fattn.fa_get_status() == fattn.FA_OK
        return o, lse, *g
    for i, x in enumerate(step(q, k, v, lens)):
        assert torch.isfinite(x).logical_or(x == -float("inf")).all()
        assert torch.equal(x.view(B // 100, 100, *x.shape[1:]), x[:100].expand(B // 100, *x[:100].shape)), i
