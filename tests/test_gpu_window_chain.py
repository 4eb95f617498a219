"""The calls of a layer with a sliding window together, as a serving loop and a training step make them: pages for the new
tokens, their q and k normed and turned into the cache, one token's attention over it; and norms, attention and the gradients
of both.  Every stage is compared with the fp64 definition on the values that reached it (the bounds are those of
the stages' own tests), and captured steps with the calls one by one."""

import os
import re
import threading

import numpy as np
import pytest
import torch

from _util import ensure_built
from exact_attention_06_gb300 import fattn, inputs
from oracle import window as ow
from test_gpu_window_decode import _check as check_decode
from test_gpu_window import _bounds, _check_fwd, _inside
from test_gpu_norm_rope import _check as check_norm
from test_gpu_norm_rope import _check_bwd as check_norm_bwd
from oracle import cross as oc

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Server:
    """A layer's cache and one step over it: pages, append, attention of the last token."""

    def __init__(self, B, Hq, Hkv, d, ps, max_pages, num_pages, W, S, seed=0):
        self.B, self.Hq, self.Hkv, self.d, self.ps, self.W, self.S = B, Hq, Hkv, d, ps, W, S
        self.L = max_pages * ps
        self.plan = fattn.fa_rope_axes_plan(d, (d // 2,))
        self.wq, self.wk = (1 + 0.2 * inputs.normal_bf16((d,), seed + i, DEV).float() for i in (1, 2))
        self.table = torch.full((B, max_pages), -1, dtype=torch.int32, device=DEV)
        self.lens, self.granted = torch.zeros(B, dtype=torch.int32, device=DEV), torch.empty(B, dtype=torch.int32, device=DEV)
        self.stack, self.n_free = torch.randperm(num_pages).to(torch.int32).to(DEV), _ints([num_pages])
        # (what no token has been written to may be anything)
        self.kp = torch.full((num_pages, Hkv, ps, d), float("nan"), dtype=torch.bfloat16, device=DEV)
        self.vp = torch.full_like(self.kp, float("inf"))

    def buffers(self, N):
        return dict(new=torch.zeros(self.B, dtype=torch.int32, device=DEV),
                    q=torch.zeros(self.B, self.Hq, N, self.d, dtype=torch.bfloat16, device=DEV),
                    k=torch.zeros(self.B, self.Hkv, N, self.d, dtype=torch.bfloat16, device=DEV),
                    v=torch.zeros(self.B, self.Hkv, N, self.d, dtype=torch.bfloat16, device=DEV),
                    pos=torch.zeros(1, self.B, N, dtype=torch.int32, device=DEV),
                    slots=torch.empty(self.B, N, dtype=torch.int64, device=DEV),
                    q_out=torch.zeros(self.B, self.Hq, N, self.d, dtype=torch.bfloat16, device=DEV),
                    o=torch.empty(self.B, self.Hq, self.d, dtype=torch.bfloat16, device=DEV),
                    lse=torch.empty(self.B, self.Hq, device=DEV))

    def step(self, x, attend=True):
        fattn.fa_pages_extend(self.table, self.lens, x["new"], self.stack, self.n_free, self.granted, x["slots"], self.ps)
        fattn.fa_norm_rope_axes_paged(x["q"], x["k"], x["v"], self.wq, self.wk, x["pos"], self.plan, x["q_out"], self.kp,
                                      self.vp, x["slots"], self.granted)
        if attend:
            fattn.fa_window_decode_paged(x["q_out"][:, :, 0].contiguous(), self.kp, self.vp, self.table, self.lens, x["o"],
                                         x["lse"], self.d ** -0.5, self.L, self.W, self.S)

    def give_back(self, n):
        fattn.fa_pages_extend(self.table, self.lens, _ints(n), self.stack, self.n_free, self.granted, None, self.ps)


class Tokens:
    """Each sequence's tokens (q, k, v before the norm) and its keys and values as the cache should hold them."""

    def __init__(self, s, seed):
        self.s, self.seed, self.k, self.v = s, seed, [None] * s.B, [None] * s.B

    def fill(self, x, new, N):
        s = self.s
        self.seed += 10
        x["new"].copy_(_ints(new))
        for i, name in enumerate("qkv"):
            x[name].copy_(inputs.normal_bf16(tuple(x[name].shape), self.seed + i, DEV))
        n0 = [0 if self.k[b] is None else self.k[b].shape[1] for b in range(s.B)]
        x["pos"].copy_((_ints(n0)[:, None] + torch.arange(N, device=DEV))[None])
        want_q, want_k = torch.empty_like(x["q"]), torch.empty_like(x["k"])
        fattn.fa_norm_rope_axes(x["q"], x["k"], s.wq, s.wk, x["pos"], s.plan, want_q, want_k)
        for b, n in enumerate(new):
            if n > 0:
                k, v = want_k[b, :, :n].clone(), x["v"][b, :, :n].clone()
                self.k[b] = k if self.k[b] is None else torch.cat([self.k[b], k], 1)
                self.v[b] = v if self.v[b] is None else torch.cat([self.v[b], v], 1)
        return want_q

    def cut(self, b, n):
        self.k[b], self.v[b] = (None, None) if n == 0 else (self.k[b][:, :n], self.v[b][:, :n])

    def lens(self):
        return [0 if k is None else k.shape[1] for k in self.k]

    def check(self, x, what):
        s, lens = self.s, self.lens()
        L = max(max(lens), 1)
        k, v = (torch.zeros(s.B, s.Hkv, L, s.d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        for b, n in enumerate(lens):
            if n:
                k[b, :, :n], v[b, :, :n] = self.k[b], self.v[b]
        assert s.lens.tolist() == lens, what
        check_decode(x["o"], x["lse"], x["q_out"][:, :, 0], k, v, lens, s.d ** -0.5, L, s.W, s.S, what)


@pytest.mark.parametrize("d,ps,W,S", [(128, 64, 100, 4), (64, 128, 1000, 0), (128, 64, 64, 65), (64, 64, 3, 128)])
def test_a_serving_loop(d, ps, W, S):
    B, N = 5, 150
    s = Server(B, 8, 2, d, ps, 8, 30, W, S)
    t, x, one = Tokens(s, 100), s.buffers(N), s.buffers(1)
    want = t.fill(x, [150, 3, 64, 0, 129], N)
    s.step(x, attend=False)
    for b, n in enumerate([150, 3, 64, 0, 129]):
        assert torch.equal(x["q_out"][b, :, :n], want[b, :, :n]) and (x["q_out"][b, :, n:] == 0).all()
    for turn in range(3):
        t.fill(one, [1, 1, 1, 1 if turn else 0, 1], 1)
        s.step(one)
        t.check(one, f"token {turn}")
    # drafts: three tokens each, two taken back; the rows they leave hold what they held
    drafts = s.buffers(3)
    t.fill(drafts, [3] * B, 3)
    s.step(drafts, attend=False)
    s.give_back([-2] * B)
    for b in range(B):
        t.cut(b, t.lens()[b] - 2)
    t.fill(one, [1] * B, 1)
    s.step(one)
    t.check(one, "after drafts")
    # requests 0 and 4 end, their pages go to longer prompts in their place
    lens = t.lens()
    s.give_back([-lens[0], 0, 0, 0, -lens[4]])
    t.cut(0, 0)
    t.cut(4, 0)
    t.fill(x, [140, 0, 0, 0, 150], N)
    s.step(x, attend=False)
    for turn in range(2):
        t.fill(one, [1] * B, 1)
        s.step(one)
        t.check(one, f"new requests, token {turn}")
    held = sum(-(-n // ps) for n in t.lens())
    assert int(s.n_free) == 30 - held and int((s.table >= 0).sum()) == held


def test_a_pool_that_runs_out():
    """A sequence that is refused its page keeps its length, its q is left as it was, no cache row changes for it, and it goes
    on when another sequence has given pages back."""
    B, W, S = 3, 50, 2
    s = Server(B, 4, 1, 64, 64, 4, 4, W, S)
    t, x, one = Tokens(s, 31), s.buffers(128), s.buffers(1)
    t.fill(x, [64, 128, 64], 128)
    s.step(x, attend=False)
    assert int(s.n_free) == 0
    one["new"].fill_(1)
    kp, vp = s.kp.clone(), s.vp.clone()
    one["q"].copy_(inputs.normal_bf16(tuple(one["q"].shape), 5, DEV))
    one["q_out"].fill_(7)
    s.step(one)
    assert s.granted.tolist() == [0, 0, 0] and s.lens.tolist() == [64, 128, 64]
    assert (one["q_out"] == 7).all() and (one["slots"] == -1).all()
    for a, b in ((s.kp, kp), (s.vp, vp)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    s.give_back([0, -128, 0])
    t.cut(1, 0)
    t.fill(one, [1, 1, 0], 1)
    s.step(one)
    assert s.granted.tolist() == [1, 1, 0]
    t.check(one, "after pages came back")


def test_a_captured_decode_step():
    """One graph of a step, replayed while sequences cross pages; its scratch is the graph's own."""
    B, W, S = 4, 90, 5
    s = Server(B, 8, 2, 128, 64, 6, 24, W, S)
    t, x, one = Tokens(s, 7), s.buffers(70), s.buffers(1)
    t.fill(x, [60, 64, 1, 70], 70)
    s.step(x, attend=False)
    saved = [y.clone() for y in (s.table, s.lens, s.stack, s.n_free)]
    one["new"].fill_(1)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        s.step(one)
    for a, b in zip((s.table, s.lens, s.stack, s.n_free), saved):
        assert torch.equal(a, b)  # (a capture runs nothing)
    for turn in range(8):
        t.fill(one, [1] * B, 1)
        graph.replay()
        torch.cuda.synchronize()
        t.check(one, f"replay {turn}")
    assert fattn.fa_get_status() == fattn.FA_OK


def _train(x, out, W, S, scale, plan):
    q, k, v, wq, wk, pos, do = x
    qn, kn, o, lse, dqn, dkn, dv, dq, dk, dwq, dwk = out
    fattn.fa_norm_rope_axes(q, k, wq, wk, pos, plan, qn, kn)
    fattn.fa_window_fwd(qn, kn, v, o, lse, scale, W, S)
    fattn.fa_window_bwd(qn, kn, v, o, do, lse, dqn, dkn, dv, scale, W, S)
    fattn.fa_norm_rope_axes_bwd(q, k, wq, wk, pos, plan, dqn, dkn, dq, dk, dwq, dwk)


def _train_state(B, Hq, Hkv, N, d, seed):
    q, k, v = (inputs.normal_bf16((B, H, N, d), seed + i, DEV) for i, H in enumerate((Hq, Hkv, Hkv)))
    wq, wk = (1 + 0.2 * inputs.normal_bf16((d,), seed + 5 + i, DEV).float() for i in range(2))
    pos = torch.arange(N, dtype=torch.int32, device=DEV).expand(1, B, N).contiguous()
    x = [q, k, v, wq, wk, pos, inputs.normal_bf16((B, Hq, N, d), seed + 8, DEV)]
    new = lambda like, **kw: torch.full(like.shape, float("nan"), dtype=kw.get("dtype", like.dtype), device=DEV)  # noqa: E731
    out = [new(q), new(k), new(q), torch.empty(B, Hq, N, device=DEV), new(q), new(k), new(v), new(q), new(k), new(wq), new(wk)]
    return x, out


@pytest.mark.parametrize("B,Hq,Hkv,N,d,W,S", [(2, 4, 2, 333, 128, 90, 4), (1, 6, 2, 500, 64, 257, 33), (3, 2, 2, 40, 64, 7, 0)])
def test_a_training_step(B, Hq, Hkv, N, d, W, S):
    plan, scale = fattn.fa_rope_axes_plan(d, (d // 2,)), d ** -0.5
    x, out = _train_state(B, Hq, Hkv, N, d, 3)
    _train(x, out, W, S, scale, plan)
    assert fattn.fa_get_status() == fattn.FA_OK
    q, k, v, wq, wk, pos, do = x
    qn, kn, o, lse, dqn, dkn, dv, dq, dk, dwq, dwk = out
    axis, rates = oc.rope_rates(d, (d // 2,))
    p = pos.cpu()
    check_norm(qn, q, wq, p, axis, rates, False, 1e-6, "q")
    check_norm(kn, k, wk, p, axis, rates, False, 1e-6, "k")
    bounds = _bounds(qn, kn, v, scale, W, S)
    _check_fwd(o, lse, qn, kn, v, scale, W, S, bounds=bounds)
    ref, _, otol, _, eps = bounds
    want, bound = ow.window_backward(qn, kn, v, do, scale, W, S, rel=U + 4 * eps + 2.0 ** -10,
                                     o_err=otol + U * (np.abs(ref) + otol))
    for n, g in (("dq", dqn), ("dk", dkn), ("dv", dv)):
        tol = bound[n] * (1 + 2.0 ** -6) + 1e-30
        _inside(g, want[n], tol + U * (np.abs(want[n]) + tol), n)
    check_norm_bwd(dq, dwq, q, wq, dqn, p, axis, rates, False, 1e-6, "q")
    check_norm_bwd(dk, dwk, k, wk, dkn, p, axis, rates, False, 1e-6, "k")


def test_two_captured_training_steps_at_once():
    """Two graphs of two streams, replayed together with each other's inputs in turn, against the calls one by one; an eager
    step of the same tensors between captures."""
    sizes, W, S, plan = (2, 8, 2, 600, 128), 130, 9, fattn.fa_rope_axes_plan(128, (64,))
    states = [_train_state(*sizes, seed) for seed in (1, 50)]
    bufs = [([y.clone() for y in x], out) for x, out in states]
    want = []
    for x, out in states:
        _train(x, out, W, S, 0.09, plan)
        want.append([y.clone() for y in out])
        _train(x, out, W, S, 0.09, plan)
        assert all(torch.equal(a, b) for a, b in zip(want[-1], out))
    streams, graphs = [torch.cuda.Stream(), torch.cuda.Stream()], []
    torch.cuda.synchronize()
    for s, (x, out) in zip(streams, bufs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            _train(x, out, W, S, 0.09, plan)
    for turn in range(4):
        for i, (x, out) in enumerate(bufs):
            for a, b in zip(x, states[(i + turn) % 2][0]):
                a.copy_(b)
            for y in out:
                y.fill_(float("nan"))
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for i, (_, out) in enumerate(bufs):
            assert all(torch.equal(a, b) for a, b in zip(out, want[(i + turn) % 2])), f"graph {i}, turn {turn}"
    assert fattn.fa_get_status() == fattn.FA_OK


def test_calls_from_two_threads():
    sizes, W, S, plan = (1, 8, 4, 400, 64), 70, 3, fattn.fa_rope_axes_plan(64, (32,))
    states = [_train_state(*sizes, seed) for seed in (1, 60)]
    want, wrong = [], []
    for x, out in states:
        _train(x, out, W, S, 0.12, plan)
        torch.cuda.synchronize()
        want.append([y.clone() for y in out])

    def work(i):
        x, _ = states[i]
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                out = [torch.empty_like(y) for y in want[i]]
                _train(x, out, W, S, 0.12, plan)
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(a, b) for a, b in zip(out, want[i])):
                    wrong.append(i)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and fattn.fa_get_status() == fattn.FA_OK


def test_the_examples_of_the_readme():
    """They run, and the serving step's outputs are those of one key (the token's own)."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")
    with open(path) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    names = {}
    for block in blocks:
        exec(block, names)
    torch.cuda.synchronize()
    assert fattn.fa_get_status() == fattn.FA_OK
    assert names["lens"].tolist() == [1] * 8 and names["granted"].tolist() == [1] * 8 and int(names["n_free"]) == 1016
    own = names["v"][:, :, 0].repeat_interleave(4, 1)
    assert torch.equal(names["o"], own)  # (a softmax over one key)
