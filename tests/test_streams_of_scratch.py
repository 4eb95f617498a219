"""Scratch that a call allocates itself belongs to the stream its kernels run on, however the stream is named:
otherwise its memory would go to another stream's tensors while the kernels still use it."""

import contextlib

import pytest
import torch

from _util import ensure_built
from exact_attention_06_gb300 import fattn


class _Recorder:
    """torch.cuda's streams, by handle, without a GPU; like torch's, an ExternalStream of 0 is a stream of the pool."""

    def __init__(self, monkeypatch):
        self.entered = []
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: handle or "pool")
        monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: 0)
        monkeypatch.setattr(torch.cuda, "stream", self.enter)

    @contextlib.contextmanager
    def enter(self, stream):
        self.entered.append(getattr(stream, "cuda_stream", stream))
        yield


@pytest.mark.parametrize("handle,owner", [(0, 0), (1, 0), (2, 2), (0x7f00deadbe00, 0x7f00deadbe00)])
def test_scratch_is_allocated_on_the_stream_of_a_raw_handle(monkeypatch, handle, owner):
    seen = _Recorder(monkeypatch)
    assert fattn._workspace_on(handle, 512, "cpu").numel() == 512
    assert seen.entered == [owner]


def test_scratch_is_allocated_on_a_stream_object(monkeypatch):
    seen = _Recorder(monkeypatch)
    stream = type("Stream", (), {"cuda_stream": 48})()
    fattn._workspace_on(stream, 512, "cpu")
    assert seen.entered == [48]


def _stream_of(address):
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= address < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("no segment holds the address")


@pytest.mark.gpu
def test_the_allocator_holds_scratch_for_the_kernels_stream():
    side = torch.cuda.Stream()
    for stream, handle in ((0, 0), (1, 0), (side.cuda_stream, side.cuda_stream), (side, side.cuda_stream),
                           (torch.cuda.default_stream(), 0)):
        t = fattn._workspace_on(stream, 3 << 20, torch.device("cuda", torch.cuda.current_device()))
        assert _stream_of(t.data_ptr()) == handle, stream


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["none", "default", "legacy", "object", "side"])
def test_a_call_with_scratch_of_its_own_keeps_to_its_stream(kind):
    """The segments that a call takes from the device are its stream's, and its results are those of a call with a
    workspace."""
    ensure_built()
    B, H, Nq, Nk, d = 1, 8, 4096, 300, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    q, do = (torch.randn(B, H, Nq, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    k, v = (torch.randn(B, 1, Nk, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    o, lse = torch.empty_like(q), torch.empty(B, H, Nq, device="cuda")
    grads = [[torch.empty_like(x) for x in (q, k, v)] for _ in range(2)]
    n = fattn.fa_cross_bwd_workspace_bytes(B, H, 1, Nq, Nk, d)
    assert n > 1 << 20  # (a segment of its own)
    fattn.fa_cross_fwd(q, k, v, o, lse, 0.1)
    fattn.fa_cross_bwd(q, k, v, o, do, lse, *grads[0], 0.1, workspace=torch.empty(n, dtype=torch.uint8, device="cuda"))
    side = torch.cuda.Stream()
    stream, handle = {"none": (None, 0), "default": (0, 0), "legacy": (1, 0), "object": (side, side.cuda_stream),
                      "side": (side.cuda_stream, side.cuda_stream)}[kind]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    before = {s["address"] for s in torch.cuda.memory_snapshot()}
    fattn.fa_cross_bwd(q, k, v, o, do, lse, *grads[1], 0.1, stream=stream)
    new = [s for s in torch.cuda.memory_snapshot() if s["address"] not in before]
    torch.cuda.synchronize()
    assert {s["stream"] for s in new} <= {handle}
    assert kind in ("none", "default", "legacy") or new
    assert fattn.fa_get_status() == fattn.FA_OK
    assert all(torch.equal(x, y) for x, y in zip(*grads))


class _Library:
    """Every size is 512 bytes and every call succeeds."""

    def __getattr__(self, name):
        return lambda *args: 512 if name.endswith("bytes") else 0


@pytest.mark.parametrize("handle,owner", [(0, 0), (0x7f00deadbe00, 0x7f00deadbe00), (None, None)])
@pytest.mark.parametrize("call", ["fa_bwd", "fa_decode_paged"])
def test_the_other_calls_allocate_on_their_stream_too(monkeypatch, call, handle, owner):
    seen = _Recorder(monkeypatch)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: type("Stream", (), {"cuda_stream": 0})())
    monkeypatch.setattr(fattn, "_need", lambda *args: None)
    monkeypatch.setattr(fattn, "lib", _Library)
    x, lse = torch.zeros(1, 2, 64, 64, dtype=torch.bfloat16), torch.zeros(1, 2, 64)
    if call == "fa_bwd":
        fattn.fa_bwd(x, x, x, x, x, lse, x, x, x, 0.1, stream=handle)
    else:
        table = torch.zeros(1, 1, dtype=torch.int32)
        fattn.fa_decode_paged(x[:, :, 0], x, x, table, table[0], x[:, :, 0], lse[:, :, 0], 0.1, 64, stream=handle)
    assert seen.entered == ([] if owner is None else [owner])


@pytest.mark.gpu
def test_a_backward_on_a_side_stream_keeps_its_scratch():
    """fa_bwd's row sums, on a side stream behind a long wait: a tensor that the current stream allocates and fills after
    the call must not lie in them."""
    ensure_built()
    B, H, N, d = 2, 8, 4096, 64
    g = torch.Generator(device="cuda").manual_seed(4)
    q, k, v, do = (torch.randn(B, H, N, d, generator=g, device="cuda").bfloat16() for _ in range(4))
    o, lse = torch.empty_like(q), torch.empty(B, H, N, device="cuda")
    fattn.fa_fwd(q, k, v, o, lse, 0.1)
    want, got = ([torch.empty_like(q) for _ in range(3)] for _ in range(2))
    fattn.fa_bwd(q, k, v, o, do, lse, *want, 0.1)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    n = fattn.fa_bwd_workspace_bytes(B, H, N)
    for stream in (side, side.cuda_stream):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)  # some 10 ms
        fattn.fa_bwd(q, k, v, o, do, lse, *got, 0.1, stream=stream)
        other = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        assert fattn.fa_get_status() == fattn.FA_OK
        assert all(torch.equal(x, y) for x, y in zip(want, got))
        assert all((t == 255).all() for t in other)
        del other


@pytest.mark.parametrize("handle,owner", [(0, 0), (1, 0), (0x7f00deadbe00, 0x7f00deadbe00)])
def test_a_handle_may_be_an_object_that_is_a_number(monkeypatch, handle, owner):
    """(fa_bwd and fa_decode_paged take whatever int() does.)"""
    seen = _Recorder(monkeypatch)
    number = type("Handle", (), {"__int__": lambda self: handle})()
    fattn._workspace_on(number, 512, "cpu")
    assert seen.entered == [owner]
