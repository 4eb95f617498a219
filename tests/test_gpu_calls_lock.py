"""The compiled calls release the interpreter's lock while the library enqueues, as ctypes does for the others: a call that
waits for room in the launch queue must not keep out the thread or host function that the GPU is waiting for."""

import ctypes

import pytest
import torch

from _util import ensure_built
from exact_attention_06_gb300 import fattn

pytestmark = pytest.mark.gpu
NAMES = ("fa_cross_fwd", "fa_cross_workspace_bytes", "fa_cross_bwd", "fa_cross_bwd_workspace_bytes", "fa_rope_axes",
         "fa_rope_axes_paged")


@pytest.fixture
def holds_lock():
    """The module bound to a function that returns 1 in the place of the library's where the calling thread holds the
    lock, else 0 (and takes no arguments: those passed are ignored)."""
    ensure_built()
    fattn._load_calls()
    address = lambda f: ctypes.cast(f, ctypes.c_void_p).value  # noqa: E731
    check = address(ctypes.pythonapi.PyGILState_Check)
    library = {n: address(getattr(fattn.lib(), n)) for n in NAMES}
    fattn._calls.bind(*(library[n] if n.endswith("bytes") else check for n in NAMES))
    yield
    fattn._calls.bind(*library.values())


def test_the_lock_is_free_while_a_call_is_enqueued(holds_lock):
    x = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    q, k, lse = x(1, 4, 40, 64), x(1, 2, 300, 64), torch.zeros(1, 4, 40, device="cuda")
    kn, pool, plan, ws = x(1, 2, 40, 64), x(2, 2, 64, 64), fattn.fa_rope_axes_plan(64, (32,)), \
        torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    m = fattn._calls
    for scratch in (None, ws):
        assert m.cross_fwd(q, k, k, q, lse, 0.1, None, scratch, None, 0) == 0
        assert m.cross_bwd(q, k, k, q, q, lse, q, k, k, 0.1, None, scratch, None, 0) == 0
    assert m.rope_axes(q, kn, i(1, 1, 40), plan, q, kn, False, None) == 0
    assert m.rope_axes_paged(q, kn, kn, i(1, 1, 40), plan, q, pool, pool, i(1, 2), i(1), None, None) == 0
    assert m.rope_axes_paged("q", kn, kn, i(1, 1, 40), plan, q, pool, pool, i(1, 2), i(1), None, None) == -1
