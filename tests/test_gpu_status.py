"""fa_get_status over the kernels of every file: cheap when nothing was raised, and what was raised is told once."""

import threading
import time

import pytest
import torch

from _util import ensure_built
from exact_attention_06_gb300 import fattn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _median(f, n=200):
    times = []
    for _ in range(n):
        t = time.perf_counter()
        f()
        times.append(time.perf_counter() - t)
    return sorted(times)[n // 2]


def test_it_costs_a_kernel_and_a_copy():
    """However many words there are: a kernel, a copy and two waits, each less than a copy and a wait (item())."""
    x = torch.zeros(1, device="cuda")
    for _ in range(20):
        fattn.fa_get_status()
        x.item()
    torch.cuda.synchronize()
    status, copy = _median(fattn.fa_get_status), _median(x.item)
    assert status <= 4 * copy, f"{status * 1e6:.1f} us, a copy and a wait {copy * 1e6:.1f} us"


def _run_out(Nq, Nk, backward):
    """A wait of one cycle in the kernel that such sizes take."""
    q, k = (torch.ones(1, 2, n, 128, dtype=torch.bfloat16, device="cuda") for n in (Nq, Nk))
    o, lse, g = torch.empty_like(q), torch.zeros(1, 2, Nq, device="cuda"), [torch.empty_like(x) for x in (q, k, k)]
    if backward:
        fattn.fa_cross_bwd(q, k, k, q, q, lse, *g, 0.1, wait_budget_cycles=1)
    else:
        fattn.fa_cross_fwd(q, k, k, o, lse, 0.1, wait_budget_cycles=1)


@pytest.mark.parametrize("Nq,Nk,backward", [(600, 700, False), (5000, 77, False), (600, 700, True), (5000, 77, True)])
def test_a_status_is_told_once(Nq, Nk, backward):
    """... also to several threads that ask at once, on streams of their own."""
    assert fattn.fa_get_status() == fattn.FA_OK
    _run_out(Nq, Nk, backward)
    torch.cuda.synchronize()
    told, start = [], threading.Barrier(8)

    def ask():
        with torch.cuda.stream(torch.cuda.Stream()):
            start.wait()
            try:
                told.append(fattn.fa_get_status())
            except fattn.FattnError as e:
                told.append(e.status)
    threads = [threading.Thread(target=ask) for _ in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert sorted(told) == [fattn.FA_OK] * 7 + [fattn.FA_ERR_TIMEOUT]
    assert fattn.fa_get_status() == fattn.FA_OK
