"""Block tables and slots of the paged cache on the GPU: integers, equal to the definition on Python lists."""

import pytest
import torch

from _util import ensure_built
from exact_attention_06_gb300 import fattn
from oracle import window as ow

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


class Cache:
    """The state of the calls, on the GPU and on lists."""

    def __init__(self, B, max_pages, num_pages, ps, seed=0, lens=None):
        g = torch.Generator().manual_seed(seed)
        ids = torch.randperm(num_pages, generator=g).tolist()
        self.ps, self.num = ps, num_pages
        self.lens = lens or [0] * B
        self.table = [[-1] * max_pages for _ in range(B)]
        for b, n in enumerate(self.lens):
            for i in range(-(-n // ps)):
                self.table[b][i] = ids.pop()
        self.free = len(ids)
        self.stack = ids + [-5] * (num_pages - len(ids))
        self.dev = [torch.tensor(x, dtype=torch.int32, device=DEV) for x in (self.table, self.lens, self.stack, [self.free])]

    def extend(self, new, N=0, stream=None):
        t, n, stack, free = self.dev
        B = len(new)
        granted = torch.full((B,), 77, dtype=torch.int32, device=DEV)
        whole = torch.full((B * N + 64,), 7, dtype=torch.int64, device=DEV)
        slots = whole[32:32 + B * N].view(B, N) if N else None
        news = torch.tensor(new, dtype=torch.int32, device=DEV)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        fattn.fa_pages_extend(t, n, news, stack, free, granted, slots, self.ps, stream=stream)
        if stream is not None:
            torch.cuda.current_stream().wait_stream(stream)
        assert fattn.fa_get_status() == fattn.FA_OK
        assert (whole[:32] == 7).all() and (whole[-32:] == 7).all()
        assert news.tolist() == new
        self.table, self.lens, self.stack, self.free, want, want_slots = ow.pages_extend(
            self.table, self.lens, new, self.stack, self.free, self.ps, N)
        assert granted.tolist() == want
        assert t.tolist() == self.table and n.tolist() == self.lens
        assert free.tolist() == [self.free] and stack.tolist() == self.stack
        if N:
            assert slots.tolist() == want_slots
        return want


@pytest.mark.parametrize("ps", [64, 128, 192])
@pytest.mark.parametrize("B", [1, 2, 16, 17, 100, 129, 511, 512, 513, 1500])
def test_a_serving_run(B, ps):
    """Prompts, then single tokens and drafts, rejected ones, finished requests and new ones in the same calls."""
    mp = 6
    c = Cache(B, mp, max(1, B * 4), ps, seed=B)
    g = torch.Generator().manual_seed(B + ps)
    draw = lambda lo, hi: torch.randint(lo, hi, (B,), generator=g).tolist()  # noqa: E731
    c.extend(draw(0, 3 * ps), N=3 * ps if B <= 129 else 5)
    for _ in range(3):
        c.extend([1] * B, N=1)
        c.extend(draw(0, 6), N=6)
        c.extend([-min(x, n) for x, n in zip(draw(0, 6), c.lens)])
        c.extend([-n if x < 2 else x for x, n in zip(draw(0, 2 * ps), c.lens)], N=2)
    assert sum(len([p for p in row if p >= 0]) for row in c.table) + c.free == c.num


def test_giving_back_restores_the_stack():
    c = Cache(70, 8, 500, 64, seed=1, lens=[(37 * b) % 300 for b in range(70)])
    before = [x.clone() for x in c.dev]
    new = [(53 * b) % 200 for b in range(70)]
    assert c.extend(new, N=4) == new
    c.extend([-x for x in new])
    assert all(torch.equal(a, b) for a, b in zip(before, c.dev))


def test_runs_out_of_pages_and_of_room():
    c = Cache(6, 2, 7, 64, seed=2, lens=[64, 64, 63, 64, 0, 128])
    assert c.extend([64, 65, 1, 64, 0, 1], N=3)[5] == 0  # a table's end; 7 pages, 6 in use: one to hand out
    c.extend([1] * 6, N=1)
    c.extend([-1000, 0, -2 ** 31, 2 ** 31 - 1, -1, 0])
    c.extend([3, 4, 5, 6, 7, 8], N=8)


def test_lengths_out_of_range_are_clamped():
    c = Cache(3, 2, 10, 64, seed=3, lens=[0, 128, 10])
    c.lens = [-5, 2 ** 31 - 1, 10]
    c.dev[1].copy_(torch.tensor(c.lens))
    c.extend([1, 1, 1], N=1)
    c.extend([0, -200, 0])


@pytest.mark.parametrize("n_free", [-3, 0, 10 ** 6])
def test_a_count_out_of_range_is_clamped(n_free):
    c = Cache(2, 4, 12, 64, seed=4)
    c.stack = list(range(12))
    c.free = n_free
    c.dev[2].copy_(torch.tensor(c.stack)), c.dev[3].fill_(n_free)
    c.extend([70, 70], N=2)


def test_long_prompts_and_slots_of_pages_outside_the_pool():
    c = Cache(3, 300, 1000, 64, seed=5)
    c.extend([64 * 300, 64 * 123 + 7, 1], N=64 * 300)
    c.table[0][2] = 1000
    c.dev[0][0, 2] = 1000
    c.extend([-64 * 299, 0, 64 * 200], N=9)
    c.table[2][199] = -1  # the page that the next tokens start in
    c.dev[0][2, 199] = -1
    c.lens[2] = 64 * 199 + 3
    c.dev[1][2] = c.lens[2]
    c.extend([0, 0, 70], N=70)


def test_a_page_given_back_twice_stays_inside_the_stack():
    c = Cache(2, 2, 3, 64, seed=6)
    t, n, stack, free = c.dev
    t.copy_(torch.tensor([[0, 1], [0, 1]]))
    n.fill_(128)
    free.fill_(3)  # (all three already free: four pages more than fit)
    guard = torch.full((3 + 64,), 9, dtype=torch.int32, device=DEV)
    mine = guard[32:35]
    granted = torch.empty(2, dtype=torch.int32, device=DEV)
    fattn.fa_pages_extend(t, n, -n, mine, free, granted, None, 64)
    assert fattn.fa_get_status() == fattn.FA_OK
    assert free.item() == 3 and (guard[:32] == 9).all() and (guard[35:] == 9).all() and n.tolist() == [0, 0]


def test_other_streams_and_replays():
    c = Cache(40, 8, 400, 64, seed=7)
    s = torch.cuda.Stream()
    for _ in range(4):
        c.extend([65] * 40, N=70, stream=s)
        c.extend([-60] * 40, stream=s)
    # a captured step, replayed: tokens taken and one given back
    t, n, stack, free = c.dev
    more, less = (torch.full((40,), x, dtype=torch.int32, device=DEV) for x in (3, -1))
    granted, slots = torch.empty(40, dtype=torch.int32, device=DEV), torch.empty(40, 3, dtype=torch.int64, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fattn.fa_pages_extend(t, n, more, stack, free, granted, slots, 64)
        fattn.fa_pages_extend(t, n, less, stack, free, granted, None, 64)
    for _ in range(50):
        graph.replay()
        torch.cuda.synchronize()
        state = ow.pages_extend(c.table, c.lens, [3] * 40, c.stack, c.free, 64, 3)
        assert slots.tolist() == state[5]
        c.table, c.lens, c.stack, c.free = state[:4]
        c.table, c.lens, c.stack, c.free, _, _ = ow.pages_extend(c.table, c.lens, [-1] * 40, c.stack, c.free, 64)
        assert t.tolist() == c.table and n.tolist() == c.lens and stack.tolist() == c.stack and free.item() == c.free
