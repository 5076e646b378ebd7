"""Page plans on the GPU against the plan made a page at a time."""
import numpy as np
import pytest
import torch

import gpu_common as gc
import kv_common as kc
import round_common as rc

pytestmark = pytest.mark.gpu
PAGE, LENGTH, POOL = 12, 13, 14


@pytest.fixture(scope="module")
def ssdv():
    return gc.cuda_lib()


class State:
    """Requests that hold pages for `length` tokens, the first `shared` columns pages of others."""

    def __init__(self, length, page, width, free, shared=None, seed=0):
        g = np.random.default_rng(seed)
        self.page, B = page, len(length)
        self.shared = np.zeros(B, dtype=np.int64) if shared is None else np.asarray(shared)
        self.held = np.maximum(self.shared, -(-np.asarray(length) // page))
        self.pool = int((self.held - self.shared).sum()) + free + 5
        ids = g.permutation(self.pool)
        self.table = np.full((B, width), -1)
        at = 0
        for b in range(B):
            self.table[b, :self.shared[b]] = self.pool - 1 - np.arange(self.shared[b])
            own = int(self.held[b] - self.shared[b])
            self.table[b, self.shared[b]:self.held[b]] = ids[at:at + own]
            at += own
        self.n_free = free
        self.stack = np.full(self.pool, -1)
        self.stack[:free] = ids[at:at + free]

    def tensors(self):
        return [kc.ints(self.table), kc.ints(self.held), kc.ints(self.stack), kc.ints([self.n_free])]


def check(ssdv, s, length, new, n, in_place=False, uniform=False, status=0, keep=False):
    length, new = np.asarray(length), np.asarray(new)
    t = s.tensors()
    ws = torch.zeros(ssdv._kv_plan_bytes(len(length)), dtype=torch.uint8, device="cuda")
    got = ssdv.kv_plan(*t, kc.ints(length), n, s.page, n_new=None if uniform else kc.ints(new),
                       n_shared=kc.ints(s.shared) if s.shared.any() else None, out=t if in_place else None, workspace=ws)
    assert ssdv.read_status(ws) == status
    table, held, stack, free, served = rc.plan(s.table, s.held, s.stack, s.n_free, length, new, s.page, s.shared)
    want = (table, held, stack, [free], rc.slots(table, length, new, served, s.page, n))
    for name, x, y in zip(("table", "held", "stack", "free", "slots"), got, want):
        assert np.array_equal(x.cpu().numpy(), y), name
    if not in_place:
        for x, y in zip(t, (s.table, s.held, s.stack, [s.n_free])):
            assert np.array_equal(x.cpu().numpy(), y)
    if keep:
        s.table, s.held, s.stack, s.n_free = table, held, stack, free
    return served


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,page", [(1, 16), (3, 48), (31, 64), (32, 16), (33, 16), (200, 32), (1024, 16), (2500, 16)])
def test_rounds(ssdv, B, page, in_place):
    """Requests that go on, end and begin, for a few rounds; in one CTA and, in the larger batches, in two kernels."""
    g = np.random.default_rng(B)
    length = g.integers(0, 300, B)
    s = State(length, page, 40, 40 * B // 2 + 7, seed=B)
    n = 9
    for r in range(4):
        new = g.integers(0, n + 1, B)
        end = g.random(B) < 0.2
        length = np.where(end, 0, length)
        new = np.where(end & (g.random(B) < 0.5), 0, new)
        check(ssdv, s, length, new, n, in_place=in_place, keep=True)
        length = length + g.integers(0, new + 1)


@pytest.mark.parametrize("n", [0, 1, 255, 256, 257, 3000])
def test_prompts_and_slots(ssdv, n):
    """Many slots a request, none among them; counts at a page's and a chunk's end."""
    length = np.array([0, 15, 16, 17, 0, 100])
    new = np.minimum([n, n, max(n - 1, 0), 16, 0, 1], n)
    for in_place in (False, True):
        check(ssdv, State(length, 16, 200, 900), length, new, n, in_place=in_place)
    check(ssdv, State(length, 16, 200, 1200), length, np.full(6, n), n, uniform=True)


@pytest.mark.parametrize("in_place", [False, True])
def test_too_few_pages(ssdv, in_place):
    """Requests are served in order until one does not fit; what is given back counts."""
    length = np.array([40, 0, 64, 10, 64, 16, 160])
    s = State(length, 16, 12, 2, seed=3)
    s2 = State(length, 16, 12, 0, seed=4)
    now = length.copy()
    now[0] = 0  # ends: three pages come back
    served = check(ssdv, s, now, [0, 33, 5, 5, 20, 1, 0], 40, in_place=in_place, status=POOL)
    assert served.tolist() == [True, True, True, True, False, False, True]
    served = check(ssdv, s2, length, [0, 1, 0, 6, 0, 0, 1], 8, in_place=in_place, status=POOL)
    assert served.tolist() == [True, False, True, True, True, True, False]
    check(ssdv, State(length, 16, 12, 0, seed=5), length, [0, 0, 0, 6, 0, 0, 0], 8, in_place=in_place)


@pytest.mark.parametrize("in_place", [False, True])
def test_shared_columns(ssdv, in_place):
    """Columns of others are neither taken nor given; a request that ends keeps only those."""
    length, shared = np.array([50, 64, 200, 48]), [3, 4, 0, 3]
    s = State(length, 16, 20, 30, shared=shared)
    check(ssdv, s, [0, 64, 0, 48], [0, 9, 1, 40], 40, in_place=in_place, keep=True)
    assert s.held.tolist() == [3, 5, 1, 6]


@pytest.mark.parametrize("in_place", [False, True])
def test_bad_requests_keep_what_they_had(ssdv, in_place):
    length = np.array([50, 64, 20, 48, 30, 30])
    for at, what, value in ((1, "length", -1), (1, "new", -1), (1, "new", 9), (1, "length", 16 * 10 - 1), (1, "held", 11),
                            (1, "held", -1), (1, "shared", 6), (1, "shared", -1), (1, "length", 2 ** 31 - 1)):
        s = State(length, 16, 10, 30, shared=[1] * 6)
        now, new = length.copy(), np.full(6, 8)
        {"length": now, "new": new, "held": s.held, "shared": s.shared}[what][at] = value
        if what == "new" and value == 9:  # above n
            t = s.tensors()
            ws = torch.zeros(ssdv._kv_plan_bytes(6), dtype=torch.uint8, device="cuda")
            got = ssdv.kv_plan(*t, kc.ints(now), 8, 16, n_new=kc.ints(new), n_shared=kc.ints(s.shared), workspace=ws)
            assert ssdv.read_status(ws) == LENGTH
            assert (got[4][1] == -1).all() and got[1][1] == s.held[1] and np.array_equal(got[0][1].cpu(), s.table[1])
            assert (got[4][2] >= 0).all()
            continue
        served = check(ssdv, s, now, new, 8, in_place=in_place, status=LENGTH)
        assert served.tolist() == [True, False, True, True, True, True]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n_free", [-1, 1 << 30, None])
def test_broken_stack_changes_nothing(ssdv, n_free, in_place):
    """n_free out of range, or more pages than the pool has once those given back lie on it."""
    length = np.array([50, 64, 200])
    s = State(length, 16, 20, 30)
    s.n_free = s.pool if n_free is None else n_free
    t = s.tensors()
    ws = torch.zeros(ssdv._kv_plan_bytes(3), dtype=torch.uint8, device="cuda")
    got = ssdv.kv_plan(*t, kc.ints([0, 64, 200]), 8, 16, out=t if in_place else None, workspace=ws)
    assert ssdv.read_status(ws) == PAGE
    for x, y in zip(got, (s.table, s.held, s.stack, [s.n_free])):
        assert np.array_equal(x.cpu().numpy(), y)
    assert (got[4] == -1).all()


def test_large_batch_gives_everything_back(ssdv):
    """More requests than the CTA has threads, all pages of which come back in order, and go again."""
    B = 3001
    length = np.arange(B) % 97
    s = State(length, 16, 8, 0)
    check(ssdv, s, np.zeros(B, dtype=int), np.zeros(B, dtype=int), 1, in_place=True, keep=True)
    assert s.n_free == s.pool - 5 and (s.table == -1).all()
    check(ssdv, s, np.zeros(B, dtype=int), length, 96, in_place=True, keep=True)
    assert s.n_free == 0


def test_page_numbers_past_32_bits_of_slots(ssdv):
    """Slots of a pool with more than 2^31 tokens."""
    s = State([0, 5], 1 << 16, 2, 3)
    s.stack[:3] = [70000, 2 ** 31 - 1, 9]
    s.table[1, 0] = 60000
    check(ssdv, s, [0, 5], [3, 2], 3)


def test_capture_and_streams(ssdv):
    """A captured plan in place advances at each replay; a plan on another stream gives the same."""
    length = np.array([10, 30, 47, 5])
    s = State(length, 16, 30, 60)
    t, lens, step = s.tensors(), kc.ints(length), kc.ints([16] * 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws = torch.zeros(ssdv._kv_plan_bytes(4), dtype=torch.uint8, device="cuda")
    with torch.cuda.stream(side):
        other = ssdv.kv_plan(*t, lens, 16, 16, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ssdv.kv_plan(*t, lens, 16, 16, out=t, workspace=ws)
        lens += step
    for r in range(5):
        graph.replay()
        table, held, stack, free, served = rc.plan(s.table, s.held, s.stack, s.n_free, length, np.full(4, 16), 16, s.shared)
        want = (table, held, stack, [free], rc.slots(table, length, np.full(4, 16), served, 16, 16))
        for x, y in zip(got, want):
            assert np.array_equal(x.cpu().numpy(), y), r
        if r == 0:
            for x, y in zip(other, want):
                assert np.array_equal(x.cpu().numpy(), y)
        s.table, s.held, s.stack, s.n_free = table, held, stack, free
        length = length + 16
    assert ssdv.read_status(ws) == 0
