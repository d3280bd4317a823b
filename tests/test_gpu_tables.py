"""pkv_batch_tables on the GPU against the definition, request by request: block tables,
slots, positions, query offsets, context lengths, the ring and its state, all equal."""
import random

import pytest
import torch

import serving_ref as R
from paged_kv_attention_09_gb300 import pkv

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Step:
    def __init__(self, N, head, ring, count, cached, new, bt, T, with_starts=True, with_positions=True):
        B, MB = len(cached), len(bt[0]) if bt else 1
        self.state0 = [head, count, 0, 0]
        self.args = (ring, self.state0, cached, new, bt, T)
        self.pool = pkv.PagePool(i32(ring), i32(self.state0))
        self.cached, self.new = i32(cached), i32(new)
        self.bt = i32(bt) if bt else torch.zeros(0, MB, dtype=torch.int32, device="cuda")
        self.context = i32([7] * B)
        self.starts = i32([7] * (B + 1)) if with_starts else None
        self.positions = i32([7] * T) if with_positions else None
        self.slots = i32([7] * T)
        self.status = i32([0])

    def call(self, **kw):
        return pkv.pkv_batch_tables(self.pool, self.cached, self.new, self.bt, self.context, self.starts,
                                    self.positions, self.slots, self.status, **kw)

    def check(self, want=None):
        torch.cuda.synchronize()
        w = R.tables(*self.args) if want is None else want
        got = dict(bt=self.bt.tolist(), context=self.context.tolist(), slots=self.slots.tolist(),
                   ring=self.pool.ring.tolist(), state=self.pool.state.tolist(), status=int(self.status[0]))
        if self.starts is not None:
            got["starts"] = self.starts.tolist()
        if self.positions is not None:
            got["positions"] = self.positions.tolist()
        for k, v in got.items():
            assert v == w[k], k
        return w


def draw(seed, B, MB, N, max_cached, max_new, ended=0.1, none=0.1, short=False, head=None, pad=0, **kw):
    rng = random.Random(seed)
    cached = [rng.randint(0, min(max_cached, MB * 16)) for _ in range(B)]
    new = [-1 if rng.random() < ended else 0 if rng.random() < none else
           rng.randint(1, max(1, min(max_new, MB * 16 - c))) if c < MB * 16 else 0 for c in cached]
    perm = rng.sample(range(N), N)
    bt, at = [], 0
    for c in cached:
        n = R.pages(c)
        bt.append(perm[at:at + n] + [-1] * (MB - n))
        at += n
    assert at <= N, "the pool is too small for the test"
    need = sum(R.pages(c + n) - R.pages(c) for c, n in zip(cached, new) if n > 0)
    free = perm[at:]
    if short:
        free = free[:need // 2]
    head = rng.randrange(N) if head is None else head
    ring = [-9] * N
    for i, p in enumerate(free):
        ring[(head + i) % N] = p
    T = sum(max(n, 0) for n in new) + pad
    return Step(N, head, ring, len(free), cached, new, bt, T, **kw)


@pytest.mark.parametrize("B,MB,N,max_cached,max_new", [
    (1, 1, 1, 0, 16), (1, 4, 8, 37, 1), (2, 8, 64, 100, 40), (31, 16, 700, 200, 1), (256, 8, 4096, 100, 1),
    (257, 16, 5000, 150, 90), (1023, 4, 5000, 40, 20), (1024, 4, 5000, 40, 20), (1025, 4, 5000, 40, 20),
    (2500, 3, 9000, 30, 18), (3, 400, 1500, 1000, 5000)])
@pytest.mark.parametrize("short", [False, True])
def test_against_the_definition(B, MB, N, max_cached, max_new, short):
    s = draw(B + MB, B, MB, N, max_cached, max_new, short=short, pad=B % 7)
    s.call()
    s.check()


def test_ring_wraps_and_everything_is_returned():
    s = draw(3, 40, 6, 300, 90, 1, ended=0.9, head=297)
    s.call()
    w = s.check()
    assert w["state"][1] > s.state0[1]


def test_no_requests_and_no_rows():
    s = Step(4, 1, [0, 1, 2, 3], 2, [], [], [], 3)
    s.call()
    s.check()
    s = Step(4, 1, [0, 1, 2, 3], 2, [5, 0], [0, 0], [[3, -1], [-1, -1]], 0)
    s.call()
    s.check()


def test_optional_outputs():
    s = draw(4, 20, 8, 400, 100, 30, with_starts=False, with_positions=False)
    s.call()
    s.check()


@pytest.mark.parametrize("case", ["negative", "beyond", "rows", "page", "ring", "state", "returned twice", "released"])
def test_bad_input_is_reported_and_stays_in_bounds(case):
    cached, new, T = [20, 7, 40, 33], [3, 12, -1, 30], 45
    bt = [[1, 2, -1, -1], [3, -1, -1, -1], [4, 5, 6, -1], [7, 8, 9, -1]]
    ring, head, count = list(range(20)), 10, 10
    if case == "negative":
        cached[1], cached[2] = -5, -1
    elif case == "beyond":
        new[0], cached[2] = 60, 65
    elif case == "rows":
        T = 40  # the last request's rows pass the end: none of them is served
    elif case == "page":
        bt[0][1], bt[2][1] = 20, 25
    elif case == "ring":
        ring[10], ring[11] = -3, 20
    elif case == "state":
        head = 20
    elif case == "returned twice":
        count = 20
        head = 0
    elif case == "released":
        bt[2][0] = -1  # given back before (a window moved past it)
    s = Step(20, head, ring, count, cached, new, bt, T)
    s.call()
    w = s.check()
    assert (w["status"] != 0) == (case != "released")


def test_huge_lengths_do_not_overflow():
    big = 2**31 - 1
    s = Step(8, 0, list(range(8)), 8, [big, 0, big, 1], [big, big, 1, 1], [[0, 1]] * 3 + [[2, -1]], 40)
    s.call()
    s.check()
    s = Step(8, 0, list(range(8)), 8, [0] * 3000, [big] * 2999 + [1], [[-1]] * 3000, 10)
    s.call()
    s.check()


def test_replayed_graph_steps_on_the_pool_in_place():
    """One captured step replayed: each replay extends every request by a token, ends one
    and the pages flow round, exactly as the definition says, step after step."""
    rng = random.Random(0)
    B, MB, N = 24, 6, 90
    s = Step(N, 0, list(range(N)), N, [0] * B, [1] * B, [[-1] * MB for _ in range(B)], B + 3)
    s.call()  # (a first call outside the capture)
    w = s.check()
    g = torch.cuda.CUDAGraph()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=st):
        s.call()
    for step in range(60):
        cached = [c for c in w["context"]]
        new = []
        for b in range(B):
            if cached[b] > 0 and rng.random() < 0.04:
                new.append(-1)
            else:
                new.append(1 if cached[b] < MB * 16 else -1)
        s.cached.copy_(i32(cached))
        s.new.copy_(i32(new))
        s.status.zero_()
        g.replay()
        torch.cuda.synchronize()
        w = R.tables(w["ring"], w["state"], cached, new, w["bt"], B + 3)
        s.check(w)
    assert w["state"][1] <= N




def test_other_stream_and_bound_call():
    s = draw(8, 50, 8, 800, 100, 30)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    call = s.call(stream=st, bound=True)
    assert s.slots[0].item() == 7  # nothing issued yet
    call()
    s.check()


def test_numbers_of_rows_beyond_one_block_share_the_pool_update():
    """Many blocks (a long prompt): the last one updates the pool once."""
    s = Step(4096, 7, [(i * 5) % 4096 for i in range(4096)], 4000, [3, 100, 50], [40000, -1, 20001],
             [[-1] * 2600, list(range(7)) + [-1] * 2593, [100, 101, 102, 103] + [-1] * 2596], 60001 + 13)
    s.args[4][0][0] = 99
    s.bt[0, 0] = 99
    s.call()
    w = s.check()
    assert w["state"][2] == 0
    # (the ring also lists pages 99 .. 103 that the tables name: slots may repeat here)
    assert sum(x >= 0 for x in w["slots"]) == 60001
