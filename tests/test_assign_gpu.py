"""Page tables and slots from lengths (fa_page_assign) against the definition one page after another (cache8_ref.assign):
random steps of batches whose sequences grow, shrink, end and run out of pages, with and without windows."""
import random

import pytest
import torch

import attention_fa_fwd_03_gb300 as fa
import cache8_ref as ref

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def clear():
    torch.cuda.synchronize()
    return fa.fa_device_status() == 0


class State:
    def __init__(self, B, mp, ids):
        self.table = i32([[-1] * mp for _ in range(B)])
        self.held = i32([[0, 0, 0]] * B)
        self.free = i32(ids)
        self.count = i32([len(ids), 0])

    def lists(self):
        return self.table.tolist(), [tuple(x) for x in self.held.tolist()], self.free.tolist(), int(self.count[0])


def step(st, lens, page, T, new=None, window=0, sinks=0, with_slots=True, stream=None):
    """One call, compared with the definition from the same state."""
    table, held, free, count = st.lists()
    want = ref.assign(table, lens, held, free, count, page, T, len(free), new, window, sinks)
    slots = torch.full((len(lens), T), -99, dtype=torch.int64, device="cuda") if with_slots else None
    fa.fa_page_assign(st.table, i32(lens), st.held, st.free, st.count, page, T, new_lens=None if new is None else i32(new),
                      window=window, sinks=sinks, slots=slots, stream=stream)
    assert clear()
    table, held, free, count = st.lists()
    assert table == want[0]
    assert held == want[1]
    assert free[:count] == want[2] and st.count.tolist() == [len(want[2]), want[3]]
    if with_slots:
        assert slots.tolist() == want[4]
    assert sorted([p for r in table for p in r if p >= 0] + free[:count]) == sorted(range(len(free)))  # none lost, none twice


@pytest.mark.parametrize("seed", range(12))
def test_random_steps(seed):
    rng = random.Random(seed)
    B, page, mp = rng.choice([1, 2, 7, 33, 100]), rng.choice([16, 32, 64, 256]), rng.randint(1, 40)
    P = rng.randint(1, B * mp + 4)
    ids = list(range(P))
    rng.shuffle(ids)
    st = State(B, mp, ids)
    window, sinks = (0, 0) if seed % 3 == 0 else (rng.randint(1, mp * page), rng.choice([0, 4, rng.randint(0, 200)]))
    lens = [0] * B
    for _ in range(8):
        T = rng.choice([1, rng.randint(1, 40), rng.randint(1, mp * page)])
        for b in range(B):
            kind = rng.random()
            if kind < 0.1:
                lens[b] = 0
            elif kind < 0.2:
                lens[b] = rng.randint(0, mp * page)  # taken back, or filled from elsewhere
            else:
                lens[b] = min(mp * page, lens[b] + rng.randint(0, T))
        new = [rng.randint(0, min(T, n)) for n in lens] if min(lens) < T or rng.random() < 0.7 else None
        step(st, lens, page, T, new, window, sinks, with_slots=rng.random() < 0.8)


def test_many_sequences():
    """More sequences than a block has threads, and more slots than one launch writes."""
    rng = random.Random(5)
    B, page, mp = 2500, 16, 3
    ids = list(range(B * mp - 400))
    rng.shuffle(ids)
    st = State(B, mp, ids)
    for window, sinks in ((0, 0), (17, 3), (17, 3)):
        lens = [rng.randint(0, mp * page) for _ in range(B)]
        new = [rng.randint(0, min(20, n)) for n in lens]
        step(st, lens, page, 20, new, window, sinks)


def test_long_prompts():
    st = State(3, 600, list(range(1700))[::-1])
    step(st, [9000, 1, 5000], 16, 9000, [9000, 1, 5000])
    step(st, [9001, 2, 0], 16, 1, [1, 1, 0], 1000, 100)
    step(st, [9002, 3, 9600], 16, 9600, [1, 1, 9600], 1000, 100)
    step(st, [0, 0, 0], 16, 1, [0, 0, 0], 1000, 100)
    assert st.count.tolist() == [1700, 0]


def test_states_and_lengths_out_of_range():
    """Clamped and reported; nothing outside the arrays is read or written (guards around them stay)."""
    B, mp, P = 4, 5, 12
    whole = torch.full((B * mp + 3 * B + P + 2 + 8,), 77, dtype=torch.int32, device="cuda")
    table, held = whole[2:2 + B * mp].view(B, mp), whole[2 + B * mp:2 + B * mp + 3 * B].view(B, 3)
    free, count = whole[4 + B * mp + 3 * B:4 + B * mp + 3 * B + P], whole[6 + B * mp + 3 * B + P:8 + B * mp + 3 * B + P]
    table.copy_(i32([[0, 1, -5, 999, 4]] * B))
    held.copy_(i32([[0, 0, 5], [-3, 9, 2], [2, 1, 99], [7, 7, 7]]))
    free.copy_(i32(list(range(P))))
    count.copy_(i32([P + 50, 3]))
    before = whole.clone()
    slots = torch.empty(B, 3, dtype=torch.int64, device="cuda")
    fa.fa_page_assign(table, i32([0, -4, 1 << 30, 3]), held, free, count, 16, 3, new_lens=i32([0, 2, 9, -1]), window=20, sinks=3,
                      slots=slots)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == 4
    inside = torch.zeros_like(whole, dtype=torch.bool)
    for lo, n in ((2, B * mp + 3 * B), (4 + B * mp + 3 * B, P), (6 + B * mp + 3 * B + P, 2)):
        inside[lo:lo + n] = True
    assert torch.equal(whole[~inside], before[~inside])
    h = held.tolist()
    assert all(0 <= a <= f <= e <= mp for a, f, e in h)
    assert 0 <= int(count[0]) <= P and int(slots.max()) < P * 16


def test_captured_and_replayed():
    """A captured call replayed at other lengths, and on another stream than the tensors' own."""
    B, mp, page = 6, 20, 16
    ids = list(range(B * mp))
    a, b = State(B, mp, ids), State(B, mp, ids)
    lens, new = i32([0] * B), i32([0] * B)
    slots = torch.empty(B, 40, dtype=torch.int64, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        fa.fa_page_assign(a.table, lens, a.held, a.free, a.count, page, 40, new_lens=new, window=50, sinks=10, slots=slots)
    rng = random.Random(1)
    now = [0] * B
    for _ in range(8):
        m = [rng.randint(0, 40) for _ in range(B)]
        now = [min(mp * page, x + y) for x, y in zip(now, m)]
        m = [min(x, y) for x, y in zip(now, m)]
        lens.copy_(i32(now))
        new.copy_(i32(m))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        step(b, now, page, 40, m, 50, 10)
        assert a.lists()[:2] == b.lists()[:2] and a.count.tolist() == b.count.tolist()
