"""GPU: page bookkeeping on the device (kvq_pages_assign) against a plain
sequential allocator, step by step: every table, ring, slot and prefix sum is a
whole number and must be equal."""
import numpy as np
import pytest
import torch

from bit_kv_cache_19_b200 import kvq
from bit_kv_cache_19_b200.runtime import DevicePageAllocator

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Plain:
    """The definition, one sequence after the other."""

    def __init__(self, ids, batch, max_pages, span):
        self.table = -np.ones((batch, max_pages), np.int64)
        self.held = np.zeros(batch, np.int64)
        self.ids, self.head, self.count, self.span = np.array(ids), 0, len(ids), span

    def step(self, lens, n_new, n_slots):
        n_pages, B = len(self.ids), len(lens)
        cu = np.concatenate([[0], np.cumsum(np.maximum(n_new, 0))])
        need = -(-(lens + n_new) // self.span)
        ok = (lens >= 0) & (n_new >= 0) & (need <= self.table.shape[1]) & (cu[1:] <= n_slots)
        refused = ~ok
        for b in np.nonzero(ok)[0]:
            for j in range(need[b], self.held[b]):
                self.ids[(self.head + self.count) % n_pages] = self.table[b, j]
                self.count += 1
                self.table[b, j] = -1
            self.held[b] = min(self.held[b], need[b])
        out = False
        for b in np.nonzero(ok)[0]:
            take = need[b] - self.held[b]
            if take and (out or take > self.count):
                out = refused[b] = True
                continue
            for j in range(self.held[b], need[b]):
                self.table[b, j] = self.ids[self.head]
                self.head, self.count = (self.head + 1) % n_pages, self.count - 1
            self.held[b] = need[b]
        slots, pos = [], []
        for b in range(B):
            for j in range(max(n_new[b], 0)):
                t = lens[b] + j
                pos.append(t)
                slots.append(-1 if refused[b] else
                             self.table[b, t // self.span] * self.span + t % self.span)
        return cu, np.array(slots[:n_slots], np.int64), np.array(pos[:n_slots], np.int64), refused


def run(batch, n_pages, page_tiles, max_pages, steps, seed, n_slots=None, graph=False):
    rng = np.random.default_rng(seed)
    span = 32 * page_tiles
    A = DevicePageAllocator(n_pages, page_tiles, batch, max_pages)
    ids = rng.permutation(n_pages)
    A.free_ids.copy_(torch.from_numpy(ids.astype(np.int32)))
    P = Plain(ids, batch, max_pages, span)
    lens = np.zeros(batch, np.int64)
    some_refused = False
    for kind in steps:
        if kind == "decode":
            n_new = np.ones(batch, np.int64)
        elif kind == "prefill":
            n_new = rng.integers(0, 3 * span, batch)
        elif kind == "mixed":
            n_new = rng.integers(0, 40, batch) * rng.integers(0, 2, batch)
            gone = rng.random(batch) < 0.3
            lens[gone], n_new[gone] = 0, 0
        elif kind == "rollback":
            lens, n_new = np.maximum(lens - rng.integers(0, span, batch), 0), np.zeros(batch, np.int64)
        elif kind == "bad":
            n_new = rng.integers(-3, 4, batch)
            lens = np.where(rng.random(batch) < 0.1, -5, lens)
        total = int(np.maximum(n_new, 0).sum())
        cap = total + 5 if n_slots is None else n_slots
        A.status.zero_()
        slots = torch.full((cap,), -77, dtype=torch.int64, device=DEV)
        pos = torch.full((cap,), -77, dtype=torch.int32, device=DEV)
        dl, dn = (torch.from_numpy(x.astype(np.int32)).to(DEV) for x in (lens, n_new))
        cu, _, _ = A.assign(dl, dn, slots=slots, pos=pos)
        wcu, wslots, wpos, refused = P.step(lens, n_new, cap)
        n = len(wslots)
        assert np.array_equal(cu.cpu().numpy(), wcu)
        assert np.array_equal(slots[:n].cpu().numpy(), wslots)
        assert np.array_equal(pos[:n].cpu().numpy(), wpos)
        assert (slots[n:] == -77).all() and (pos[n:] == -77).all()  # left as they were
        assert np.array_equal(A.table.cpu().numpy(), P.table)
        assert np.array_equal(A.held.cpu().numpy(), P.held)
        assert A.free_ring.cpu().tolist() == [P.head, P.count]
        free = A.free_ids.cpu().numpy()[(P.head + np.arange(P.count)) % n_pages]
        assert np.array_equal(free, P.ids[(P.head + np.arange(P.count)) % n_pages])
        assert A.flags() == (kvq.FLAG_CAPACITY if refused.any() else 0)
        some_refused |= bool(refused.any())
        lens = np.where(refused | (lens < 0), np.maximum(lens, 0), lens + np.maximum(n_new, 0))
        # every page is in exactly one place
        assert sorted(np.concatenate([P.table[P.table >= 0], free]).tolist()) == list(range(n_pages))
    return some_refused


@pytest.mark.parametrize("batch", [1, 5, 33, 300, 769, 2100])
@pytest.mark.parametrize("page_tiles", [1, 4])
def test_steps(batch, page_tiles):
    steps = ["prefill", "decode", "mixed", "decode", "rollback", "mixed", "prefill", "mixed"]
    assert not run(batch, 14 * batch, page_tiles, 14, steps, batch + page_tiles)


@pytest.mark.parametrize("batch,n_pages,max_pages,n_slots", [
    (7, 9, 20, None),      # the pool runs out
    (40, 400, 3, None),    # rows too short
    (40, 400, 9, 700),     # slots too few
    (900, 1500, 4, 9000), (1, 1, 1, 10)])
def test_refusals(batch, n_pages, max_pages, n_slots):
    assert run(batch, n_pages, 1, max_pages, ["prefill", "bad", "mixed", "prefill", "mixed",
                                              "decode"] * 2, 17, n_slots=n_slots)


def test_no_slots_and_no_positions():
    A = DevicePageAllocator(4, 1, 2, 2)
    n = torch.tensor([0, 0], dtype=torch.int32, device=DEV)
    lens = torch.tensor([40, 0], dtype=torch.int32, device=DEV)
    empty = torch.empty(0, dtype=torch.int64, device=DEV)
    cu = torch.empty(3, dtype=torch.int32, device=DEV)
    kvq.pages_assign(A.state, lens, n, cu, empty, None, A.ws, A.status)
    assert A.held.tolist() == [2, 0] and cu.tolist() == [0, 0, 0] and A.flags() == 0


@pytest.mark.parametrize("ring", [[-1, 4], [4, 1], [0, 5], [0, -1]])
def test_a_broken_ring_moves_nothing(ring):
    A = DevicePageAllocator(4, 1, 2, 2)
    A.free_ring.copy_(torch.tensor(ring))
    i32 = dict(dtype=torch.int32, device=DEV)
    cu, slots, _ = A.assign(torch.zeros(2, **i32), torch.tensor([3, 4], **i32), 7)
    assert A.flags() == kvq.FLAG_BAD_PAGE
    assert A.free_ring.tolist() == ring and (A.table == -1).all() and (slots == -1).all()
    assert cu.tolist() == [0, 3, 7]


def test_pages_held_out_of_range_and_returned_twice():
    i32 = dict(dtype=torch.int32, device=DEV)
    A = DevicePageAllocator(4, 1, 2, 2)
    A.held[0] = 3  # more than a row has
    _, slots, _ = A.assign(torch.zeros(2, **i32), torch.tensor([1, 1], **i32), 2)
    assert A.flags() == kvq.FLAG_BAD_PAGE and slots.tolist() == [-1, 0]
    A = DevicePageAllocator(4, 1, 2, 2)
    A.held.fill_(2)  # as if both rows held pages that the ring still has
    A.assign(torch.zeros(2, **i32), torch.zeros(2, **i32), 0)
    assert A.flags() == kvq.FLAG_BAD_PAGE and A.free_ring.tolist() == [0, 4]


def test_captured_steps():
    """A graph of one decode step, replayed, walks on from the state it finds."""
    i32 = dict(dtype=torch.int32, device=DEV)
    A, B = DevicePageAllocator(64, 1, 3, 20), DevicePageAllocator(64, 1, 3, 20)
    la, lb = (torch.tensor([0, 31, 64], **i32) for _ in range(2))
    one = torch.ones(3, **i32)
    cu, slots, pos = A.assign(la, one, 3)  # before capture: pages of the first tokens
    B.assign(lb, one, 3)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            A.assign(la, one, cu=cu, slots=slots, pos=pos)
            la += 1
    torch.cuda.synchronize()
    for _ in range(70):
        g.replay()
        _, want, wpos = B.assign(lb, one, 3)
        lb += 1
        torch.cuda.synchronize()
        assert torch.equal(slots, want) and torch.equal(pos, wpos)
        assert torch.equal(A.table, B.table)
