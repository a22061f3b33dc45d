"""GPU: kvq_paged_append_ragged on slots that a slot map cannot hold. Each case breaks
one rule only (lengths match, slots stay consecutive unless that is the rule) in a
pool that lies between guard pages: the tile concerned is skipped and flagged, every
other byte is that of the unbroken call, and the guards stay as they were.
"""
import numpy as np
import pytest
import torch

from bit_kv_cache_19_b200 import kvq

pytestmark = pytest.mark.gpu
DEV = "cuda"
I32 = dict(dtype=torch.int32, device=DEV)
N_NEW = [40, 33, 100, 10]  # a full tile and a part; a full tile and one row; ...
TILES, N_KV = 2, 2  # tiles per page
SPAN = 32 * TILES


class Pool:
    """Sequences of no tokens yet over n_pages pages with two guard pages on each side."""

    def __init__(self):
        rng = np.random.default_rng(3)
        self.cfg = kvq.make_cfg(N_KV, 3, 2, v_seed=4)
        plans = kvq.plan_build(self.cfg, 2, np.exp(rng.standard_normal((N_KV, 64))))
        self.plans = torch.from_numpy(np.frombuffer(plans.tobytes(), np.uint8).copy()).to(DEV)
        self.ptrs = kvq.ptr_array([self.plans] * len(N_NEW), DEV)
        need = [-(-n // SPAN) for n in N_NEW]
        self.n_pages = sum(need) + 1
        self.bytes = kvq.page_bytes(self.cfg, TILES)
        order = rng.permutation(self.n_pages)
        slots, at = [], 0
        for n, m in zip(N_NEW, need):
            slots += [int(order[at + t // SPAN]) * SPAN + t % SPAN for t in range(n)]
            at += m
        self.slots = torch.tensor(slots, dtype=torch.int64, device=DEV)
        self.cu = torch.tensor(np.cumsum([0] + N_NEW), **I32)
        self.k, self.v = (torch.from_numpy(rng.standard_normal((sum(N_NEW), N_KV, 128))).to(
            DEV).bfloat16() for _ in range(2))

    def append(self, slots, rope):
        """(every page with the guards [n_pages + 4, TILES, bytes per tile], lengths, flags)."""
        whole = torch.full(((self.n_pages + 4) * self.bytes,), 0xA5, dtype=torch.uint8, device=DEV)
        lens, status = torch.zeros(len(N_NEW), **I32), torch.zeros(1, **I32)
        kvq.paged_append_ragged(self.cfg, self.ptrs, self.k, self.v, self.cu, slots,
                                whole[2 * self.bytes:], self.n_pages, TILES, lens, status, rope)
        return (whole.view(self.n_pages + 4, TILES, -1).cpu(), lens.tolist(),
                int(status.item()))


def _shift(pages):
    def change(s, rows, pool):
        page = int(s[rows[0]]) // SPAN
        s[rows[0]:rows[1]] += (pages(pool) - page) * SPAN
    return change


def _swap(i, j):
    def change(s, rows, pool):
        s[rows[0] + i], s[rows[0] + j] = int(s[rows[0] + j]), int(s[rows[0] + i])
    return change


def _one(i, by):
    def change(s, rows, pool):
        s[rows[0] + i] += by
    return change


FIRST = (73, 105)  # the first tile of sequence 2, rows of the packed batch
LATER = (105, 137)  # its second tile
SINGLE = (72, 73)  # the second tile of sequence 1: one row
CASES = [
    ("page past the pool", FIRST, _shift(lambda p: p.n_pages)),
    ("page past the pool", LATER, _shift(lambda p: p.n_pages)),
    ("page past the pool", SINGLE, _shift(lambda p: p.n_pages + 1)),
    ("page far past the pool", LATER, _shift(lambda p: 1 << 40)),
    ("page before the pool", FIRST, _shift(lambda p: -1)),
    ("page before the pool", LATER, _shift(lambda p: -2)),
    ("page before the pool", SINGLE, _shift(lambda p: -2)),
    ("two slots exchanged", LATER, _swap(3, 4)),
    ("two slots exchanged", FIRST, _swap(1, 30)),
    ("one slot twice", LATER, _one(17, -1)),
    ("one slot of another tile", FIRST, _one(30, 32)),
    ("first slot repeated", LATER, _one(1, -1)),
    ("last slot", LATER, _one(31, 1)),
    ("another position in the tile", SINGLE, _one(0, 1)),
]


@pytest.mark.parametrize("rope", [0.0, 1e4])
@pytest.mark.parametrize("what,rows,change", CASES, ids=[f"{c[0]}-{c[1][0]}" for c in CASES])
def test_bad_slots_skip_their_tile_only(what, rows, change, rope):
    pool = Pool()
    want, lens, flags = pool.append(pool.slots, rope)
    assert flags == 0 and lens == N_NEW
    slot = int(pool.slots[rows[0]])  # the tile's right place stays as it was
    page, tile = 2 + slot // SPAN, slot % SPAN // 32
    assert not bool((want[page, tile] == 0xA5).all())
    want[page, tile] = 0xA5
    bad = pool.slots.clone()
    change(bad, rows, pool)
    got, lens, flags = pool.append(bad, rope)
    assert flags == kvq.FLAG_BAD_PAGE and lens == N_NEW
    assert torch.equal(got, want)
    assert bool((got[:2] == 0xA5).all()) and bool((got[-2:] == 0xA5).all())
