"""GPU: kvq_paged_append_ragged, the quantize-append of a packed ragged batch
through slot maps: records bit for bit those of kvq_paged_quantize_append and of
the oracle; refused and bad slots; and a serving loop (assign, append, decode
behind a shared prefix) in a captured graph."""
import numpy as np
import pytest
import torch

import oracle_pipeline as op
import synth
from bit_kv_cache_19_b200 import kvq
from bit_kv_cache_19_b200.runtime import (DevicePageAllocator, PackedLayer, PagedLayer,
                                          prefix_workspace)

pytestmark = pytest.mark.gpu
DEV = "cuda"
I32 = dict(dtype=torch.int32, device=DEV)


def layer(cfg, plans, batch, page_tiles, max_pages, n_pages=None):
    n_pages = n_pages or batch * max_pages
    A = DevicePageAllocator(n_pages, page_tiles, batch, max_pages)
    A.free_ids.copy_(torch.randperm(n_pages, generator=torch.Generator().manual_seed(3)))
    P = PagedLayer(cfg, batch, n_pages, page_tiles, max_pages, layer=2, pages=A)
    P.set_plans(plans)
    return P


def rows(rng, n, n_kv, E, dtype):
    sig = np.sqrt(np.concatenate([E, E], axis=1) / 2)
    k = torch.from_numpy(rng.standard_normal((n, n_kv, 128)) * sig).to(DEV).to(dtype)
    return k, torch.from_numpy(rng.standard_normal((n, n_kv, 128))).to(DEV).to(dtype)


def setup(seed, n_kv, bk, bv, mode=0):
    rng = np.random.default_rng(seed)
    cfg = kvq.make_cfg(n_kv, bk, bv, v_seed=4, alloc_mode=mode)
    E = np.exp(rng.standard_normal((n_kv, 64)) - np.arange(64) / 7.0)
    return rng, cfg, E, kvq.plan_build(cfg, 2, E)


@pytest.mark.parametrize("bk,bv,n_kv,dtype,page_tiles,mode,rope", [
    (3, 2, 4, torch.bfloat16, 4, 0, 0.0),
    (3, 3, 2, torch.float16, 1, 0, 0.0),
    (5, 6, 3, torch.float32, 2, 0, 0.0),
    (2, 2, 1, torch.bfloat16, 1, kvq.ALLOC_ROTATE_KEYS, 0.0),
    (8, 8, 1, torch.bfloat16, 2, 0, 0.0),
    (1, 1, 2, torch.bfloat16, 1, kvq.ALLOC_UNIFORM, 0.0),
    (3, 3, 2, torch.bfloat16, 2, 0, 1e6),
    (4, 7, 1, torch.float32, 1, kvq.ALLOC_ROTATE_KEYS, 1e4)])
def test_equals_the_padded_append(bk, bv, n_kv, dtype, page_tiles, mode, rope):
    rng, cfg, E, plans = setup(bk * 10 + bv, n_kv, bk, bv, mode)
    B = 9
    steps = [[0, 1, 31, 32, 33, 64, 65, 200, 5], [1] * B, [3, 0, 0, 40, 31, 1, 63, 64, 129],
             [0] * B, [0, 95, 1, 0, 0, 0, 0, 0, 2]]
    P = layer(cfg, plans, B, page_tiles, 16)
    Q = PagedLayer(cfg, B, B * 16, page_tiles, 16, layer=2)  # host pages, one call per sequence
    Q.set_plans(plans)
    want = np.zeros(B, np.int64)
    for n_new in steps:
        total = sum(n_new)
        k, v = rows(rng, total + 3, n_kv, E, dtype)
        k[total:] = float("nan")  # rows behind the last sequence are not read
        cu, slots, _ = P.assign(torch.tensor(n_new, **I32), total + 3)
        P.append_ragged(k, v, cu, slots, rope)
        at = 0
        for b, n in enumerate(n_new):
            want[b] += n
            if n:
                Q.reserve(b, int(want[b]))
                pg = kvq.Pages(Q.pool.data_ptr(), Q.table.data_ptr() + 4 * b * Q.table.shape[1],
                               Q.n_pages, page_tiles, Q.table.shape[1])
                kvq.paged_quantize_append(cfg, Q.plan_ptrs[b:b + 1], k[None, at:at + n],
                                          v[None, at:at + n], pg, Q.lens[b:b + 1], Q.status, rope)
            at += n
        assert P.lens.cpu().tolist() == want.tolist() == Q.lens.cpu().tolist()
    assert P.flags() == 0 and Q.flags() == 0 and P.dev_pages.flags() == 0
    for b in range(B):
        for h in range(n_kv):
            n_tiles = -(-int(want[b]) // 32)
            assert np.array_equal(P.head_records(b, h, n_tiles), Q.head_records(b, h, n_tiles))


def test_against_the_oracle():
    rng, cfg, E, plans = setup(77, 2, 3, 3)
    lens = [70, 0, 33]
    data = [(synth.to_bf16_bits(rng.standard_normal((n, 2, 128)) *
                                np.sqrt(np.concatenate([E, E], 1) / 2)),
             synth.to_bf16_bits(rng.standard_normal((n, 2, 128)))) for n in lens]
    P = layer(cfg, plans, 3, 1, 4)
    k, v = (torch.from_numpy(np.concatenate([d[i] for d in data]).view(np.int16)).view(
        torch.bfloat16).to(DEV) for i in (0, 1))
    cu, slots, pos = P.assign(torch.tensor(lens, **I32), sum(lens))
    P.append_ragged(k, v, cu, slots)
    assert pos.tolist() == [t for n in lens for t in range(n)]
    for b, n in enumerate(lens):
        if not n:
            continue
        kh, vh = op.bf16_heads(*data[b])
        _, heads = op.layer(kh, vh, 3, 3, 4, 2, E=E)
        for h in range(2):
            nw = 128 * 6
            assert np.array_equal(P.head_records(b, h, -(-n // 32))[:, :nw],
                                  heads[h]["rec"][:, :nw])
            got = P.head_records(b, h, -(-n // 32)).view(np.float16).reshape(-1, 2 * nw + 64)
            assert np.array_equal(got[:, 2 * nw:2 * nw + 32].reshape(-1)[:n],
                                  heads[h]["knorm"].astype(np.float16))


def test_refused_and_bad_slots():
    rng, cfg, E, plans = setup(5, 2, 3, 2)
    P = layer(cfg, plans, 4, 1, 3)
    n_new = torch.tensor([40, 20, 200, 10], **I32)  # the third does not fit its row
    k, v = rows(rng, 270, 2, E, torch.bfloat16)
    cu, slots, _ = P.assign(n_new, 270)
    assert P.dev_pages.flags() == kvq.FLAG_CAPACITY
    before = P.pool.clone()
    P.append_ragged(k, v, cu, slots)
    assert P.flags() == 0 and P.lens.tolist() == [40, 20, 0, 10]
    assert not torch.equal(P.pool, before)

    def run(change, flag, lens=None):
        P.lens.copy_(torch.tensor([40, 20, 0, 10], **I32))
        P.status.zero_()
        c, s = cu.clone(), slots.clone()
        change(c, s)
        pool = P.pool.clone()
        P.append_ragged(k, v, c, s)
        assert P.flags() == flag, P.flags()
        P.lens.copy_(torch.tensor([0] * 4, **I32))
        return torch.equal(P.pool, pool)

    def none(c, s):
        s.fill_(-1)
    assert run(none, 0)

    def outside(c, s):
        s.fill_(10 ** 12)
    P.lens.zero_()
    assert run(outside, kvq.FLAG_BAD_PAGE)

    def negative(c, s):
        s.fill_(-2)
    assert run(negative, kvq.FLAG_BAD_PAGE)

    def cu_past(c, s):
        c.copy_(torch.tensor([0, 5000, 5000, 5000, 5000], **I32))
        s.fill_(-1)
    assert run(cu_past, kvq.FLAG_CAPACITY)

    def cu_negative(c, s):
        c.copy_(torch.tensor([-5, 3, 3, 3, 3], **I32))
        s.fill_(-1)
    assert run(cu_negative, kvq.FLAG_CAPACITY)


def test_length_that_is_not_the_slots():
    rng, cfg, E, plans = setup(6, 1, 3, 3)
    P = layer(cfg, plans, 1, 1, 3)
    k, v = rows(rng, 10, 1, E, torch.bfloat16)
    cu, slots, _ = P.assign(torch.tensor([10], **I32), 10)
    for rope in (0.0, 1e4):
        for bad, flag in ((5, kvq.FLAG_BAD_PAGE), (-32, kvq.FLAG_CAPACITY)):
            P.lens.fill_(bad)
            P.status.zero_()
            P.append_ragged(k, v, cu, slots, rope)
            assert P.flags() == flag and P.lens.tolist() == [bad]


def test_bad_plan_and_non_finite_tokens():
    rng, cfg, E, plans = setup(8, 2, 3, 3)
    P = layer(cfg, plans, 2, 1, 3)
    k, v = rows(rng, 50, 2, E, torch.bfloat16)
    k[7, 1, 3] = float("nan")
    cu, slots, _ = P.assign(torch.tensor([20, 30], **I32), 50)
    P.append_ragged(k, v, cu, slots)
    assert P.flags() == kvq.FLAG_NONFINITE
    P.status.zero_()
    P.lens.zero_()
    P.plans[0] ^= 1
    pool = P.pool.clone()
    P.append_ragged(k[:, :, :], v, cu, slots)
    assert P.flags() & kvq.FLAG_BAD_PLAN
    head0 = P.pool.view(-1, 2, kvq.tile_bytes(cfg))[:, 0]
    assert torch.equal(head0, pool.view(-1, 2, kvq.tile_bytes(cfg))[:, 0])


def test_serving_loop_in_a_graph():
    """Assign, append and decode behind a shared prefix, captured once and replayed
    step by step, against one contiguous cache per sequence and eager calls."""
    rng, cfg, E, plans = setup(9, 2, 3, 3)
    B, n_q, pre = 3, 8, 150
    kp, vp = rows(rng, pre, 2, E, torch.bfloat16)
    X = layer(cfg, plans, 1, 2, 4)
    cu, slots, _ = X.assign(torch.tensor([pre], **I32), pre)
    X.append_ragged(kp, vp, cu, slots)
    P = layer(cfg, plans, B, 2, 4)
    gs = torch.tensor([0, B], **I32)
    n_new = torch.tensor([1, 0, 2], **I32)
    k, v = rows(rng, 3, 2, E, torch.bfloat16)
    q = torch.randn(B, n_q, 128, device=DEV, dtype=torch.bfloat16)
    out, ws = torch.empty(B, n_q, 128, device=DEV), prefix_workspace(cfg, B, n_q, 1)
    bufs = dict(cu=torch.empty(B + 1, **I32), pos=torch.empty(3, **I32),
                slots=torch.empty(3, dtype=torch.int64, device=DEV))

    def step():
        cu, slots, _ = P.assign(n_new, **bufs)
        P.append_ragged(k, v, cu, slots)
        P.decode_prefix(q, X, gs, out=out, ws=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()  # the first step eagerly
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step()
    torch.cuda.synchronize()
    C = PackedLayer(cfg, B, 400, layer=2)
    C.set_plans(plans)
    C.append(kp[None].expand(B, -1, -1, -1).contiguous(), vp[None].expand(B, -1, -1, -1).contiguous())
    first = True
    for i in range(45):
        if not first:
            k2, v2 = rows(rng, 3, 2, E, torch.bfloat16)
            k.copy_(k2)
            v.copy_(v2)
            n = [int(x) for x in rng.multinomial(3, [0.3, 0.3, 0.4])]
            n_new.copy_(torch.tensor(n, **I32))
            g.replay()
        else:
            n = [1, 0, 2]
        at = 0
        for b in range(B):
            if n[b]:
                kvq.quantize_append(cfg, C.plan_ptrs[b:b + 1], k[None, at:at + n[b]],
                                    v[None, at:at + n[b]], C.cache_ptrs[b:b + 1],
                                    C.lens[b:b + 1], C.cap, C.status)
            at += n[b]
        want = C.decode(q)
        torch.cuda.synchronize()
        # kvq_decode_attn is good to 2e-3; the prefix call's fp32 output far below
        assert op.rel_err(out.cpu().numpy(), want.cpu().numpy()) <= 2.5e-3
        assert (C.lens - pre).tolist() == P.lens.tolist()
        first = False
    assert P.flags() == 0 and P.dev_pages.flags() == 0 and C.flags() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_rows_at_an_odd_address(dtype):
    rng, cfg, E, plans = setup(31, 2, 3, 2)
    n_new = [33, 0, 7]
    got = []
    for off in (0, 1):
        P = layer(cfg, plans, 3, 1, 4)
        if not off:
            k, v = rows(rng, 40, 2, E, dtype)
        else:
            k, v = (torch.cat([x.new_zeros(1), x.flatten()])[1:].view(x.shape) for x in (k, v))
            assert k.data_ptr() % 16 != 0 and v.data_ptr() % 16 != 0
        cu, slots, _ = P.assign(torch.tensor(n_new, **I32), 40)
        P.append_ragged(k, v, cu, slots)
        assert P.flags() == 0
        got.append(P.pool.clone())
    assert torch.equal(got[0], got[1])
