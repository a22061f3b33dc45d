"""GPU: decode behind shared prefixes (kvq_prefix_decode_attn, paged and
contiguous) against a plain fp64 attention over the oracle's dequantized keys
and values.

Error bound, per output coordinate: with A = sum_t p_t |v_hat_t| and
D = max_t sum_i |q_i k_hat_i| / sqrt(128), an error of at most d in each logit
and a relative error of at most e in each weight change the output by at most
((exp(2 d) - 1) + e) A, and storing it adds half a step u of its type times |o|.
bf16 outputs: the query rows and the weights are rounded to fp16 once, d = 2^-11
D and e = 2^-11. fp16 and fp32 outputs: both are pairs of fp16 terms (22 bits);
what is left is fp32 arithmetic: d = 2^-19 D (an inner product of 8 tensor-core
steps, each good to 2^-23, scaling, exponential), e = 2^-22 + n 2^-24 / 4 (sums
of n weights, four to a lane). 2^-15 A covers weights below fp16's normal range
(at most 2^-25 each where the largest is 2^6 or more). The rotation inside width
groups (k_rot) mixes coordinates: there D is bounded by |q a| |k / a|.
"""
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
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def dev_bf16(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).to(DEV)


class Setup:
    """Plans, and the same tokens as oracle heads and as device rows."""

    def __init__(self, seed, n_kv, bits_k, bits_v, rotate=False):
        self.rng = np.random.default_rng(seed)
        mode = kvq.ALLOC_ROTATE_KEYS if rotate else 0
        self.rotate, self.n_kv = rotate, n_kv
        self.cfg = kvq.make_cfg(n_kv, bits_k, bits_v, v_seed=11, alloc_mode=mode)
        self.E = np.exp(self.rng.standard_normal((n_kv, 64)) - np.arange(64) / 6.0)
        self.plans = kvq.plan_build(self.cfg, 1, self.E)

    def tokens(self, n):
        sig = np.sqrt(np.concatenate([self.E, self.E], axis=1) / 2)
        kb = synth.to_bf16_bits(self.rng.standard_normal((n, self.n_kv, 128)) * sig[None])
        return kb, synth.to_bf16_bits(self.rng.standard_normal((n, self.n_kv, 128)))

    def heads(self, kb, vb):
        """[(k_hat, v_hat)] per KV head, fp64 [n, 128]."""
        if len(kb) == 0:
            return [(np.zeros((0, 128)), np.zeros((0, 128)))] * self.n_kv
        kh, vh = op.bf16_heads(kb, vb)
        _, hs = op.layer(kh, vh, self.cfg.bits_k, self.cfg.bits_v, 11, 1, E=self.E, pack=False,
                         rotate_keys=self.rotate)
        return [(h["khat"], h["vhat"]) for h in hs]

    def a_hat(self, h):
        return np.tile(self.plans[h]["a_hat"].astype(np.float64), 2)


def reference(S, q, pre, own, group_of, dtype):
    """fp64 outputs [B, n_q, 128] and the error bound of each coordinate."""
    B, n_q = q.shape[:2]
    G = n_q // S.n_kv
    out, tol = np.zeros((B, n_q, 128)), np.zeros((B, n_q, 128))
    for b in range(B):
        for h in range(S.n_kv):
            parts = ([pre[group_of[b]][h]] if group_of[b] is not None else []) + [own[b][h]]
            k, v = (np.concatenate([x[i] for x in parts]) for i in (0, 1))
            if not len(k):
                continue
            for g in range(h * G, (h + 1) * G):
                s = k @ q[b, g] / np.sqrt(128)
                p = np.exp(s - s.max())
                p /= p.sum()
                out[b, g] = p @ v
                A = p @ np.abs(v)
                if S.rotate:
                    a = np.where(S.a_hat(h) > 0, S.a_hat(h), 1.0)
                    D = np.linalg.norm(q[b, g] * a) * np.linalg.norm(k / a, axis=1).max()
                else:
                    D = (np.abs(k) @ np.abs(q[b, g])).max()
                D /= np.sqrt(128)
                if dtype == torch.bfloat16:
                    d, e = 2.0 ** -11 * D, 2.0 ** -11
                else:
                    d, e = 2.0 ** -19 * D, 2.0 ** -22 + len(k) * 2.0 ** -26
                tol[b, g] = U[dtype] * np.abs(out[b, g]) + (np.expm1(2 * d) + e + 2.0 ** -15) * A
    return out, tol


def check(got, ref, tol):
    err = np.abs(got.double().cpu().numpy() - ref)
    assert np.all(np.isfinite(err))
    assert np.all(err <= tol), float((err / np.where(tol > 0, tol, 1e-300)).max())


def group_of(start, B):
    out = [None] * B
    for g, (a, b) in enumerate(zip(start, start[1:])):
        for i in range(a, b):
            out[i] = g
    return out


def contiguous(S, lens, data, extra=40):
    L = PackedLayer(S.cfg, len(lens), max(max(lens), 1) + extra, layer=1)
    L.set_plans(S.plans)
    for b, (kb, vb) in enumerate(data):
        if len(kb):
            kvq.quantize_append(S.cfg, L.plan_ptrs[b:b + 1], dev_bf16(kb)[None], dev_bf16(vb)[None],
                                L.cache_ptrs[b:b + 1], L.lens[b:b + 1], L.cap, L.status)
    return L


def paged(S, lens, data, page_tiles):
    span = 32 * page_tiles
    need = [-(-n // span) for n in lens]
    n_pages, wide = sum(need) + 3, max(max(need), 1) + 1
    A = DevicePageAllocator(n_pages, page_tiles, len(lens), wide)
    perm = torch.from_numpy(S.rng.permutation(n_pages).astype(np.int32))
    A.free_ids.copy_(perm)  # pages interleave in the pool
    P = PagedLayer(S.cfg, len(lens), n_pages, page_tiles, wide, layer=1, pages=A)
    P.set_plans(S.plans)
    cu, slots, _ = P.assign(torch.tensor(lens, dtype=torch.int32, device=DEV), sum(lens))
    k, v = (dev_bf16(np.concatenate([x[i] for x in data])) for i in (0, 1))
    P.append_ragged(k, v, cu, slots)
    assert A.flags() == 0
    return P


CASES = [
    # bits_k, bits_v, n_kv, G, prefix lengths, group starts, own lengths, page_tiles, dtype
    (2, 2, 1, 4, [257], [0, 2], [20, 0], 1, torch.float32),
    (3, 2, 2, 7, [1000], [0, 5], [1, 31, 32, 33, 300], 4, torch.bfloat16),
    (3, 3, 2, 8, [128, 0, 129], [0, 2, 3, 6], [127, 128, 129, 0, 5, 260], 2, torch.bfloat16),
    (1, 1, 1, 16, [700], [0, 12], [7 * i for i in range(12)], 1, torch.bfloat16),
    (8, 8, 1, 2, [333], [0, 3], [64, 65, 1], 2, torch.float16),
    (4, 5, 3, 1, [1, 95], [1, 1, 3], [10, 0, 40, 3], 1, torch.float32),  # rows 0, 3: no prefix
    (5, 6, 1, 5, [500], [0, 40], [(13 * i) % 90 for i in range(40)], 1, torch.bfloat16),
    (6, 4, 2, 8, [400], [0, 33], [(29 * i) % 70 for i in range(33)], 2, torch.float16),
    (7, 3, 1, 3, [0], [0, 3], [0, 1, 45], 1, torch.bfloat16),
]


@pytest.mark.parametrize("bk,bv,n_kv,G,pre,start,own,page_tiles,dtype", CASES)
def test_against_fp64(bk, bv, n_kv, G, pre, start, own, page_tiles, dtype):
    S = Setup(bk * 100 + bv, n_kv, bk, bv)
    B = len(own)
    pd, od = [S.tokens(n) for n in pre], [S.tokens(n) for n in own]
    q = torch.from_numpy(S.rng.standard_normal((B, n_kv * G, 128))).to(dtype)
    ref, tol = reference(S, q.double().numpy(), [S.heads(*x) for x in pd],
                         [S.heads(*x) for x in od], group_of(start, B), dtype)
    gs = torch.tensor(start, dtype=torch.int32, device=DEV)
    P, Q = contiguous(S, pre, pd), contiguous(S, own, od)
    got = Q.decode_prefix(q.to(DEV), P, gs)
    check(got, ref, tol)
    assert got.dtype == dtype and Q.flags() == 0
    PP, QQ = paged(S, pre, pd, page_tiles), paged(S, own, od, page_tiles)
    again = QQ.decode_prefix(q.to(DEV), PP, gs)
    assert torch.equal(again, got)  # where the tokens lie does not matter
    assert QQ.flags() == 0 and QQ.lens.cpu().tolist() == own


@pytest.mark.parametrize("q_dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_types(q_dtype, out_dtype):
    S = Setup(3, 1, 3, 3)
    pd, od = [S.tokens(150)], [S.tokens(n) for n in (9, 70)]
    q = torch.from_numpy(S.rng.standard_normal((2, 6, 128))).to(q_dtype)
    ref, tol = reference(S, q.double().numpy(), [S.heads(*x) for x in pd],
                         [S.heads(*x) for x in od], [0, 0], out_dtype)
    out = torch.empty(2, 6, 128, dtype=out_dtype, device=DEV)
    gs = torch.tensor([0, 2], dtype=torch.int32, device=DEV)
    contiguous(S, [9, 70], od).decode_prefix(q.to(DEV), contiguous(S, [150], pd), gs, out=out)
    check(out, ref, tol)
    if out_dtype == torch.float32:  # independent roundings add as their root
        err = np.linalg.norm(out.double().cpu().numpy() - ref) / np.linalg.norm(ref)
        assert err <= 2e-5, err


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rotated_keys(dtype):
    S = Setup(5, 2, 3, 4, rotate=True)
    pd, od = [S.tokens(300)], [S.tokens(n) for n in (33, 0, 129)]
    q = torch.from_numpy(S.rng.standard_normal((3, 8, 128))).to(dtype)
    ref, tol = reference(S, q.double().numpy(), [S.heads(*x) for x in pd],
                         [S.heads(*x) for x in od], [0, 0, 0], dtype)
    gs = torch.tensor([0, 3], dtype=torch.int32, device=DEV)
    got = contiguous(S, [33, 0, 129], od).decode_prefix(q.to(DEV), contiguous(S, [300], pd), gs)
    check(got, ref, tol)


@pytest.mark.parametrize("scale", [1e-20, 6.0, 40.0])
def test_sharp_logits_and_uneven_value_norms(scale):
    """Logits from nearly equal to one that takes all; values whose norms differ
    by 10^4, so that the softmax reference moves within and between tiles."""
    S = Setup(6, 1, 4, 4)
    pre, own = 900, [300, 2]
    pd, od = [S.tokens(pre)], [S.tokens(n) for n in own]

    def scaled(d):
        kb, vb = d
        f = 10.0 ** S.rng.uniform(-2, 2, (len(vb), 1, 1))
        return kb, synth.to_bf16_bits(synth.bf16_bits_to_f64(vb) * f)
    pd, od = [scaled(x) for x in pd], [scaled(x) for x in od]
    q = torch.from_numpy(S.rng.standard_normal((2, 4, 128)) * scale).float()
    gs = torch.tensor([0, 2], dtype=torch.int32, device=DEV)
    P, Q = contiguous(S, [pre], pd), contiguous(S, own, od)
    for dtype in (torch.bfloat16, torch.float32):
        ref, tol = reference(S, q.double().numpy(), [S.heads(*x) for x in pd],
                             [S.heads(*x) for x in od], [0, 0], dtype)
        out = torch.empty(2, 4, 128, dtype=dtype, device=DEV)
        Q.decode_prefix(q.to(DEV), P, gs, out=out)
        check(out, ref, tol)


def test_same_as_one_cache_per_sequence():
    """Prefix and own tokens in one cache give the framework's decode (within the
    two calls' bounds: 2e-3 for kvq_decode_attn)."""
    S = Setup(7, 2, 3, 3)
    pre, own = 513, [40, 1, 200]
    pd, od = S.tokens(pre), [S.tokens(n) for n in own]
    whole = [tuple(np.concatenate([pd[i], x[i]]) for i in (0, 1)) for x in od]
    q = torch.from_numpy(S.rng.standard_normal((3, 16, 128))).to(torch.bfloat16).to(DEV)
    gs = torch.tensor([0, 3], dtype=torch.int32, device=DEV)
    out = torch.empty(3, 16, 128, dtype=torch.float32, device=DEV)
    contiguous(S, own, od).decode_prefix(q, contiguous(S, [pre], [pd]), gs, out=out)
    one = contiguous(S, [pre + n for n in own], whole).decode(q)
    assert op.rel_err(out.cpu().numpy(), one.cpu().numpy()) <= 4e-3


def test_many_rows_and_a_dirty_workspace_and_repeats():
    """More than 256 rows per KV head (several row tiles, a sequence's heads over
    two of them), a workspace full of NaN bytes, the same bits on every run."""
    S = Setup(8, 1, 3, 2)
    B, G = 61, 7
    own = [(11 * i) % 50 for i in range(B)]
    pd, od = [S.tokens(640), S.tokens(35)], [S.tokens(n) for n in own]
    start = [0, 55, 61]
    q = torch.from_numpy(S.rng.standard_normal((B, G, 128))).to(torch.bfloat16)
    ref, tol = reference(S, q.double().numpy(), [S.heads(*x) for x in pd],
                         [S.heads(*x) for x in od], group_of(start, B), torch.bfloat16)
    gs = torch.tensor(start, dtype=torch.int32, device=DEV)
    P, Q = contiguous(S, [640, 35], pd), contiguous(S, own, od)
    ws = prefix_workspace(S.cfg, B, G, 2).fill_(0xFF)
    first = Q.decode_prefix(q.to(DEV), P, gs, ws=ws)
    check(first, ref, tol)
    for _ in range(5):
        assert torch.equal(Q.decode_prefix(q.to(DEV), P, gs, ws=ws), first)
    f32 = torch.empty(B, G, 128, dtype=torch.float32, device=DEV)
    Q.decode_prefix(q.to(DEV), P, gs, ws=ws, out=f32)
    ref, tol = reference(S, q.double().numpy(), [S.heads(*x) for x in pd],
                         [S.heads(*x) for x in od], group_of(start, B), torch.float32)
    check(f32, ref, tol)
    # a smaller call on the same workspace, then the first again
    Q2 = contiguous(S, own[:3], od[:3])
    Q2.decode_prefix(q[:3].to(DEV), P, torch.tensor([0, 1, 3], dtype=torch.int32, device=DEV),
                     ws=ws)
    assert torch.equal(Q.decode_prefix(q.to(DEV), P, gs, ws=ws), first)


def test_nan_query_row_stays_alone():
    S = Setup(9, 1, 3, 3)
    pd, od = [S.tokens(200)], [S.tokens(n) for n in (10, 20)]
    q = torch.from_numpy(S.rng.standard_normal((2, 4, 128))).to(torch.bfloat16)
    gs = torch.tensor([0, 2], dtype=torch.int32, device=DEV)
    P, Q = contiguous(S, [200], pd), contiguous(S, [10, 20], od)
    clean = Q.decode_prefix(q.to(DEV), P, gs)
    for bad in (float("nan"), float("inf")):
        q2 = q.clone()
        q2[0, 1, 5] = bad
        got = Q.decode_prefix(q2.to(DEV), P, gs)
        assert torch.isnan(got[0, 1]).all()
        keep = torch.ones(2, 4, dtype=torch.bool)
        keep[0, 1] = False
        assert torch.equal(got[keep], clean[keep])


def test_flags():
    S = Setup(10, 1, 3, 3)
    pd, od = [S.tokens(100)], [S.tokens(n) for n in (40, 50)]
    q = torch.randn(2, 4, 128, device=DEV, dtype=torch.bfloat16)
    P, Q = paged(S, [100], pd, 1), paged(S, [40, 50], od, 1)

    def run(start, **kw):
        Q.status.zero_()
        out = Q.decode_prefix(q, P, torch.tensor(start, dtype=torch.int32, device=DEV), **kw)
        assert torch.isfinite(out.float()).all()
        return Q.flags()
    assert run([0, 2]) == 0
    assert run([0, 3]) == kvq.FLAG_BAD_PAGE  # past the batch
    assert run([2, 1]) == kvq.FLAG_BAD_PAGE  # descending
    assert run([-1, 2]) == kvq.FLAG_BAD_PAGE
    assert run([0, 2], max_prefix_len=64) == kvq.FLAG_CAPACITY
    assert run([0, 2], max_len=45) == kvq.FLAG_CAPACITY
    saved = Q.table.clone()
    Q.table[1, 1] = Q.n_pages  # outside the pool: placeholder bytes, flagged
    assert run([0, 2]) == kvq.FLAG_BAD_PAGE
    Q.table[1, 1] = -5
    assert run([0, 2]) == kvq.FLAG_BAD_PAGE
    Q.table.copy_(saved)
    lens = Q.lens.clone()
    Q.lens[1] = Q.cap  # pages it does not hold (-1)
    assert run([0, 2]) == kvq.FLAG_BAD_PAGE
    Q.lens[1] = -7  # a negative length is an empty sequence
    assert run([0, 2]) == 0
    Q.lens.copy_(lens)
    plans = Q.plans.clone()
    Q.plans[0] ^= 1  # magic
    assert run([0, 2]) & kvq.FLAG_BAD_PLAN
    Q.plans.copy_(plans)
    assert run([0, 2]) == 0


def test_other_value_signs_are_flagged():
    S = Setup(12, 1, 3, 3)
    T = Setup(12, 1, 3, 3)
    T.plans = T.plans.copy()
    T.plans["v_sign"][0, 0] ^= 1
    od = [S.tokens(20), S.tokens(20)]
    Q, R = contiguous(S, [20, 20], od), contiguous(T, [20, 20], od)
    Q.plan_ptrs[1] = R.plan_ptrs[1]
    q = torch.randn(2, 4, 128, device=DEV, dtype=torch.bfloat16)
    Q.decode_prefix(q, contiguous(S, [60], [S.tokens(60)]),
                    torch.tensor([0, 2], dtype=torch.int32, device=DEV))
    assert Q.flags() == kvq.FLAG_BAD_PLAN


def test_graph_replay_follows_lengths_and_two_streams():
    S = Setup(13, 2, 3, 2)
    pre, own = [300], [60, 5, 90]
    pd, od = [S.tokens(n) for n in pre], [S.tokens(n) for n in own]
    P, Q = contiguous(S, pre, pd), contiguous(S, own, od)
    gs = torch.tensor([0, 3], dtype=torch.int32, device=DEV)
    q = torch.from_numpy(S.rng.standard_normal((3, 8, 128))).to(torch.bfloat16).to(DEV)
    out = torch.empty_like(q)
    ws = prefix_workspace(S.cfg, 3, 8, 1)
    Q.decode_prefix(q, P, gs, out=out, ws=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            Q.decode_prefix(q, P, gs, out=out, ws=ws)
    for lens, plen in (([60, 5, 90], 300), ([10, 0, 33], 129), ([0, 0, 0], 1)):
        Q.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        P.lens.fill_(plen)
        g.replay()
        got = out.clone()
        want = Q.decode_prefix(q, P, gs)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    # two streams, a workspace each
    want = Q.decode_prefix(q, P, gs).clone()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    wa, wb = (prefix_workspace(S.cfg, 3, 8, 1) for _ in range(2))
    oa, ob = torch.empty_like(q), torch.empty_like(q)
    torch.cuda.synchronize()
    for _ in range(10):
        with torch.cuda.stream(a):
            Q.decode_prefix(q, P, gs, out=oa, ws=wa)
        with torch.cuda.stream(b):
            Q.decode_prefix(q, P, gs, out=ob, ws=wb)
    torch.cuda.synchronize()
    assert torch.equal(oa, want) and torch.equal(ob, want) and Q.flags() == 0


def test_pages_past_four_gigabytes():
    S = Setup(14, 1, 3, 3)
    tb = kvq.page_bytes(S.cfg, 1)
    n_pages = (5 << 30) // tb
    pd, od = [S.tokens(200)], [S.tokens(n) for n in (70, 3)]
    near = paged(S, [200], pd, 1), paged(S, [70, 3], od, 1)
    q = torch.from_numpy(S.rng.standard_normal((2, 8, 128))).to(torch.bfloat16).to(DEV)
    gs = torch.tensor([0, 2], dtype=torch.int32, device=DEV)
    want = near[1].decode_prefix(q, near[0], gs)
    far = []
    for data, lens in ((pd, [200]), (od, [70, 3])):
        need = [-(-n // 32) for n in lens]
        A = DevicePageAllocator(n_pages, 1, len(lens), max(need))
        A.free_ids.copy_(torch.arange(n_pages - 1, -1, -1, dtype=torch.int32))
        if not far:
            L = PagedLayer(S.cfg, len(lens), n_pages, 1, max(need), layer=1, pages=A)
        else:
            L = PagedLayer(S.cfg, len(lens), n_pages, 1, max(need), layer=1, pages=A)
        L.set_plans(S.plans)
        cu, slots, _ = L.assign(torch.tensor(lens, dtype=torch.int32, device=DEV), sum(lens))
        assert int(slots.min()) * tb > 32 * 2 ** 32
        k, v = (dev_bf16(np.concatenate([x[i] for x in data])) for i in (0, 1))
        L.append_ragged(k, v, cu, slots)
        far.append(L)
    assert torch.equal(far[1].decode_prefix(q, far[0], gs), want) and far[1].flags() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_query_at_an_odd_address_and_output_in_its_place(dtype):
    S = Setup(23, 2, 3, 3)
    pre, own = [200], [40, 0, 131]
    P, Q = contiguous(S, pre, [S.tokens(200)]), contiguous(S, own, [S.tokens(n) for n in own])
    gs = torch.tensor([0, 3], dtype=torch.int32, device=DEV)
    q = torch.from_numpy(S.rng.standard_normal((3, 8, 128))).to(dtype).to(DEV)
    want = Q.decode_prefix(q, P, gs)
    odd = torch.empty(q.numel() + 1, dtype=dtype, device=DEV)[1:].view(q.shape)
    odd.copy_(q)
    assert odd.data_ptr() % 16 != 0
    assert torch.equal(Q.decode_prefix(odd, P, gs, out=torch.empty_like(q)), want)
    with pytest.raises(kvq.KVQError):  # outputs are stored 16 bytes at a time
        Q.decode_prefix(q, P, gs, out=odd)
    for _ in range(5):
        x = q.clone()
        assert torch.equal(Q.decode_prefix(x, P, gs, out=x), want)
    assert Q.flags() == 0


def test_short_pointer_arrays_are_refused():
    S = Setup(29, 1, 2, 2)
    P, Q = contiguous(S, [40], [S.tokens(40)]), contiguous(S, [5, 6], [S.tokens(5), S.tokens(6)])
    gs = torch.tensor([0, 2], dtype=torch.int32, device=DEV)
    q = torch.zeros(2, 4, 128, dtype=torch.bfloat16, device=DEV)
    ws = prefix_workspace(S.cfg, 2, 4, 1)
    for plans, pre, own in ((Q.plan_ptrs[:1], P.cache_ptrs, Q.cache_ptrs),
                            (Q.plan_ptrs, P.cache_ptrs[:0], Q.cache_ptrs),
                            (Q.plan_ptrs, P.cache_ptrs, Q.cache_ptrs[:1])):
        with pytest.raises(kvq.KVQError):
            kvq.prefix_decode_attn(S.cfg, plans, pre, P.lens, gs, P.cap, own, Q.lens, Q.cap, q,
                                   torch.empty_like(q), ws, Q.status)
