"""GPU: the shared-prefix decode at the ends of what its interface allows: more
prefixes than sequences in a workspace of exactly the size asked for, and the longest
context."""
import numpy as np
import pytest
import torch

import synth
from bit_kv_cache_19_b200 import kvq
from bit_kv_cache_19_b200.runtime import DevicePageAllocator, PagedLayer, prefix_workspace
from test_gpu_prefix_decode import (DEV, Setup, check, contiguous, dev_bf16, group_of,
                                    reference)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("end", [5, 4])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_many_empty_prefixes_in_an_exact_workspace(dtype, end):
    """1024 prefixes, of which five sequences use three: nothing is written past the
    workspace, which does not grow with the prefixes that no sequence has. end: with 4
    the last sequence lies behind every group."""
    S = Setup(51, 2, 3, 3)
    n_prefixes, own = 1024, [3, 40, 0, 70, 33]
    used = {7: 100, 500: 257, 1023: 31}  # prefix: tokens
    lens = [used.get(g, 0) for g in range(n_prefixes)]
    edge = {7: (0, 1), 500: (1, 3), 1023: (3, end)}
    start, at = [], 0
    for g in range(n_prefixes):
        start.append(edge[g][0] if g in edge else at)
        at = edge[g][1] if g in edge else at
    start.append(end)
    pd = {g: S.tokens(n) for g, n in used.items()}
    od = [S.tokens(n) for n in own]
    none = ([], [])
    P = contiguous(S, list(used.values()), list(pd.values()))
    Q = contiguous(S, own, od)
    caches = torch.zeros(n_prefixes, dtype=torch.int64, device=DEV)
    caches[list(used)] = P.cache_ptrs
    q = torch.from_numpy(S.rng.standard_normal((5, 14, 128))).to(dtype)
    out = torch.empty(5, 14, 128, dtype=dtype, device=DEV)
    need = kvq.prefix_decode_workspace_bytes(S.cfg, 5, 14, n_prefixes)
    room = torch.full((need + (1 << 20),), 0xEE, dtype=torch.uint8, device=DEV)
    kvq.prefix_decode_attn(
        S.cfg, Q.plan_ptrs, caches, torch.tensor(lens, dtype=torch.int32, device=DEV),
        torch.tensor(start, dtype=torch.int32, device=DEV), 300, Q.cache_ptrs, Q.lens, Q.cap,
        q.to(DEV), out, room[:need], Q.status)
    assert Q.flags() == 0 and bool((room[need:] == 0xEE).all())
    heads = [S.heads(*pd.get(g, none)) for g in range(n_prefixes)]
    ref, tol = reference(S, q.double().numpy(), heads, [S.heads(*x) for x in od],
                         group_of(start, 5), dtype)
    check(out, ref, tol)


@pytest.mark.parametrize("shared", [False, True])
def test_longest_context(shared):
    """2^31 - 32 tokens, the most a block table holds: every entry is the same page of 32
    tokens, so the output is the mean of its 32 values (q = 0: all weights are one power
    of two). Bound on the error's norm relative to the mean of the values' norms: a stream
    of the at least 100 CTAs adds at most 2^31 / 100 / 2 / 16 products of 16 tokens to one
    fp32 sum (the sums of the weights stay exact below 2^24 units), each addition good to
    2^-23: 2^-23 * 671089 = 0.08. What the test is for is that the tokens are there at
    all: the values share a mean near their norm."""
    S = Setup(53, 1, 1, 1)
    n, wide = (1 << 31) - 32, (1 << 26) - 1
    kb, vb = S.tokens(32)
    base = S.rng.standard_normal(128)
    vb = synth.to_bf16_bits(base + 0.1 * S.rng.standard_normal((32, 1, 128)))
    P = PagedLayer(S.cfg, 1, 1, 1, 1, layer=1, pages=DevicePageAllocator(1, 1, 1, 1))
    P.set_plans(S.plans)
    cu, slots, _ = P.assign(torch.tensor([32], dtype=torch.int32, device=DEV), 32)
    P.append_ragged(dev_bf16(kb), dev_bf16(vb), cu, slots)
    table = torch.zeros(1, wide, dtype=torch.int32, device=DEV)
    long, none = kvq.make_pages(P.pool, table, 1, 1), kvq.make_pages(P.pool, table[:, :1], 1, 1)
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    zero, gs = torch.zeros_like(lens), torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    q = torch.zeros(1, 2, 128, dtype=torch.bfloat16, device=DEV)
    out = torch.empty_like(q)
    ws = prefix_workspace(S.cfg, 1, 2, 1)
    args = (long, lens, gs, n, none, zero) if shared else (none, zero, gs, 32, long, lens)
    kvq.paged_prefix_decode_attn(S.cfg, P.plan_ptrs, *args, 32 if shared else n, q, out, ws,
                                 P.status)
    assert P.flags() == 0
    v = S.heads(kb, vb)[0][1]
    ref, size = v.mean(axis=0), np.linalg.norm(v, axis=1).mean()
    assert np.linalg.norm(ref) > 0.5 * size
    for h in range(2):
        err = np.linalg.norm(out[0, h].double().cpu().numpy() - ref)
        assert err <= 0.08 * size + 2.0 ** -8 * np.linalg.norm(ref), err / size
