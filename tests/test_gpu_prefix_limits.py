"""GPU: the shared-prefix decode at the ends of what its interface allows: more
prefixes than sequences, in a workspace of exactly the size asked for."""
import numpy as np
import pytest
import torch

from bit_kv_cache_19_b200 import kvq
from test_gpu_prefix_decode import DEV, Setup, check, contiguous, group_of, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_many_empty_prefixes_in_an_exact_workspace(dtype):
    """1024 prefixes, of which five sequences use three: nothing is written past the
    workspace, which does not grow with the prefixes that no sequence has."""
    S = Setup(51, 2, 3, 3)
    n_prefixes, own = 1024, [3, 40, 0, 70, 33]
    used = {7: 100, 500: 257, 1023: 31}  # prefix: tokens
    lens = [used.get(g, 0) for g in range(n_prefixes)]
    edge = {7: (0, 1), 500: (1, 3), 1023: (3, 5)}
    start, at = [], 0
    for g in range(n_prefixes):
        start.append(edge[g][0] if g in edge else at)
        at = edge[g][1] if g in edge else at
    start.append(5)
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
