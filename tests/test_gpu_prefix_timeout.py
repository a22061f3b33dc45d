"""GPU: a bounded wait of the shared-prefix decode that runs out. With the test hook
kvq_debug_decode_stall the warp that issues the matrix products waits a few
microseconds on a barrier that nothing arrives on, at a step that differs between CTAs,
and leaves; the copies in flight land, every other role gives up, tensor memory is
freed, and the call returns with TIMEOUT. The next call on the same workspace gives
the bits it gave before."""
import numpy as np
import pytest
import torch

from bit_kv_cache_19_b200 import kvq
from bit_kv_cache_19_b200.runtime import prefix_workspace
from test_gpu_prefix_decode import DEV, Setup, contiguous

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch,G,out_dtype", [
    (40, 8, torch.bfloat16),  # 320 rows of a KV head: both streams share the tiles
    (6, 4, torch.bfloat16), (40, 8, torch.float32), (1, 1, torch.float16)])
def test_wait_that_runs_out(batch, G, out_dtype):
    S = Setup(61, 2, 3, 3)
    data = S.tokens(4000)
    P = contiguous(S, [4000], [data])
    own = [(97 * i) % 300 for i in range(batch)]
    Q = contiguous(S, own, [(data[0][:n], data[1][:n]) for n in own])
    q = torch.from_numpy(S.rng.standard_normal((batch, 2 * G, 128))).bfloat16().to(DEV)
    gs = torch.tensor([0, batch], dtype=torch.int32, device=DEV)
    ws = prefix_workspace(S.cfg, batch, 2 * G, 1)
    out = torch.empty(q.shape, dtype=out_dtype, device=DEV)
    want = Q.decode_prefix(q, P, gs, out=out, ws=ws).clone()
    assert Q.flags() == 0
    try:
        assert kvq.lib().kvq_debug_decode_stall(20000) == kvq.OK  # ~10 us at 2 GHz
        for _ in range(3):
            Q.decode_prefix(q, P, gs, out=out, ws=ws)
        torch.cuda.synchronize()
    finally:
        assert kvq.lib().kvq_debug_decode_stall(0) == kvq.OK
    assert Q.flags() == kvq.FLAG_TIMEOUT
    Q.status.zero_()
    for _ in range(3):
        assert torch.equal(Q.decode_prefix(q, P, gs, out=out, ws=ws), want)
    assert Q.flags() == 0 and np.isfinite(want.float().cpu().numpy()).all()
