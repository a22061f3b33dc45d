"""Workspace sizes of the shared-prefix decode (host only)."""
import pytest

from bit_kv_cache_19_b200 import kvq

ENTRY = 28  # bytes of the group tables for one prefix: 4 + 4 + 8, and rounding


@pytest.mark.parametrize("n_kv,n_q,batch", [(2, 16, 8), (8, 32, 1), (1, 1, 100)])
def test_prefixes_that_no_sequence_can_have_cost_a_table_entry(n_kv, n_q, batch):
    """No more groups have a sequence than there are sequences."""
    cfg = kvq.make_cfg(n_kv, 3, 3)
    size = [kvq.prefix_decode_workspace_bytes(cfg, batch, n_q, n) for n in (1, batch, 1024)]
    assert size[0] <= size[1] <= size[2] <= size[1] + 1024 * ENTRY
