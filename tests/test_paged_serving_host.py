"""Refusals of the paged-serving calls: every argument error is found before any
CUDA call, so they are tested on the CPU through the C interface; the Python
binding refuses tensors it cannot pass on."""
import ctypes

import pytest
import torch

from bit_kv_cache_19_b200 import kvq
from bit_kv_cache_19_b200.runtime import PackedLayer, PagedLayer

A = ctypes.create_string_buffer(1 << 12)
BASE = (ctypes.addressof(A) + 511) & ~511  # a non-null, aligned address; never read


def _expect(code, name, args):
    assert getattr(kvq.lib(), name)(*args) == code, kvq.lib().kvq_last_error()
    assert kvq.lib().kvq_last_error()


def _state(**kw):
    f = dict(block_table=BASE, held=BASE, free_ids=BASE, free_ring=BASE, n_pages=8, page_tiles=2,
             max_pages=4)
    f.update(kw)
    return kvq.PageState(*[f[n] for n, _ in kvq.PageState._fields_])


def test_pages_assign_refusals():
    ws = kvq.pages_assign_workspace_bytes(3)
    assert ws > 0 and kvq.pages_assign_workspace_bytes(0) == 0
    assert kvq.pages_assign_workspace_bytes(65536) == 0

    def args(state=None, lens=BASE, n_new=BASE, batch=3, n_slots=9, cu=BASE, slots=BASE, pos=None,
             w=BASE, n=ws, status=BASE):
        return [state or _state(), lens, n_new, batch, n_slots, cu, slots, pos, w, n, status, None]
    for kw in (dict(lens=None), dict(n_new=None), dict(cu=None), dict(slots=None), dict(w=None),
               dict(status=None), dict(batch=0), dict(batch=65536), dict(n_slots=-1),
               dict(n_slots=1 << 31), dict(w=BASE + 8)):
        _expect(kvq.ERR_ARG, "kvq_pages_assign", args(**kw))
    for kw in (dict(block_table=None), dict(held=None), dict(free_ids=None), dict(free_ring=None),
               dict(n_pages=0), dict(n_pages=1 << 31), dict(page_tiles=3), dict(page_tiles=0),
               dict(page_tiles=1 << 21), dict(max_pages=0), dict(max_pages=1 << 26)):
        _expect(kvq.ERR_ARG, "kvq_pages_assign", args(state=_state(**kw)))
    _expect(kvq.ERR_WORKSPACE, "kvq_pages_assign", args(n=ws - 1))


def test_append_ragged_refusals():
    cfg = kvq.make_cfg(2, 3, 3)

    def args(c=cfg, plans=BASE, k=BASE, v=BASE, dtype=kvq.BF16, n=5, cu=BASE, slots=BASE, batch=2,
             pool=BASE, n_pages=8, page_tiles=2, lens=BASE, rope=0.0, status=BASE):
        return [ctypes.byref(c), plans, k, v, dtype, n, cu, slots, batch, pool, n_pages, page_tiles,
                lens, rope, status, None]
    for kw in (dict(plans=None), dict(k=None), dict(v=None), dict(cu=None), dict(slots=None),
               dict(pool=None), dict(lens=None), dict(status=None), dict(dtype=3), dict(dtype=-1),
               dict(n=-1), dict(n=1 << 31), dict(batch=0), dict(batch=65536), dict(pool=BASE + 8),
               dict(n_pages=0), dict(n_pages=1 << 31), dict(page_tiles=6), dict(rope=1.0),
               dict(rope=-3.0), dict(rope=float("inf")), dict(rope=float("nan")),
               dict(c=kvq.make_cfg(2, 9, 3)), dict(c=kvq.make_cfg(0, 3, 3))):
        _expect(kvq.ERR_ARG, "kvq_paged_append_ragged", args(**kw))
    _expect(kvq.ERR_UNSUPPORTED, "kvq_paged_append_ragged",
            args(c=kvq.make_cfg(2, 3, 3, head_dim=64)))
    assert kvq.lib().kvq_paged_append_ragged(*args(n=0, k=None, v=None, slots=None)) == kvq.OK


@pytest.mark.parametrize("paged", [False, True])
def test_prefix_decode_refusals(paged):
    cfg = kvq.make_cfg(2, 3, 3)
    ws = kvq.prefix_decode_workspace_bytes(cfg, 4, 8, 2)
    assert ws > 0
    for bad in ((0, 8, 2), (4, 7, 2), (4, 34, 2), (4, 8, 0), (4, 8, 1025), (65536, 8, 2)):
        assert kvq.prefix_decode_workspace_bytes(cfg, *bad) == 0
    name = "kvq_paged_prefix_decode_attn" if paged else "kvq_prefix_decode_attn"
    pages = ctypes.byref(kvq.Pages(BASE, BASE, 8, 2, 4)) if paged else BASE

    def args(c=cfg, plans=BASE, pre=pages, pre_lens=BASE, start=BASE, n_pre=2, max_pre=64,
             own=pages, lens=BASE, batch=4, max_len=64, q=BASE, qt=kvq.BF16, n_q=8, out=BASE,
             ot=kvq.BF16, w=BASE, n=ws, status=BASE):
        return [ctypes.byref(c), plans, pre, pre_lens, start, n_pre, max_pre, own, lens, batch,
                max_len, q, qt, n_q, out, ot, w, n, status, None]
    for kw in (dict(plans=None), dict(pre=None), dict(pre_lens=None), dict(start=None),
               dict(own=None), dict(lens=None), dict(q=None), dict(out=None), dict(w=None),
               dict(status=None), dict(n_pre=0), dict(n_pre=1025), dict(max_pre=0),
               dict(max_pre=1 << 31), dict(batch=0), dict(batch=65536), dict(max_len=0),
               dict(max_len=1 << 31), dict(qt=3), dict(ot=7), dict(n_q=7), dict(n_q=34),
               dict(n_q=0), dict(w=BASE + 16), dict(out=BASE + 8)):
        _expect(kvq.ERR_ARG, name, args(**kw))
    _expect(kvq.ERR_WORKSPACE, name, args(n=ws - 1))
    _expect(kvq.ERR_UNSUPPORTED, name, args(c=kvq.make_cfg(2, 3, 3, head_dim=96)))
    if paged:
        for bad in (kvq.Pages(None, BASE, 8, 2, 4), kvq.Pages(BASE, None, 8, 2, 4),
                    kvq.Pages(BASE, BASE, 8, 3, 4), kvq.Pages(BASE, BASE, 0, 2, 4)):
            _expect(kvq.ERR_ARG, name, args(pre=ctypes.byref(bad)))
            _expect(kvq.ERR_ARG, name, args(own=ctypes.byref(bad)))


def test_binding_refuses_what_it_cannot_pass():
    """CPU tensors, other types, shapes and strides raise before the library is
    called."""
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(kvq.KVQError):
        kvq.pages_assign(_state(), i, i, torch.zeros(4, dtype=torch.int32),
                         torch.zeros(2, dtype=torch.int64), None, i, i)
    with pytest.raises(kvq.KVQError):
        kvq.make_page_state(torch.zeros(3, 4, dtype=torch.int64), i, i,
                            torch.zeros(2, dtype=torch.int64), 1)
    x = torch.zeros(5, 2, 128)
    with pytest.raises(kvq.KVQError):
        kvq.paged_append_ragged(kvq.make_cfg(2, 3, 3), i, x, x, i, i.long(), x, 1, 1, i, i)
    with pytest.raises(kvq.KVQError):
        kvq.prefix_decode_attn(kvq.make_cfg(2, 3, 3), i, i, i, i, 4, i, i, 4, x, x, x, i)
    with pytest.raises(kvq.KVQError):
        kvq._DTYPES[torch.int8]


def test_layer_on_host_pages_refuses_device_assignment():
    L = PagedLayer.__new__(PagedLayer)
    L.dev_pages = None
    with pytest.raises(RuntimeError):
        L.assign(None)
    L.alloc = None
    with pytest.raises(RuntimeError):
        L.reserve(0, 5)
    with pytest.raises(RuntimeError):
        L.release(0)


def test_host_memory_is_not_passed_to_the_gpu(monkeypatch):
    """Workspaces, status words and pools on the host, and lengths of another
    batch than the block table's, raise before the library is called."""
    def no_call():
        raise AssertionError("the library was called")

    monkeypatch.setattr(kvq, "_need", lambda *a: None)
    monkeypatch.setattr(kvq, "_ptrs", lambda *a: None)
    monkeypatch.setattr(kvq, "lib", no_call)
    i, x, cfg = torch.zeros(3, dtype=torch.int32), torch.zeros(3, 2, 128), kvq.make_cfg(2, 3, 3)
    page = torch.zeros(1 << 14, dtype=torch.uint8)
    calls = [lambda: kvq.pages_assign(_state(), i, i, i, i, None, i, i),
             lambda: kvq.paged_append_ragged(cfg, i, x, x, i, i, page, 1, 1, i, i),
             lambda: kvq.prefix_decode_attn(cfg, i, i, i, i, 4, i, i, 4, x, x, x, i),
             lambda: kvq.paged_prefix_decode_attn(cfg, i, None, i, i, 4, None, i, 4, x, x, x, i)]
    for call in calls:
        with pytest.raises(kvq.KVQError, match="not on a GPU"):
            call()
    monkeypatch.setattr(kvq, "_on_device", lambda **k: None)
    state = kvq.make_page_state(torch.zeros(4, 2, dtype=torch.int32), i, i, i, 1)
    with pytest.raises(kvq.KVQError, match="block table of 4 rows"):
        kvq.pages_assign(state, i, i, i, i, None, i, i)


@pytest.mark.parametrize("kind", [PackedLayer, PagedLayer])
@pytest.mark.parametrize("other", [(1, 3, 3), (2, 2, 3), (2, 3, 2)])
def test_prefix_of_another_format(kind, other):
    L, P = kind.__new__(kind), kind.__new__(kind)
    L.cfg, P.cfg = kvq.make_cfg(2, 3, 3), kvq.make_cfg(*other)
    with pytest.raises(ValueError, match="heads or bits"):
        L.decode_prefix(None, P, None)
