"""The Python binding's checks of what the library cannot see behind an address: block
tables and pools that are too short. On the CPU: the library is never called."""
import pytest
import torch

from bit_kv_cache_19_b200 import kvq

CFG = kvq.make_cfg(2, 3, 2)
PAGE = 4 * 2 * (512 * 5 + 128)  # four tiles of two KV heads


class OnGpu:
    """A CPU tensor that says it is on a GPU; only its address is taken."""

    def __init__(self, tensor, device=0):
        self.tensor, self.where = tensor, device
        self.is_cuda, self.device = True, f"cuda:{device}"

    def get_device(self):
        return self.where

    def __getattr__(self, name):
        return getattr(self.tensor, name)


@pytest.fixture
def no_call(monkeypatch):
    def called():
        raise AssertionError("the library was called")
    monkeypatch.setattr(kvq, "lib", called)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)


def _i32(*shape, device=0):
    return OnGpu(torch.zeros(*shape, dtype=torch.int32), device)


def _pages(rows, n_pages=5, pool_bytes=5 * PAGE):
    pool = OnGpu(torch.zeros(pool_bytes, dtype=torch.uint8))
    return kvq.make_pages(pool, _i32(rows, 6), n_pages, 4)


def _calls(pages, prefix, batch=3, n_prefixes=2):
    """Each call that follows block tables, for `batch` sequences."""
    x = OnGpu(torch.zeros(batch, 4, 128, dtype=torch.bfloat16))
    k = OnGpu(torch.zeros(batch, 1, 2, 128, dtype=torch.bfloat16))
    o, s, ptrs = OnGpu(torch.zeros(batch, 4, 128)), _i32(1), OnGpu(torch.zeros(9).long())
    lens = _i32(batch)
    return {
        "append": lambda: kvq.paged_quantize_append(CFG, ptrs, k, k, pages, lens, s),
        "decode": lambda: kvq.paged_decode_attn(CFG, ptrs, pages, lens, 64, x, o, s, s),
        "partial": lambda: kvq.paged_decode_attn_partial(CFG, ptrs, pages, lens, 64, x, o, s, s),
        "step": lambda: kvq.paged_append_decode(CFG, ptrs, k, k, pages, lens, 64, x, o, s, s),
        "prefix": lambda: kvq.paged_prefix_decode_attn(
            CFG, ptrs, prefix, _i32(n_prefixes), _i32(n_prefixes + 1), 64, pages, lens, 64, x, o,
            s, s)}


@pytest.mark.parametrize("call", ["append", "decode", "partial", "step", "prefix"])
def test_short_block_tables_and_pools_are_refused(call, no_call):
    with pytest.raises(kvq.KVQError, match="pages: block table of 2 rows for 3"):
        _calls(_pages(2), _pages(2))[call]()
    with pytest.raises(kvq.KVQError, match="pages: pool of"):
        _calls(_pages(3, pool_bytes=5 * PAGE - 1), _pages(2))[call]()
    for rows in (3, 7):  # enough: the call goes through to the library
        with pytest.raises(AssertionError, match="the library was called"):
            _calls(_pages(rows), _pages(2))[call]()
    # a bare description says nothing about its arrays
    with pytest.raises(AssertionError, match="the library was called"):
        _calls(kvq.Pages(16, 16, 5, 4, 6), kvq.Pages(16, 16, 5, 4, 6))[call]()


@pytest.mark.parametrize("call", ["append", "decode", "partial", "step"])
def test_lengths_in_mapped_host_memory_still_go_through(call, no_call, monkeypatch):
    """The calls over plain block tables take lengths, tables and pools at any address
    the GPU can read."""
    host = kvq.make_pages(torch.zeros(5 * PAGE, dtype=torch.uint8),
                          torch.zeros(3, 6, dtype=torch.int32), 5, 4)
    with pytest.raises(AssertionError, match="the library was called"):
        _calls(host, host)[call]()
    monkeypatch.setattr(OnGpu, "get_device", lambda self: self.where if self.tensor.dim() != 1
                        or len(self.tensor) != 3 else -1)
    pages = _pages(3)
    with pytest.raises(AssertionError, match="the library was called"):
        _calls(pages, pages)[call]()


def test_short_prefix_table_is_refused(no_call):
    with pytest.raises(kvq.KVQError, match="prefix_pages: block table of 1 rows for 2"):
        _calls(_pages(3), _pages(1))["prefix"]()
    with pytest.raises(kvq.KVQError, match="prefix_pages: pool of"):
        _calls(_pages(3), _pages(2, n_pages=6))["prefix"]()


@pytest.mark.parametrize("table", [torch.zeros(3, 6, dtype=torch.int64), torch.zeros(18).int(),
                                   torch.zeros(6, 3, dtype=torch.int32).t()])
def test_block_table_of_another_kind_is_refused(table):
    with pytest.raises(kvq.KVQError, match="block_table"):
        kvq.make_pages(OnGpu(torch.zeros(5 * PAGE)), OnGpu(table), 5, 4)


def test_prefix_call_refuses_pages_in_host_memory(no_call):
    args = _arguments(0)
    for name in ("pool", "table", "prefix_table"):
        args[name] = _arguments(0)[name].tensor
        with pytest.raises(kvq.KVQError, match="pages: on devices"):
            _paged_prefix(args)
        args[name] = _arguments(0)[name]


def _arguments(device):
    """Every tensor of the paged-serving calls, on one device."""
    def on(t):
        return OnGpu(t, device)
    ptrs = torch.zeros(9).long()
    return dict(
        lens=_i32(3, device=device), n_new=_i32(3, device=device), cu=_i32(4, device=device),
        slots=on(torch.zeros(5).long()), pos=_i32(5, device=device), ws=_i32(64, device=device),
        status=_i32(1, device=device), table=_i32(3, 6, device=device),
        held=_i32(3, device=device), free_ids=_i32(5, device=device),
        free_ring=on(torch.zeros(2).long()), plan_ptrs=on(ptrs), prefix_ptrs=on(ptrs),
        cache_ptrs=on(ptrs), k=on(torch.zeros(5, 2, 128)), v=on(torch.zeros(5, 2, 128)),
        pool=on(torch.zeros(5 * PAGE, dtype=torch.uint8)), prefix_lens=_i32(2, device=device),
        group_start=_i32(3, device=device), q=on(torch.zeros(3, 4, 128)),
        out=on(torch.zeros(3, 4, 128)), prefix_table=_i32(2, 6, device=device))


def _assign(a):
    state = kvq.make_page_state(a["table"], a["held"], a["free_ids"], a["free_ring"], 4)
    kvq.pages_assign(state, a["lens"], a["n_new"], a["cu"], a["slots"], a["pos"], a["ws"],
                     a["status"])


def _append(a):
    kvq.paged_append_ragged(CFG, a["plan_ptrs"], a["k"], a["v"], a["cu"], a["slots"], a["pool"], 5,
                            4, a["lens"], a["status"])


def _prefix(a):
    kvq.prefix_decode_attn(CFG, a["plan_ptrs"], a["prefix_ptrs"], a["prefix_lens"],
                           a["group_start"], 64, a["cache_ptrs"], a["lens"], 64, a["q"], a["out"],
                           a["ws"], a["status"])


def _paged_prefix(a):
    kvq.paged_prefix_decode_attn(
        CFG, a["plan_ptrs"], kvq.make_pages(a["pool"], a["prefix_table"], 5, 4), a["prefix_lens"],
        a["group_start"], 64, kvq.make_pages(a["pool"], a["table"], 5, 4), a["lens"], 64, a["q"],
        a["out"], a["ws"], a["status"])


_SHARED = "plan_ptrs prefix_lens group_start lens q out ws status"
_TENSORS = {_assign: "lens n_new cu slots pos ws status table held free_ids free_ring",
            _append: "plan_ptrs k v cu slots pool lens status",
            _prefix: _SHARED + " prefix_ptrs cache_ptrs",
            _paged_prefix: _SHARED + " pool table prefix_table"}


@pytest.mark.parametrize("call,name", [(c, n) for c, names in _TENSORS.items()
                                       for n in names.split()])
def test_a_tensor_on_another_gpu_is_refused(call, name, no_call):
    """The library launches on the current device and takes addresses alone."""
    args = _arguments(0)
    with pytest.raises(AssertionError, match="the library was called"):
        call(args)
    args[name] = _arguments(1)[name]
    with pytest.raises(kvq.KVQError):
        call(args)


@pytest.mark.parametrize("call", list(_TENSORS))
def test_all_tensors_on_another_gpu_than_the_current_one(call, monkeypatch):
    class Lib:  # the stream is asked for before the entry point is called
        def __getattr__(self, name):
            def entry(*args):
                raise AssertionError("the library was called")
            return entry
    monkeypatch.setattr(kvq, "lib", Lib)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(kvq.KVQError, match="current device 0"):
        call(_arguments(1))


def test_all_page_state_on_another_gpu_is_refused(no_call):
    args = _arguments(0)
    for name in ("table", "held", "free_ids", "free_ring"):
        args[name] = _arguments(1)[name]
    with pytest.raises(kvq.KVQError, match="page state on device 1"):
        _assign(args)
    args = _arguments(0)
    for name in ("pool", "table", "prefix_table"):
        args[name] = _arguments(1)[name]
    with pytest.raises(kvq.KVQError, match=r"on devices \{1\}, lengths on device 0"):
        _paged_prefix(args)
