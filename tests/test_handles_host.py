"""The handles that the binding keeps C structures in: what they may be used for between and
after calls, without a GPU."""
import copy
import pickle

import pytest
import torch

import sparse_kv_long_sfi_gb300 as sfi
from sparse_kv_long_sfi_gb300 import api


@pytest.fixture
def host(monkeypatch):
    """Handles of tensors in host memory (nothing is launched here)."""
    monkeypatch.setattr(api, "_need", lambda t, dtype, name: None)
    monkeypatch.setattr(api, "_on_current_device", lambda t, name: None)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: -1, raising=False)


def _i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def _handles():
    return {
        "PagedKV4": sfi.PagedKV4(torch.zeros(5, 2, 1152, dtype=torch.uint8), _i32(3, 4), _i32(3), 2.0, 0.5),
        "CompactKV4": sfi.CompactKV4(torch.zeros(6, 1152, dtype=torch.uint8), torch.zeros(3, dtype=torch.int64), _i32(3),
                                     _i32(3)),
        "Rope": sfi.Rope(torch.arange(8), torch.zeros(8, dtype=torch.uint8), 2, True),
        "Rope without axes": sfi.Rope(torch.arange(8)),
        "PageMap": sfi.PageMap(_i32(3, 4), _i32(3), _i32(9)),
        "PagePools": sfi.PagePools([torch.arange(40).view(5, 8), torch.zeros(5, 8, dtype=torch.int64)]),
    }


def _tensors(h):
    if isinstance(h, sfi.PagePools):
        return h.pools
    return [t for t in vars(h).values() if isinstance(t, torch.Tensor)]


@pytest.mark.parametrize("name", ["PagedKV4", "CompactKV4", "Rope", "Rope without axes", "PageMap", "PagePools"])
def test_handles_are_copied_before_and_after_a_call(host, name):
    for used in (False, True):
        h = _handles()[name]
        if used:
            h.c()
        for copied in (copy.deepcopy(h), pickle.loads(pickle.dumps(h)), copy.copy(h)):
            assert type(copied) is type(h) and len(_tensors(copied)) == len(_tensors(h))
            c, own = copied.c(), h.c()
            assert c is not own
            for a, b in zip(_tensors(copied), _tensors(h)):
                assert torch.equal(a, b)
            first = c._fields_[0][0]
            if isinstance(h, sfi.PagePools):
                assert copied.addresses.tolist() == [t.data_ptr() for t in copied.pools]
                assert getattr(c, first) == copied.addresses.data_ptr()
            else:
                assert getattr(c, first) == _tensors(copied)[0].data_ptr()
            # everything but the addresses is alike
            for f, _ in c._fields_:
                if not isinstance(getattr(c, f), int) or getattr(c, f) < 4096:
                    assert getattr(c, f) == getattr(own, f), f


def test_a_tensor_that_changes_in_place_is_looked_at_again(monkeypatch):
    """A table or pool that gets another shape or other strides where it lies: the structure is made
    anew (the memory's address alone would not say so), and refused where it no longer fits."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: -1, raising=False)

    def need(t, dtype, name):  # what the binding asks for, but the device
        if t.dtype != dtype or not t.is_contiguous():
            raise ValueError(name)

    monkeypatch.setattr(api, "_need", need)
    kv = sfi.PagedKV4(torch.zeros(5, 2, 1152, dtype=torch.uint8), _i32(4, 4), _i32(4))
    assert kv.c() is kv.c() and kv.c().max_pages_per_req == 4 and kv.c().num_pages == 5
    at = kv.page_table.data_ptr()
    kv.page_table.resize_(4, 3)
    assert kv.page_table.data_ptr() == at
    assert kv.c().max_pages_per_req == 3
    kv.pool.data = kv.pool.data[:3]
    assert kv.pool.data_ptr() == kv.c().pool and kv.c().num_pages == 3
    kv.page_table.resize_(3, 4)  # a row less than there are lengths
    with pytest.raises(ValueError):
        kv.c()
    kv.seq_lens.resize_(3)
    assert kv.c().max_pages_per_req == 4
    kv.page_table.resize_(3, 3)
    assert kv.c() is kv.c()
    kv.page_table.t_()  # the same address and shape
    with pytest.raises(ValueError):
        kv.c()
    pm = sfi.PageMap(_i32(3, 4), _i32(3), _i32(9))
    assert pm.c().num_pages == 9
    pm.ref_count.resize_(7)
    assert pm.c().num_pages == 7
    comp = sfi.CompactKV4(torch.zeros(6, 1152, dtype=torch.uint8), torch.zeros(3, dtype=torch.int64), _i32(3), _i32(3))
    assert comp.c().total_pages == 6
    comp.pool.resize_(4, 1152)
    assert comp.c().total_pages == 4
    rope = sfi.Rope(torch.arange(8), torch.zeros(8, dtype=torch.uint8))
    assert rope.c().rot_dim == 16
    rope.turns.resize_(4)
    with pytest.raises(ValueError):
        rope.c()
    rope.axis.resize_(4)
    assert rope.c().rot_dim == 8
