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
