"""Trimming requests' pages, beside the other page operators and against the model on the host."""
import numpy as np
import pytest
import torch

from tests.gpu_harness import dev_i32
from tests.test_gpu_pages import Device, Model

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from sparse_kv_long_sfi_gb300 import build
    build.build()


def _sfi():
    import sparse_kv_long_sfi_gb300 as sfi
    return sfi


def _trim(m, new, reqs):
    """The model's trim: pages behind the new lengths lose a holder."""
    for r, n in zip(reqs, new):
        for i in range(-(-n // 16), -(-int(m.lens[r]) // 16)):
            m.ref[m.table[r][i]] -= 1
        m.lens[r] = n


@pytest.mark.parametrize("seed", range(4))
def test_histories(seed):
    """Reservations, forks and trims in turn: table, lengths and holders are the model's."""
    sfi = _sfi()
    g = np.random.default_rng(seed)
    m = Model(6, 20, 120, 2, 32, seed)
    d = Device(m)
    for step in range(12):
        new = [int(min(x + g.integers(0, 60), 20 * 16)) for x in m.lens]
        if m.reserve(new, list(range(6))):
            sfi.sfi_page_reserve(d.map, d.pp, dev_i32(new), workspace=d.ws, dev_status=d.st)
        reqs = g.permutation(6)[: g.integers(1, 7)].tolist()
        new = [int(g.integers(0, int(m.lens[r]) + 1)) for r in reqs]
        _trim(m, new, reqs)
        sfi.sfi_page_trim(d.map, dev_i32(new), dev_i32(reqs), dev_status=d.st)
        assert d.st.item() == 0
        d.same(m, (seed, step))


def test_shared_pages_keep_their_other_holders():
    sfi = _sfi()
    m = Model(4, 8, 30, 2, 32, 1)
    assert m.reserve([70], [0])
    d = Device(m)
    sfi.sfi_page_fork(d.map, dev_i32([0]), dev_i32([2]), dev_status=d.st)
    sfi.sfi_page_trim(d.map, dev_i32([17]), dev_i32([2]), dev_status=d.st)
    held = d.map.ref_count.cpu()[d.map.page_table.cpu()[0, :5].long()].tolist()
    assert held == [2, 2, 1, 1, 1] and d.map.seq_lens.tolist()[2] == 17 and d.st.item() == 0


@pytest.mark.parametrize("length,new", [(50, 51), (50, -1), (2 ** 31 - 1, 5), (-1, 0), (8 * 16 + 1, 0), (0, 1)])
def test_lengths_out_of_range(length, new):
    """A request whose length, or whose new one, is out of range stays as it is; the others are cut."""
    sfi = _sfi()
    m = Model(3, 8, 30, 2, 32, 2)
    assert m.reserve([100, 100], [0, 1])
    m.lens[2] = length
    d = Device(m)
    sfi.sfi_page_trim(d.map, dev_i32([30, new]), dev_i32([0, 2]), dev_status=d.st)
    assert d.st.item() == 2
    _trim(m, [30], [0])
    d.same(m, (length, new))


def test_request_ids_and_pages_out_of_range():
    sfi = _sfi()
    m = Model(3, 8, 30, 2, 32, 3)
    assert m.reserve([100, 100], [0, 1])
    d = Device(m)
    sfi.sfi_page_trim(d.map, dev_i32([0, 0]), dev_i32([3, -1]), dev_status=d.st)
    assert d.st.item() == 8
    d.same(m, "ids")
    d.st.zero_()
    d.map.page_table[0, 5] = 30
    sfi.sfi_page_trim(d.map, dev_i32([20]), dev_i32([0]), dev_status=d.st)
    assert d.st.item() == 1 and d.map.seq_lens.tolist()[0] == 20
