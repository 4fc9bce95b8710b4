"""The page operators at the ends of their ranges: lengths that only device data can say, sums
past 32 bits, pages of several chunks."""
import numpy as np
import pytest
import torch

from tests.gpu_harness import dev_i32
from tests.test_gpu_pages import Device, Model

pytestmark = pytest.mark.gpu

BAD_LEN, NO_PAGE = 2, 64


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from sparse_kv_long_sfi_gb300 import build
    build.build()


def _sfi():
    import sparse_kv_long_sfi_gb300 as sfi
    return sfi


@pytest.mark.parametrize("length", [2 ** 31 - 1, 2 ** 31 - 15, 2 ** 31 - 16, 2 ** 31 - 17, 49, -1, -2 ** 31])
def test_a_length_out_of_range_is_no_length(length):
    """A length beyond the table, up to the largest a 32-bit word holds, or below zero: the request
    is refused by every call, and nothing changes."""
    sfi = _sfi()
    m = Model(5, 3, 12, 2, 32, 4)
    assert m.reserve([20, 40], [0, 1])
    m.lens[3] = length
    d = Device(m)

    def refused(what, call):
        d.st.zero_()
        call()
        assert d.st.item() == BAD_LEN, what
        d.same(m, (length, what))

    refused("fork", lambda: sfi.sfi_page_fork(d.map, dev_i32([3]), dev_i32([4]), dev_status=d.st))
    for part in (0, 16, max(0, length - 20)):
        refused(("fork", part), lambda: sfi.sfi_page_fork(d.map, dev_i32([3]), dev_i32([4]), dev_i32([part]), dev_status=d.st))
    refused("free", lambda: sfi.sfi_page_free(d.map, dev_i32([3]), dev_status=d.st))
    refused("free twice", lambda: sfi.sfi_page_free(d.map, dev_i32([3, 3]), dev_status=d.st))
    for new in (48, 2 ** 31 - 1):
        refused(("reserve", new), lambda: sfi.sfi_page_reserve(d.map, d.pp, dev_i32([new]), dev_i32([3]), workspace=d.ws,
                                                               dev_status=d.st))
    refused("reserve that far", lambda: sfi.sfi_page_reserve(d.map, d.pp, dev_i32([2 ** 31 - 1]), dev_i32([0]),
                                                             workspace=d.ws, dev_status=d.st))
    # a compaction copies the row of such a request as it is
    table, ref, live = torch.empty_like(d.map.page_table), torch.empty_like(d.map.ref_count), dev_i32([0])
    d.st.zero_()
    sfi.sfi_page_compact(d.map, d.pp, table, ref, live, workspace=d.ws, dev_status=d.st)
    assert d.st.item() == BAD_LEN and live.item() == 5
    m.lens[3] = 0
    m.compact()
    assert np.array_equal(table.cpu().numpy(), m.table) and np.array_equal(ref.cpu().numpy(), m.ref)


def test_a_need_past_32_bits_is_refused():
    """1024 requests that ask for 2^31 pages and more between them (a table of 17 GB): the sum of
    what they need does not wrap, the reservation is refused, and nothing changes."""
    sfi = _sfi()
    n, maxp = 1024, (1 << 22) + 8
    table = torch.zeros(n, maxp, dtype=torch.int32, device="cuda")
    lens, ref = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(300, dtype=torch.int32, device="cuda")
    pm = sfi.PageMap(table, lens, ref)
    ws, st = sfi.alloc_page_workspace(pm), torch.zeros(1, dtype=torch.int32, device="cuda")

    def reserve(pages):
        st.zero_()
        sfi.sfi_page_reserve(pm, None, dev_i32(np.asarray(pages, np.int64) * 16), workspace=ws, dev_status=st)
        return st.item()

    half, whole = np.full(n, 1 << 21), np.full(n, 1 << 22)
    more = whole.copy()
    more[3] += 5
    # 2^31, 2^32, 2^32 + 5 (which is 5 modulo 2^32), and one page too many
    for pages in (half, whole, more, np.r_[np.zeros(n - 1, int), 301], np.r_[150, np.zeros(n - 2, int), 151]):
        assert reserve(pages) == NO_PAGE
        assert not lens.any() and not ref.any()
    assert table.max().item() == 0 == table.min().item()
    assert reserve(np.r_[150, np.zeros(n - 2, int), 150]) == 0  # as many as there are
    assert (ref == 1).all() and lens[0].item() == lens[-1].item() == 2400
    assert torch.equal(table[[0, -1], :150].flatten(), torch.arange(300, dtype=torch.int32, device="cuda"))
    assert table[:, 150:].max().item() == 0 == table[1:-1].max().item()


@pytest.mark.parametrize("page_bytes", [8176, 8192, 8208, 16384 + 16, 2 * 16384 + 16])
def test_pages_of_several_chunks(page_bytes):
    """Pages that end in, at and behind the first chunk of a copy, and in the third: copied by ids,
    by a reservation and by a compaction (whose number of moves the device knows), in three pools."""
    sfi = _sfi()
    rng = np.random.default_rng(page_bytes)
    m = Model(30, 6, 160, 3, page_bytes, 11)
    assert m.reserve(list(rng.integers(1, 96, 20)), list(range(20)))
    d = Device(m)
    free = np.flatnonzero(m.ref == 0)
    src, dst = rng.choice(np.flatnonzero(m.ref), 20), rng.permutation(free)[:20]
    sfi.sfi_page_copy(d.pp, dev_i32(src), dev_i32(dst), dev_status=d.st)
    for p in m.pools:
        p[dst] = p[src]
    d.same(m, "copy")
    src, dst = list(range(10)), list(range(20, 30))
    sfi.sfi_page_fork(d.map, dev_i32(src), dev_i32(dst), dev_status=d.st)
    m.fork(src, dst)
    new, reqs = list(m.lens[dst] + 1), dst
    assert (m.lens[dst] % 16 != 0).sum() > 3
    sfi.sfi_page_reserve(d.map, d.pp, dev_i32(new), dev_i32(reqs), workspace=d.ws, dev_status=d.st)
    assert m.reserve(new, reqs)
    d.same(m, "reserve")
    sfi.sfi_page_free(d.map, dev_i32(list(range(0, 20, 2))), dev_status=d.st)
    m.free(list(range(0, 20, 2)))
    table, ref = torch.empty_like(d.map.page_table), torch.empty_like(d.map.ref_count)
    live = torch.empty(1, dtype=torch.int32, device="cuda")
    sfi.sfi_page_compact(d.map, d.pp, table, ref, live, workspace=d.ws, dev_status=d.st)
    held = int((m.ref > 0).sum())
    assert (m.ref[held:] > 0).sum() > 5  # some pages move
    assert live.item() == m.compact() == held
    d.map = sfi.PageMap(table, d.map.seq_lens, ref)
    d.same(m, "compact")
    assert d.st.item() == 0
