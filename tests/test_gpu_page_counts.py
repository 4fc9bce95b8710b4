"""Page reservation over as many pages as a map can have."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from sparse_kv_long_sfi_gb300 import build
    build.build()


@pytest.mark.parametrize("free", [[-1], [-9000, -2], [0, 2 ** 30, -1]])
def test_the_last_of_all_page_ids(free):
    """2^31 - 1 pages, nearly all held: the search ends at the last id, and reports when there are too few."""
    import sparse_kv_long_sfi_gb300 as sfi
    pages = 2 ** 31 - 1
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 35 GB")
    ref_count = torch.ones(pages, dtype=torch.int32, device="cuda")
    ids = [i % pages for i in free]
    ref_count[ids] = 0
    table = torch.zeros(1, 8, dtype=torch.int32, device="cuda")
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    m = sfi.PageMap(table, lens, ref_count)
    ws = sfi.alloc_page_workspace(m)
    want = torch.tensor([16 * len(ids)], dtype=torch.int32, device="cuda")
    sfi.sfi_page_reserve(m, None, want, workspace=ws, dev_status=st)
    assert st.item() == 0 and lens.item() == want.item()
    assert table[0, :len(ids)].tolist() == sorted(ids) and (ref_count[ids] == 1).all()
    sfi.sfi_page_reserve(m, None, want + 16, workspace=ws, dev_status=st)
    assert st.item() == 64 and lens.item() == want.item()
    del ref_count, ws, m
    torch.cuda.empty_cache()
