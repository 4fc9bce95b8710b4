"""The 4-bit calls and the norm at the last positions that a page table can name, just below 2^31."""
import pytest
import torch

from tests.gpu_harness import dev_i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from sparse_kv_long_sfi_gb300 import build
    build.build()


@pytest.mark.parametrize("new", [1, 16, 33, 48])
def test_the_last_positions(new):
    """A request of 2^31 - 16 tokens (a table row of 512 MB, whose pages but the last four are page 0):
    its newest tokens are appended, read back, normed into bf16 pages and attended to in the recent
    window; the same as with a request of 64 tokens on a narrow table. Rows asked for behind the
    length stay as they were, and no page but the last ones changes."""
    import sparse_kv_long_sfi_gb300 as sfi
    hq, hkv, d, T = 4, 2, 64, 48
    shape, L = sfi.AttnShape(hq, hkv, d), 2 ** 31 - 16
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    table = torch.zeros(1, L // 16, dtype=torch.int32, device="cuda")
    table[0, -4:] = dev_i32([3, 1, 4, 2])
    g = torch.Generator().manual_seed(new)
    rand = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    k, v, q = rand(1, T, hkv, d), rand(1, T, hkv, d), rand(1, 1, hq, d)
    x = rand(1, T, hq, d)
    pool = torch.randint(0, 256, (7, hkv, 18 * d), generator=g, dtype=torch.int64).to(torch.uint8)
    pool[..., 8 * d:9 * d] = 0x38  # scales of 1
    pool[..., 17 * d:] = 0x38
    bf = rand(2, 7, hkv, 16, d)
    comp = sfi.alloc_kv4_compact(shape, [16])
    ws, lens = sfi.alloc_kv4_workspace(shape, 1), dev_i32([new])
    got = []
    for tab, n in ((table, L), (dev_i32([[3, 1, 4, 2]]), 64)):
        kv = sfi.PagedKV4(pool.cuda(), tab, dev_i32([n]))
        sfi.sfi_kv4_append(shape, kv, k, v, new_lens=lens, dev_status=st)
        rows = [torch.full((1, T, hkv, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        sfi.sfi_kv4_read(shape, kv, *rows, first=dev_i32([n - new]), dev_status=st)
        assert all((r[:, new:] == 7.0).all() for r in rows)
        out, lse = torch.full((1, 1, hq, d), float("nan"), device="cuda"), torch.full((1, 1, hq), float("nan"), device="cuda")
        sfi.sfi_kv4_fast_attn(shape, kv, comp, 0, 40, q, out, lse=lse, workspace=ws, dev_status=st)
        pages = [p.clone() for p in bf]
        sfi.sfi_qk_norm_rope(shape, None, x, k, v, torch.empty_like(x), new_lens=lens, dev_status=st,
                             kv=sfi.PagedKV(*pages, tab, dev_i32([n])))
        torch.cuda.synchronize()
        assert st.item() == 0
        got.append([kv.pool, *rows, out, lse, *pages])
    for a, b in zip(*got):
        assert torch.equal(a, b) and torch.isfinite(a.float()).all()
    touched = {[3, 1, 4, 2][p] for p in range((64 - new) // 16, 4)}
    rest = [i for i in range(7) if i not in touched]
    assert torch.equal(got[0][0].cpu()[rest], pool[rest])
    for page, before in zip(got[0][-2:], bf):
        assert torch.equal(page[rest], before[rest])
