"""One workspace of the 4-bit attention for several shapes."""
import pytest
import torch

from tests.test_gpu_kv4 import Cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from sparse_kv_long_sfi_gb300 import build
    build.build()


def test_shapes_share_a_workspace():
    """Calls of different KV heads, head sizes, query rows and batches in turn on one workspace, their
    units cut across CTAs: bit for bit what each gives on a workspace of its own, and the counters are
    zero at the end. Page tables too wide for clusters send every dense call through the workspace; the
    last shape has 1024 units, of which every third or so is cut."""
    import sparse_kv_long_sfi_gb300 as sfi
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    calls = []
    for seed, (lens, hkv, G, d, T) in enumerate([
            ([5000, 300, 2100], 8, 2, 128, 1), ([3000, 9000], 2, 4, 64, 1), ([20000], 1, 8, 128, 2),
            ([700, 1500, 40, 4100, 2600], 4, 1, 64, 3), ([400 + 7 * i for i in range(64)], 16, 2, 128, 1)]):
        c = Cache(300 + seed, lens, hkv, d)
        wide = torch.full((len(lens), 3000), -1, dtype=torch.int32, device="cuda")
        wide[:, :c.kv.page_table.shape[1]] = c.kv.page_table
        c.kv.page_table = wide
        shape = sfi.AttnShape(hkv * G, hkv, d)
        q = torch.randn(len(lens), T, hkv * G, d, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()
        calls.append((shape, c, q, T))
    sizes = [sfi.sfi_kv4_workspace_size(s, len(c.lens), T) for s, c, _, T in calls]
    shared = torch.zeros(max(sizes), dtype=torch.uint8, device="cuda")

    def run(i, ws):
        shape, c, q, T = calls[i]
        out, lse = torch.full(q.shape, float("nan"), device="cuda"), torch.full(q.shape[:3], float("nan"), device="cuda")
        sfi.sfi_kv4_dense_attn(shape, c.kv, 4, 32, q, out, lse=lse, workspace=ws, dev_status=st)
        return out, lse

    want = [run(i, torch.zeros(n, dtype=torch.uint8, device="cuda")) for i, n in enumerate(sizes)]
    order = [0, 1, 2, 3, 4, 3, 2, 1, 0, 0, 2, 4, 1, 3, 0, 4]
    got = [(i, run(i, shared)) for i in order]
    torch.cuda.synchronize()
    assert st.item() == 0
    for i, (out, lse) in got:
        assert torch.isfinite(out).all() and torch.isfinite(lse).all(), i
        assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1]), i
    assert not shared[:2048].any()
