"""Attention weights of long calls whose blocks are shared by the CTAs of a cluster: a bad page, and what each part adds."""
import pytest
import torch

from tests.test_gpu_attn_mass import _check, _expected, _problem, _run
from tests.test_gpu_window_limits import WIDE, Call

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from sparse_kv_long_sfi_gb300 import build
    build.build()


@pytest.mark.parametrize("heads,t", [((2, 1, 64), 600), ((8, 1, 128), 300), ((4, 2, 64), 1100)])
@pytest.mark.parametrize("sink,recent", [(0, WIDE), (5, 300)])
def test_few_blocks_of_many_rows(heads, t, sink, recent):
    """One request of few heads: two, four and eight CTAs work on each block; parts without a row among them."""
    lens, new = [t + 130], [t]
    c, q, lse = _problem(91, lens, heads, new, sink, recent, t)
    mass = torch.rand(1, heads[1], t + 140, generator=torch.Generator().manual_seed(9))
    got, st = _run(c, q, lse, new, sink, recent, mass, 0.5)
    assert st == 0
    _check(got, *_expected(c, q, lse, new, sink, recent, mass, 0.5), lens, mass)


@pytest.mark.parametrize("heads,t", [((2, 1, 64), 600), ((8, 1, 128), 300), ((8, 2, 64), 2500)])
@pytest.mark.parametrize("page", [-1, 1 << 20])
def test_a_bad_page_spoils_its_block_alone(heads, t, page):
    """No position of the block of 256 is written, in no part's name; all others get what they get without it."""
    c = Call(93, [t + 300], t, heads=heads, recent=WIDE).device()
    c.lse.fill_(3.0)
    c.weigh()
    torch.cuda.synchronize()
    assert c.st.item() == 0
    want = c.mass.clone()
    for block in (0, 1, (t + 299) // 256):
        c.mass.fill_(0.25)
        c.st.zero_()
        table = c.kv.page_table.clone()
        c.kv.page_table[0, 16 * block] = page
        c.weigh()
        c.kv.page_table.copy_(table)
        assert c.st.item() == 1
        assert (c.mass[:, :, 256 * block:256 * block + 256] == 0.25).all()
        keep = torch.ones(c.mass.shape[2], dtype=torch.bool, device="cuda")
        keep[256 * block:256 * block + 256] = False
        assert torch.equal(c.mass[:, :, keep], want[:, :, keep])
