"""Prompt attention where a CTA takes over items of different kinds: one and two tiles of query rows, one step and more."""
import pytest
import torch

from tests.test_gpu_window_limits import Call

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from sparse_kv_long_sfi_gb300 import build
    build.build()


@pytest.mark.parametrize("heads,t", [((8, 1, 128), 32), ((8, 1, 64), 32), ((2, 2, 64), 256)])
def test_items_of_one_tile_behind_two(heads, t):
    """Two tiles and one step, then one tile and one step, and so on: many of them on every CTA."""
    g = heads[0] // heads[1]
    small, large = 64 // g, 192 // g
    kinds = [(large, 0), (small, 0), (large, 140), (small, 300), (small, 0), (small, 0), (large, 0)]
    new, lens = [], []
    for i in range(700):
        n, behind = kinds[i % len(kinds)]
        new.append(n)
        lens.append(n + behind)
    c = Call(61, lens, t, new=new, heads=heads, sink=2, recent=1 << 20).device()
    for _ in range(3):
        c.out.fill_(7)
        c.attend()
        assert c.st.item() == 0
        for r in range(0, 700, 53):
            for i in (0, new[r] - 1):
                c.check(r, i)
        untouched = c.out.view(700, t, -1)
        behind = torch.arange(t, device="cuda")[None] >= torch.tensor(new, device="cuda")[:, None]
        assert (untouched[behind] == 7).all() and torch.isfinite(untouched).all()
