"""Window attention with NaN and infinities in V: rows that do not see them keep their values, rows that do get what the
sum gives, rows that see nothing are zero."""
import numpy as np
import pytest
import torch

from tests import window_reference as ref
from tests.test_gpu_window_limits import Call

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
WIDE = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from sparse_kv_long_sfi_gb300 import build
    build.build()


def _put(c, r, j, value, dims=slice(None)):
    c.c.v[c.c.table[r, j // 16], :, j % 16, dims] = value


def _check(c, r, i, recent):
    """NaN and infinities exactly where the sum has them, the other values within the usual bound."""
    p = c.c.lens[r] - c.new[r] + i
    for h in range(c.c.hq):
        with np.errstate(invalid="ignore"):
            o, x, _, mag, smag = ref.token(c.c, r, h, c.q[r, i, h], p, c.sink, recent)
        got = c.out[r, i, h].double().cpu().numpy()
        assert (np.isnan(got) == np.isnan(o)).all() and (got[np.isinf(o)] == o[np.isinf(o)]).all(), (r, i, h)
        fine = np.isfinite(o)
        assert (np.abs(got[fine] - o[fine]) <= ref.out_bound(o[fine], mag[fine], c.c.d)).all(), (r, i, h)
        assert abs(float(c.lse[r, i, h]) - x) <= ref.lse_bound(x, smag, c.c.d), (r, i, h)


@pytest.mark.parametrize("t,heads", [(3, (8, 2, 64)), (70, (8, 2, 64)), (300, (16, 8, 128)), (8, (2, 2, 128))])
def test_rows_that_see_nothing_are_zero(t, heads):
    """No sink and no window: nothing is seen, whatever V holds."""
    c = Call(71, [t, t + 200], t, heads=heads, sink=0, recent=0)
    c.c.v[:] = NAN
    c.device().attend()
    assert c.st.item() == 0 and (c.out == 0).all() and (c.lse == -INF).all()


@pytest.mark.parametrize("t,heads", [(4, (8, 2, 64)), (70, (8, 2, 64)), (300, (2, 2, 64)), (3, (16, 8, 128)), (150, (16, 8, 128)),
                                     (40, (8, 1, 128))])
@pytest.mark.parametrize("sink,recent", [(3, 40), (0, WIDE), (20, 130)])
def test_seen_and_hidden_together(t, heads, sink, recent):
    """Infinities in the sink, at the window's edges and among the new tokens, all dims or some."""
    lens = [t + 150, t + 9, t + 333, t + 60]
    c = Call(73, lens, t, heads=heads, sink=sink, recent=recent)
    d = heads[2]
    _put(c, 0, 0, INF, slice(0, 8))                     # seen by every row (in the sink, or causal)
    _put(c, 0, lens[0] - 1, NAN)                        # by the last row only
    _put(c, 0, lens[0] - 2, -INF, slice(4, 16))
    for j in range(t // 2):                             # some new tokens, later and later dims
        _put(c, 1, 9 + 2 * j, INF if j % 3 else -INF, slice(j % d, d))
    _put(c, 2, max(sink, lens[2] - t - recent + 2), NAN)  # seen by the first rows, if any
    _put(c, 2, max(sink, lens[2] - t - recent), NAN)
    c.device().attend()
    assert c.st.item() == 0
    rows = sorted({0, 1, 2, t // 2, t // 2 + 1, t - 3, t - 2, t - 1} & set(range(t)))
    for r in range(4):
        for i in rows:
            _check(c, r, i, recent)
    assert torch.isfinite(c.out[3]).all()


@pytest.mark.parametrize("t", [4, 256])
def test_behind_thousands_of_positions(t):
    """An infinity that every row of one request sees, one that most rows of another do not: status and neighbours."""
    heads, lens = (8, 2, 128), [7000, 6000, 8000, 300]
    c = Call(75, lens, t, heads=heads, sink=4, recent=WIDE)
    _put(c, 0, 1, INF)
    _put(c, 2, lens[2] - 2, NAN)
    c.device().attend()
    assert c.st.item() == 0
    assert (c.out[0] == INF).all() and torch.isfinite(c.out[1]).all() and torch.isfinite(c.out[3]).all()
    assert torch.isfinite(c.out[2, :t - 2]).all() and torch.isnan(c.out[2, t - 2:]).all()
    for r, i in ((0, 0), (1, 0), (1, t - 1), (2, 0), (2, t // 2), (2, t - 3), (3, t - 1)):
        _check(c, r, i, WIDE)


def test_values_that_overflow_the_sum():
    """Sums past fp32 stay what they are, and cost no other row anything."""
    t = 100
    c = Call(77, [400, 300], t, heads=(4, 2, 64), sink=2, recent=WIDE)
    c.c.v[c.c.table[0, :25], :, :, 7] = 3.0e38
    c.device().attend()
    assert c.st.item() == 0 and torch.isfinite(c.out[1]).all()
    assert torch.isfinite(c.out[0, :, :, :7]).all() and torch.isfinite(c.out[0, :, :, 8:]).all()
    for i in (0, t - 1):
        c.check(1, i)
