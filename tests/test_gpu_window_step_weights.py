"""A step's weights keep more bits than bf16 has: its output is off by its own rounding, not by theirs."""
import numpy as np
import pytest
import torch

from tests import window_reference as ref
from tests.test_gpu_window_attn import _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from sparse_kv_long_sfi_gb300 import build
    build.build()


@pytest.mark.parametrize("heads,t", [((16, 8, 128), 1), ((8, 2, 64), 1), ((8, 1, 128), 1), ((2, 2, 64), 8), ((8, 2, 64), 4),
                                     ((16, 8, 128), 5)])
@pytest.mark.parametrize("sink,recent", [(4, 256), (0, 1 << 20)])
def test_weights_in_two_terms(heads, t, sink, recent):
    """Half a bf16 step of the output, and of the sum of |w v|: the weights' two terms (2^-16), scores and sums in fp32
    (a score's error of d 2^-23 of its magnitude counts relative to its weight), the exponential (2^-22), and 2^-20 for
    the sums. A single bf16 term would be off by up to 2^-8 of that sum."""
    lens = [40, 300, 1500]
    c = ref.Cache(101, lens, *heads)
    q = ref.queries(102, len(lens), t, heads[0], heads[2])
    out, _, st = _run(c, q, None, sink, recent)
    assert st == 0
    for r, n in enumerate(lens):
        for i in range(t):
            for h in range(heads[0]):
                o, _, _, mag, smag = ref.token(c, r, h, q[r, i, h], n - t + i, sink, recent)
                err = np.abs(out[r, i, h].double().numpy() - o)
                own = 2.0 ** -16 + 2 * (c.d * 2.0 ** -23 * smag) + 2.0 ** -20
                assert (err <= 2.0 ** -8 * np.abs(o) + own * mag).all(), (r, i, h, (err / mag).max())
