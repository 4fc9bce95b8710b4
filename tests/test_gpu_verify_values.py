"""Verification of drafted tokens whose own probabilities are no probabilities: values count as at least 0 and at most
1, a NaN as 0, in the acceptance too."""
import itertools

import pytest
import torch

from tests.test_gpu_verify_tokens import _check, _problem, _run

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from sparse_kv_long_sfi_gb300 import build
    build.build()


def _counted(x):
    return torch.nan_to_num(x, nan=0.0, posinf=1.0, neginf=0.0).clamp(0, 1)


@pytest.mark.parametrize("drawn", [True, False])
def test_values_of_the_drafted_token(drawn):
    """Every pair of values of q and p at the draft, for a u of 0, of a half and next to 1."""
    values = [-INF, -0.5, -0.0, 0.0, 0.25, 0.75, 1.0, 1.5, INF, NAN]
    cases = list(itertools.product(values, values, [0.0, 0.5, 0.99999994]))
    target, draft, tokens, u = _problem(11, len(cases), 2, 300, drawn)
    for r, (q, p, x) in enumerate(cases):
        target[r, 0, tokens[r, 0]] = p
        u[r, 0] = x
        if drawn:
            draft[r, 0, tokens[r, 0]] = q
    out, acc, st = _run(target, draft, tokens, u)
    _check(_counted(target), None if draft is None else _counted(draft), tokens, u, [2] * len(cases), out, acc)
    nothing = [r for r, (_, p, _) in enumerate(cases) if not p > 0]
    assert all(acc[r] == 0 for r in nothing)  # what the target never says is not accepted
    if drawn:
        free = [r for r, (q, p, _) in enumerate(cases) if p > 0 and not q > 0]
        assert all(acc[r] >= 1 for r in free)
