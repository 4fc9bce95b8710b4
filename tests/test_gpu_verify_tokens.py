"""Verification of drafted tokens: whole numbers, against exact arithmetic."""
import numpy as np
import pytest
import torch

from tests import window_reference as ref

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


def _i32(v):
    return torch.as_tensor(v, dtype=torch.int32).cuda()


def _problem(seed, b, t, v, drawn=True, sharp=3.0):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(b, t + 1, v, generator=g) * sharp
    target = torch.softmax(logits, -1)
    draft = torch.softmax(logits[:, :t] + torch.randn(b, t, v, generator=g) * 0.5, -1)
    tokens = torch.multinomial(draft.view(b * t, v), 1, generator=g).view(b, t) if drawn else target[:, :t].argmax(-1)
    return target, draft if drawn else None, tokens.to(torch.int32), torch.rand(b, t + 1, generator=g)


def _run(target, draft, tokens, u, n=None, **kw):
    sfi = _sfi()
    b, rows, _ = target.shape
    out, acc = _i32(np.full((b, rows), -9)), _i32([-9] * b)
    st = _i32([0])
    sfi.sfi_verify_tokens(target.cuda(), None if draft is None else draft.cuda(), tokens.cuda(), u.cuda(), out, acc,
                          draft_lens=None if n is None else _i32(n), dev_status=st, **kw)
    return out.cpu(), acc.tolist(), st.item()


def _check(target, draft, tokens, u, n, out, acc, skip=()):
    for r in range(len(acc)):
        if r in skip:
            assert acc[r] == -9 and (out[r] == -9).all()
            continue
        a, x = ref.verify(target[r].numpy(), None if draft is None else draft[r].numpy(), tokens[r].tolist(),
                          u[r].numpy(), n[r])
        want = tokens[r, :a].tolist() + [x] + [-1] * (len(tokens[r]) - a)
        assert acc[r] == a and out[r].tolist() == want, (r, a, x, out[r].tolist())


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("v", [1, 2, 31, 127, 128, 129, 1000, 1024, 2049, 5003])
@pytest.mark.parametrize("t", [1, 4])
def test_against_exact_arithmetic(v, t, drawn):
    target, draft, tokens, u = _problem(v * 10 + t, 9, t, v, drawn)
    n = [t, t, 1, t, 0, t, t, max(1, t - 1), t]
    out, acc, st = _run(target, draft, tokens, u, n)
    assert st == 0
    _check(target, draft, tokens, u, n, out, acc)


def test_a_large_vocabulary_and_many_drafts():
    target, draft, tokens, u = _problem(7, 3, 40, 40001, sharp=1.0)
    draft[:, :, :] = target[:, :40]      # equal: every draft is accepted
    target[1, 35] = torch.roll(target[1, 35], 1)
    out, acc, st = _run(target, draft, tokens, u)
    assert st == 0 and acc[0] == acc[2] == 40
    _check(target, draft, tokens, u, [40] * 3, out, acc)


def test_random_numbers_at_the_ends():
    target, draft, tokens, u = _problem(3, 6, 3, 777)
    u[0], u[1], u[2] = 0.0, 0.99999994, 2.0 ** -24
    target[3, :, :100] = 0                 # a row that begins with zeros, and a sample of 0
    u[3, 3] = 0.0
    u[4, 0] = float("nan")                 # refuses
    out, acc, st = _run(target, draft, tokens, u)
    assert st == 0 and acc[4] == 0
    _check(target, draft, tokens, u, [3] * 6, out, acc)


def test_rows_that_leave_nothing():
    """p below q everywhere (the residual is empty: p itself), p zero everywhere (no token), NaN and negative values."""
    target, draft, tokens, u = _problem(4, 5, 2, 300)
    target[0, 0] = draft[0, 0] * 0.5
    u[0, 0] = 0.9
    target[1] = 0
    target[2, :, 5] = float("nan")
    target[2, :, 7] = -1.0
    draft[3] = target[3, :2]
    u[3, 0] = 1.0                          # not below one: refused, and nothing is left of p - q
    out, acc, st = _run(target, draft, tokens, u)
    assert st == 128 and acc[1] == 0 and out[1].tolist() == [-1, -1, -1]
    _check(target, draft, tokens, u, [2] * 5, out, acc)


def test_strided_rows_lengths_and_a_subset():
    """Rows of a padded vocabulary, requests by id, lengths of the cache."""
    target, draft, tokens, u = _problem(5, 4, 3, 500)
    wide_t, wide_d = torch.zeros(4, 4, 512), torch.ones(4, 3, 544)
    wide_t[..., :500], wide_d[..., :500] = target, draft
    wide_t[..., 500:] = float("nan")
    seq, new = _i32([100, 50, 60, 70]), _i32([-9] * 4)
    n = [3, 2, 3, 1]
    sfi = _sfi()
    out, acc, st = _i32(np.full((4, 4), -9)), _i32([-9] * 4), _i32([0])
    sfi.sfi_verify_tokens(wide_t.cuda()[..., :500], wide_d.cuda()[..., :500], tokens.cuda(), u.cuda(), out, acc,
                          draft_lens=_i32(n), seq_lens=seq, new_lens=new, req_ids=_i32([2, 0, 3]), dev_status=st)
    assert st.item() == 0
    _check(target, draft, tokens, u, n, out.cpu(), acc.tolist(), skip=(1,))
    a = acc.tolist()
    assert new.tolist() == [100 - 3 + a[0], -9, 60 - 3 + a[2], 70 - 1 + a[3]]


def test_refused_requests():
    target, draft, tokens, u = _problem(6, 5, 3, 200)
    tokens[1, 2] = 200
    tokens[2, 0] = -1
    tokens[4, 2] = 5000                    # behind the request's drafts: not looked at
    n = [3, 3, 3, 4, 2]
    out, acc, st = _run(target, draft, tokens, u, n)
    assert st == 8 | 2
    _check(target, draft, tokens, u, n, out, acc, skip=(1, 2, 3))


def test_the_target_distribution_comes_out():
    """One draft, many random numbers: accepted and sampled tokens together follow p. Counts of n trials are off by
    at most six standard deviations sqrt(n p (1 - p)) (and one)."""
    v, n = 8, 40000
    g = torch.Generator().manual_seed(9)
    p, q = torch.softmax(torch.randn(v, generator=g), -1), torch.softmax(torch.randn(v, generator=g), -1)
    target, draft = p.expand(n, 2, v).contiguous(), q.expand(n, 1, v).contiguous()
    tokens = torch.multinomial(q, n, replacement=True, generator=g).view(n, 1).to(torch.int32)
    out, _, st = _run(target, draft, tokens, torch.rand(n, 2, generator=g))
    assert st == 0
    count = torch.bincount(out[:, 0].long(), minlength=v).double()
    p = p.double()
    assert ((count - n * p).abs() <= 6 * (n * p * (1 - p)).sqrt() + 1).all()
