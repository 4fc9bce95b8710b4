"""Attention through a sliding window with sinks, against fp64."""
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


def _run(cache, q, new, sink, recent, **kw):
    sfi = _sfi()
    shape, kv = cache.device()
    b, t = q.shape[:2]
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((b, t, cache.hq), 7.0, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    sfi.sfi_window_attn(shape, kv, sink, recent, q.cuda(), out, lse=lse, dev_status=st,
                        new_lens=None if new is None else torch.tensor(new, dtype=torch.int32, device="cuda"), **kw)
    torch.cuda.synchronize()
    return out.cpu(), lse.cpu(), st.item()


def _check(cache, q, new, sink, recent, out, lse, tokens=None, skip=()):
    b, t = q.shape[:2]
    for r in range(b):
        n = t if new is None else new[r]
        for i in range(t):
            if i >= n or r in skip:  # not the request's: as it was
                assert (out[r, i] == 7).all() and (lse[r, i] == 7).all(), (r, i)
                continue
            if tokens is not None and i not in tokens:
                continue
            p = cache.lens[r] - n + i
            for h in range(cache.hq):
                o, x, _, mag, smag = ref.token(cache, r, h, q[r, i, h], p, sink, recent)
                err = np.abs(out[r, i, h].double().numpy() - o)
                bad = err > ref.out_bound(o, mag, cache.d)
                assert not bad.any(), (r, i, h, p, err.max(), o[bad][:3])
                got = float(lse[r, i, h])
                assert got == x or abs(got - x) <= ref.lse_bound(x, smag, cache.d), (r, i, h, got, x)


HEADS = [(16, 8, 128), (8, 2, 64), (8, 1, 128), (2, 2, 64)]


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("sink,recent", [(4, 32), (0, 1), (17, 40), (0, 1 << 20), (64, 256), (5, 0), (2 ** 31 - 1, 3)])
def test_a_step(heads, sink, recent):
    """One token per request: lengths around pages, windows and sinks."""
    lens = [1, 2, 15, 16, 17, 33, 64, 65, 300, 511]
    c = ref.Cache(1, lens, *heads)
    q = ref.queries(2, len(lens), 1, heads[0], heads[2])
    out, lse, st = _run(c, q, None, sink, recent)
    assert st == 0
    _check(c, q, None, sink, recent, out, lse)


@pytest.mark.parametrize("heads,t", [((16, 8, 128), 8), ((8, 2, 64), 4), ((8, 1, 128), 2), ((2, 2, 64), 16)])
@pytest.mark.parametrize("sink,recent", [(4, 32), (0, 1), (30, 3), (0, 1 << 20)])
def test_drafted_tokens(heads, t, sink, recent):
    """Several tokens of a step, ragged (none of some requests)."""
    new = [t, 1, 0, max(1, t - 1), t]
    lens = [t, 50, 20, 333, 129]
    c = ref.Cache(3, lens, *heads, fill=float("nan"))
    q = ref.queries(4, len(lens), t, heads[0], heads[2])
    out, lse, st = _run(c, q, new, sink, recent)
    assert st == 0
    _check(c, q, new, sink, recent, out, lse)


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("sink,recent", [(4, 32), (0, 1 << 20), (64, 100), (17, 1), (130, 20)])
def test_prompts(heads, sink, recent):
    """Prompts and chunks behind context, of lengths around the tiles, ragged; stale bytes spell NaN."""
    t = 300
    new = [300, 1, 129, 0, 257, 17]
    lens = [300, 90, 129, 40, 700, 145]
    c = ref.Cache(5, lens, *heads, fill=float("nan"))
    q = ref.queries(6, len(lens), t, heads[0], heads[2])
    out, lse, st = _run(c, q, new, sink, recent)
    assert st == 0
    some = set(range(0, 300, 37)) | {0, 1, 15, 16, 17, 31, 32, 63, 64, 127, 128, 129, 255, 256, 299}
    _check(c, q, new, sink, recent, out, lse, tokens=some)


@pytest.mark.parametrize("heads", [(8, 1, 64), (4, 4, 128)])
def test_prompts_of_other_groups(heads):
    """Eight heads of a group in 64 dims, and none shared in 128."""
    t, new, lens = 140, [140, 33, 65, 2], [140, 400, 65, 1000]
    c = ref.Cache(31, lens, *heads, fill=float("nan"))
    q = ref.queries(32, len(lens), t, heads[0], heads[2])
    out, lse, st = _run(c, q, new, 20, 70)
    assert st == 0
    _check(c, q, new, 20, 70, out, lse)
