"""Accumulated attention weights, against fp64."""
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


def _expected(cache, q, lse, new, sink, recent, mass, decay):
    """mass in fp64 and a bound of the kernel's error. A weight is exp(x - lse): the score's error (d products in
    fp32, each sum off by 2^-23 of the magnitudes), the argument's roundings (2^-24 of |x| and |lse|, a few times, in
    log2 units) and the exponential's 2^-22 count relative to it; sums add 2^-24 for each of at most rows / 4 + 8
    additions in a chain."""
    b, t = q.shape[:2]
    g = cache.hq // cache.hkv
    want, bound = mass.double().numpy().copy(), np.zeros(mass.shape)
    for r in range(b):
        n, length = new[r], cache.lens[r]
        old = want[r, :, :length] * decay
        old[:, length - n:] = 0
        bound[r, :, :length] = 2.0 ** -23 * np.abs(old)
        want[r, :, :length] = old
        for h in range(cache.hkv):
            k = cache.rows(cache.k, r, h)
            total, err = np.zeros(length), np.zeros(length)
            for i in range(n):
                see = ref.sees(length - n + i, length, sink, recent)
                for j in range(h * g, h * g + g):
                    qd = q[r, i, j].double().numpy()
                    x = k @ qd / np.sqrt(cache.d)
                    e = float(lse[r, i, j])
                    w = np.where(see, np.exp(x - e), 0)
                    rel = (2 * cache.d * 2.0 ** -24 * (np.abs(k) @ np.abs(qd)) / np.sqrt(cache.d)
                           + 2.0 ** -21 + 4 * 2.0 ** -24 * (np.abs(x) + abs(e)))
                    total += w
                    err += w * rel
            want[r, h, :length] += total
            bound[r, h, :length] += err + 2.0 ** -24 * (n * g / 4 + 16) * total
    return want, bound + 1e-30


def _problem(seed, lens, heads, new, sink, recent, t):
    c = ref.Cache(seed, lens, *heads, fill=float("nan"))
    q = ref.queries(seed + 1, len(lens), t, heads[0], heads[2])
    lse = torch.zeros(len(lens), t, heads[0])
    for r in range(len(lens)):
        for i in range(new[r]):
            for h in range(heads[0]):
                lse[r, i, h] = ref.token(c, r, h, q[r, i, h], lens[r] - new[r] + i, sink, recent)[1]
    return c, q, lse


def _run(cache, q, lse, new, sink, recent, mass, decay, **kw):
    sfi = _sfi()
    shape, kv = cache.device()
    out = mass.cuda()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    sfi.sfi_attn_mass(shape, kv, sink, recent, q.cuda(), lse.cuda(), out, decay=decay, dev_status=st,
                      new_lens=None if new is None else torch.tensor(new, dtype=torch.int32, device="cuda"), **kw)
    return out.cpu(), st.item()


def _check(got, want, bound, lens, mass):
    for r, n in enumerate(lens):
        bad = np.abs(got[r, :, :n].double().numpy() - want[r, :, :n]) > bound[r, :, :n]
        bad |= ~np.isfinite(got[r, :, :n].numpy())
        assert not bad.any(), (r, np.argwhere(bad)[:5], got[r, :, :n].numpy()[bad][:5], want[r, :, :n][bad][:5])
        assert torch.equal(got[r, :, n:], mass[r, :, n:]), r


@pytest.mark.parametrize("heads,t", [((16, 8, 128), 1), ((16, 8, 128), 9), ((8, 2, 64), 16), ((8, 1, 128), 3),
                                     ((2, 2, 64), 33), ((8, 2, 64), 90)])
@pytest.mark.parametrize("sink,recent,decay", [(4, 32, 1.0), (0, 1 << 30, 0.5), (17, 1, 0.0), (300, 5, 1.0)])
def test_against_fp64(heads, t, sink, recent, decay):
    """Every width of the query tile, ragged requests (one without new tokens), lengths around pages and blocks."""
    lens = [t, max(300, t), 256 + t, t + 15, 513]
    new = [t, t, max(1, t // 2), 0, max(1, t - 1)]
    c, q, lse = _problem(11, lens, heads, new, sink, recent, t)
    mass = torch.rand(len(lens), heads[1], max(lens) + 3, generator=torch.Generator().manual_seed(5))
    got, st = _run(c, q, lse, new, sink, recent, mass, decay)
    assert st == 0
    _check(got, *_expected(c, q, lse, new, sink, recent, mass, decay), lens, mass)


@pytest.mark.parametrize("heads", [(4, 2, 128), (8, 1, 64)])
def test_long_prompts(heads):
    """More query tiles than the ring and the double buffer hold."""
    t, lens, new = 700, [700, 900, 1030], [700, 650, 5]
    c, q, lse = _problem(13, lens, heads, new, 3, 1 << 30, t)
    mass = torch.zeros(len(lens), heads[1], max(lens))
    got, st = _run(c, q, lse, new, 3, 1 << 30, mass, 1.0)
    assert st == 0
    _check(got, *_expected(c, q, lse, new, 3, 1 << 30, mass, 1.0), lens, mass)
    again, _ = _run(c, q, lse, new, 3, 1 << 30, mass, 1.0)
    assert torch.equal(got, again)
    # a token's weights sum to one
    total = torch.stack([got[r, :, :n].double().sum() for r, n in enumerate(lens)])
    assert torch.allclose(total, torch.tensor(new, dtype=torch.float64) * heads[0], rtol=1e-5)


def test_a_nan_that_no_query_sees_stays_alone():
    """NaN keys outside the window, and query rows behind the request's tokens."""
    heads, t, lens, new = (16, 8, 128), 40, [400, 400], [40, 30]
    sink, recent = 2, 50
    c, q, lse = _problem(17, lens, heads, new, sink, recent, t)
    mass = torch.rand(2, 8, 400, generator=torch.Generator().manual_seed(6))
    want = _expected(c, q, lse, new, sink, recent, mass, 1.0)
    for r in range(2):  # positions that none of the new tokens sees
        for j in range(2, lens[r] - new[r] + 1 - recent):
            c.k[c.table[r, j // 16], :, j % 16] = float("nan")
    q[1, 30:] = float("nan")
    lse[1, 30:] = float("nan")
    got, st = _run(c, q, lse, new, sink, recent, mass, 1.0)
    assert st == 0
    _check(got, *want, lens, mass)


@pytest.mark.parametrize("heads,d_lens", [((8, 2, 64), (300, 560)), ((4, 2, 128), (128, 400))])
def test_more_blocks_than_the_gpu_holds(heads, d_lens):
    """Many requests in a call of more than 128 query rows: a CTA works through several blocks, of all lengths."""
    t = 160 * heads[1] // heads[0]
    g = torch.Generator().manual_seed(21)
    lens = torch.randint(*d_lens, (60,), generator=g).tolist()
    new = [0 if r % 11 == 3 else min(t, lens[r]) - r % 7 for r in range(60)]
    c, q, lse = _problem(22, lens, heads, new, 5, 200, t)
    mass = torch.rand(60, heads[1], max(lens) + 5, generator=g)
    got, st = _run(c, q, lse, new, 5, 200, mass, 0.5)
    assert st == 0
    _check(got, *_expected(c, q, lse, new, 5, 200, mass, 0.5), lens, mass)
    again, _ = _run(c, q, lse, new, 5, 200, mass, 0.5)
    assert torch.equal(got, again)
