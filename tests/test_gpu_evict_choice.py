"""Eviction over every kernel that chooses: rows up to 4096 candidates, up to 16384, and longer ones by the Selector;
short rows in wide buffers, ties, zeros of both signs, infinities and NaN; refused requests, of which nothing is written."""
import numpy as np
import pytest
import torch

from tests import window_reference as ref

pytestmark = pytest.mark.gpu
SINK, RECENT = 4, 32
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from sparse_kv_long_sfi_gb300 import build
    build.build()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Evicted:
    """One call; every output begins as -5."""

    def __init__(self, c, mass, k, k_cap=None, sink=SINK, recent=RECENT, lens=None):
        import sparse_kv_long_sfi_gb300 as sfi
        shape, kv = c.device()
        if lens is not None:
            kv.seq_lens.copy_(_i32(lens))
        b = len(k)
        idx = torch.full((b, c.hkv, max(k) if k_cap is None else k_cap), -5, dtype=torch.int32, device="cuda")
        count, new, st = _i32([-5] * b), _i32([-5] * b), _i32([0])
        out = torch.full_like(mass, -5.0, device="cuda")
        sfi.sfi_kv_evict(shape, kv, mass.cuda(), sink, recent, _i32(k), idx, count, new, mass_out=out, dev_status=st)
        self.c, self.mass, self.k, self.sink, self.recent = c, mass, k, sink, recent
        self.idx, self.count, self.new, self.out, self.status = idx.cpu(), count.tolist(), new.tolist(), out.cpu(), st.item()
        self.pools = kv.k_pool.cpu(), kv.v_pool.cpu()

    def check(self, skip=()):
        c = self.c
        for r in range(len(self.k)):
            if r in skip:
                self.untouched(r)
                continue
            n = c.lens[r]
            lo, hi = min(self.sink, n), max(min(self.sink, n), n - self.recent)
            pages = torch.from_numpy(c.table[r].astype(np.int64))
            for h in range(c.hkv):
                w = self.mass[r, h, lo:hi].numpy().astype(np.float64)
                nan = np.isnan(w)
                order = np.lexsort((np.arange(hi - lo), -np.where(nan, 0, w), nan))
                best = np.sort(order[:self.k[r]]) + lo
                kept = np.concatenate([np.arange(lo), best, np.arange(hi, n)])
                assert self.count[r] == len(best) and self.new[r] == len(kept)
                assert (self.idx[r, h, :len(best)].numpy() == best).all() and (self.idx[r, h, len(best):] == -5).all()
                assert np.array_equal(self.out[r, h, :len(kept)].numpy(), self.mass[r, h, kept].numpy(), equal_nan=True)
                assert (self.out[r, h, len(kept):] == -5).all()
                for was, now in zip((c.k, c.v), self.pools):
                    was, now = (x[pages, h].reshape(-1, c.d).view(torch.int16) for x in (was, now))
                    assert torch.equal(now[:len(kept)], was[kept]) and torch.equal(now[len(kept):n], was[len(kept):n])

    def untouched(self, r):
        """Nothing of a refused request has changed."""
        assert self.count[r] == self.new[r] == -5 and (self.idx[r] == -5).all() and (self.out[r] == -5).all()
        pages = torch.from_numpy(self.c.table[r][:-(-self.c.lens[r] // 16)].astype(np.int64))
        for was, now in zip((self.c.k, self.c.v), self.pools):
            assert torch.equal(was[pages].view(torch.int16), now[pages].view(torch.int16))


def _weights(kind, b, hkv, n, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "few values":
        return torch.randint(0, 40, (b, hkv, n), generator=g).float() / 8
    if kind == "all equal":
        return torch.full((b, hkv, n), 0.375)
    if kind == "one digit":  # keys that differ in their lowest byte alone
        return (torch.randint(0, 200, (b, hkv, n), generator=g, dtype=torch.int32) + 0x3f800000).view(torch.float32)
    w = torch.randn(b, hkv, n, generator=g)
    if kind == "special":
        pick = torch.randint(0, 12, (b, hkv, n), generator=g)
        for i, x in enumerate((NAN, -NAN, INF, -INF, 0.0, -0.0, 1e-45)):
            w = torch.where(pick == i, torch.tensor(x), w)
    return w


KINDS = ["any", "few values", "all equal", "one digit", "special"]
EDGES = [4095, 4096, 4097, 9000, 16383, 16384, 16385, 32768, 40001]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("candidates", EDGES)
def test_rows_as_long_as_the_buffer(candidates, kind):
    """The longest row fills the weights, on both sides of each choice's limit."""
    n = candidates + SINK + RECENT
    lens = [n, n - 1, max(100, n // 3)]
    c = ref.Cache(81, lens, 2, 2, 64)
    mass = _weights(kind, 3, 2, n, candidates)
    for k in ([candidates // 8, 1000, 700], [candidates - 1, 1, 0]):
        e = Evicted(c, mass, k)
        assert e.status == 0
        e.check()


@pytest.mark.parametrize("width", [300, 4096 + SINK + RECENT + 1, 16384 + SINK + RECENT, 16384 + SINK + RECENT + 1, 70001])
def test_short_rows_in_wide_buffers(width):
    """What the buffer's width chooses makes no difference."""
    lens = [0, 1, 36, 37, 100, 255, 300, 290]
    c = ref.Cache(83, lens, 8, 2, 128)
    mass = _weights("special", 8, 2, width, 5)
    e = Evicted(c, mass, [5, 5, 5, 1, 20, 200, 100, 300])
    assert e.status == 0
    e.check()


@pytest.mark.parametrize("width", [400, 9000, 20000])
def test_nothing_of_a_refused_request_is_written(width):
    """Lengths beyond the table but within the weights, below zero; more rows than idx holds."""
    lens = [200, 300, 250, 260]
    c = ref.Cache(85, lens, 8, 2, 64)
    assert c.table.shape[1] * 16 == 320
    mass, k = _weights("any", 4, 2, width, 6), [50, 60, 70, 80]
    for r, length, bit in ((1, 321, 2), (2, width, 2), (0, width + 1, 2), (3, -1, 2)):
        e = Evicted(c, mass, k, lens=[length if i == r else n for i, n in enumerate(lens)])
        assert e.status == bit, (r, length)
        e.check(skip=(r,))
    e = Evicted(c, mass, [50, 60, 91, 80], k_cap=90)
    assert e.status == 4
    e.check(skip=(2,))
    e = Evicted(c, mass, [50, -1, 70, 80])
    assert e.status == 4
    e.check(skip=(1,))


@pytest.mark.parametrize("more", [0, 1])
def test_the_most_candidates(more):
    """262144 candidates are taken, one more is not; the other request is cut all the same."""
    n = 262144 + more + SINK + RECENT
    c = ref.Cache(87, [n, 500], 1, 1, 64)
    e = Evicted(c, _weights("any", 2, 1, n, 7), [3000, 100])
    assert e.status == 4 * more
    e.check(skip=(0,) if more else ())
