"""Eviction by attention weight, bit for bit."""
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
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _evict(c, mass, sink, recent, k, k_cap=None, with_mass=True, st=None, **kw):
    sfi = _sfi()
    shape, kv = c.device()
    b = len(c.lens)
    idx = torch.full((b, c.hkv, max(k) if k_cap is None else k_cap), -5, dtype=torch.int32, device="cuda")
    count, new = _i32([-5] * b), _i32([-5] * b)
    out = torch.full_like(mass, -5.0).cuda() if with_mass else None
    st = _i32([0])
    sfi.sfi_kv_evict(shape, kv, mass.cuda(), sink, recent, _i32(k), idx, count, new, mass_out=out, dev_status=st, **kw)
    return kv, idx.cpu(), count.tolist(), new.tolist(), None if out is None else out.cpu(), st.item()


def _check(c, kv, idx, count, new, out, mass, sink, recent, k, skip=()):
    b, hkv = len(c.lens), c.hkv
    wk, wv = c.k.clone(), c.v.clone()
    for r in range(b):
        if r in skip:
            assert new[r] == -5
            continue
        for h in range(hkv):
            kept, best = ref.keep(mass[r, h].double().tolist(), c.lens[r], sink, recent, k[r])
            assert new[r] == len(kept) and count[r] == len(best), (r, h)
            assert idx[r, h, :len(best)].tolist() == best, (r, h)
            assert (idx[r, h, len(best):] == -5).all()
            for pool, want in ((c.k, wk), (c.v, wv)):
                for i, j in enumerate(kept):
                    want[c.table[r, i // 16], h, i % 16] = pool[c.table[r, j // 16], h, j % 16]
            if out is not None:
                assert torch.equal(out[r, h, :len(kept)], mass[r, h, kept]), (r, h)
                assert (out[r, h, len(kept):] == -5).all()
    same = lambda a, z: torch.equal(a.cpu().view(torch.int16), z.view(torch.int16))  # noqa: E731
    assert same(kv.k_pool, wk) and same(kv.v_pool, wv)


def _mass(seed, b, hkv, n):
    """Few different values, so that many are equal."""
    return torch.randint(0, 40, (b, hkv, n), generator=torch.Generator().manual_seed(seed)).float() / 8


@pytest.mark.parametrize("heads", [(16, 8, 128), (8, 2, 64), (1, 1, 128)])
@pytest.mark.parametrize("sink,recent", [(4, 32), (0, 0), (17, 1), (64, 100), (1000, 3), (0, 5000)])
def test_rows_move_in_order(heads, sink, recent):
    """Lengths around pages, chunks and windows; from nothing kept to everything kept."""
    lens = [0, 1, 17, 100, 160, 700, 1030, 2500]
    c = ref.Cache(21, lens, *heads)
    for k in ([5, 0, 1, 10, 60, 300, 900, 1500], [0] * 8, [3000] * 8, [1] * 8):
        mass = _mass(3, len(lens), heads[1], max(lens) + 2)
        got = _evict(c, mass, sink, recent, k)
        assert got[-1] == 0
        _check(c, *got[:-1], mass, sink, recent, k)


def test_one_row_out_of_each():
    """All but one candidate kept: nearly every row moves by one place."""
    lens, k = [900, 901, 1000], [899 - 36, 900 - 36, 999 - 36]
    c = ref.Cache(23, lens, 16, 8, 128)
    mass = torch.rand(3, 8, 1000, generator=torch.Generator().manual_seed(1))
    got = _evict(c, mass, 4, 32, k)
    _check(c, *got[:-1], mass, 4, 32, k)


def test_many_units_and_whole_rows():
    """Enough units for whole rows per CTA."""
    lens = [300 + i for i in range(40)]
    c = ref.Cache(25, lens, 8, 8, 64)
    k = [100 + i for i in range(40)]
    mass = _mass(4, 40, 8, 340)
    got = _evict(c, mass, 8, 20, k, with_mass=False)
    _check(c, *got[:-1], mass, 8, 20, k)


def test_a_subset_and_refused_requests():
    """Requests by id; a length beyond the table or the weights, more rows than idx holds."""
    lens = [200, 300, 250, 260, 270]
    c = ref.Cache(27, lens, 8, 2, 64)
    mass = _mass(5, 5, 2, 300)
    k = [50, 60, 70, 80, 90]
    got = _evict(c, mass, 4, 16, k, req_ids=_i32([3, 0]))
    assert got[-1] == 0
    _check(c, *got[:-1], mass, 4, 16, k, skip=(1, 2, 4))
    real = list(lens)
    for r, bad, what in ((1, 300 + 32, 2), (2, -1, 2)):
        c.lens[r] = bad
        got = _evict(c, mass, 4, 16, k)
        c.lens[r] = real[r]
        assert got[-1] & what, (r, bad)
        kv, idx, count, new, out, _ = got
        wants = [new[i] for i in range(5) if i != r]
        assert wants == [4 + k[i] + 16 for i in range(5) if i != r] and new[r] == -5
    got = _evict(c, mass, 4, 16, [50, 60, 91, 80, 90], k_cap=90)
    assert got[-1] == 4 and got[3][2] == -5 and got[3][1] == 80


def test_a_bad_page_stays_as_it_was():
    lens, k = [200], [50]
    c = ref.Cache(29, lens, 8, 2, 64)
    mass = _mass(6, 1, 2, 200)
    c.table[0, 7] = c.pages + 3
    kv, _, _, new, _, st = _evict(c, mass, 4, 16, k)
    assert st == 1 and new == [70]
    kept, _ = ref.keep(mass[0, 0].double().tolist(), 200, 4, 16, 50)
    page0 = c.table[0, 0]
    for i in range(16):
        j = kept[i]
        if j // 16 != 7:
            assert torch.equal(kv.k_pool[page0, 0, i].cpu(), c.k[c.table[0, j // 16], 0, j % 16])
