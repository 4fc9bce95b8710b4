"""The 4-bit cache against plain numpy in 64 bits: append and read to the bit, compaction to
the bit, dense and sparse attention, one to sixteen query rows, ragged lengths, garbage and
NaN behind the mask, subsets, graphs, refusals.

Tolerances. The kernel works on the same codes as the reference, and its products are exact.
A logit is a sum of D products in fp32 (the matrix instruction rounds towards zero, 2^-23):
|dx| <= D 2^-23 scale sum |q k|. A probability is then off by 2 max |dx| (its own and the
normaliser's), 2^-21 for the exponential and 2^-21 for its two fp16 terms, and the output's
sum adds at most (n / 8 + 64) 2^-23 (two matrix steps per 16 tokens, and the merges), all
relative to sum p |v|. A probability is taken times 2^7 over that of the running maximum, so
that the normaliser is at least 2^7; its second fp16 term ends at fp16's last bit, 2^-24,
half of which is lost: each token adds up to 2^-25 / 2^7 |v| = 2^-32 |v| however small its
probability. The log-sum-exp has the same relative error inside its logarithm, and
its own rounding (2^-22 of its value)."""
import math

import numpy as np
import pytest
import torch

from tests import kv4_reference as ref
from tests.gpu_harness import dev_i32, dev_i64

pytestmark = pytest.mark.gpu

SENTINEL = -7.0e30


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from sparse_kv_long_sfi_gb300 import build
    build.build()


def _sfi():
    import sparse_kv_long_sfi_gb300 as sfi
    return sfi


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


class Cache:
    """A 4-bit pool of random codes and plausible scales; everything behind the lengths is
    arbitrary bytes, NaN scales among them."""

    def __init__(self, seed, lens, hkv, d, g_k=1.0, g_v=1.0, spare=3):
        self.rng = np.random.default_rng(seed)
        self.lens, self.hkv, self.d, self.g_k, self.g_v = list(lens), hkv, d, g_k, g_v
        need = [max(1, -(-n // 16)) for n in lens]
        pages = sum(need) + spare
        ids = self.rng.permutation(pages)
        self.table = np.full((len(lens), max(need)), -1, np.int32)
        at = 0
        for r, n in enumerate(need):
            self.table[r, :n] = ids[at:at + n]
            at += n
        self.pool = self.rng.integers(0, 256, (pages, hkv, 18 * d)).astype(np.uint8)
        sk, sv = (o[2] for o in ref.offsets(d))
        lo, hi = int(np.searchsorted(ref.E4M3, 0.05)), int(np.searchsorted(ref.E4M3, 0.5))
        for r, L in enumerate(lens):
            for pos in range(L):
                blk, row = self.pool[self.table[r, pos // 16]], pos % 16
                for s in (sk, sv):
                    blk[:, s[row, ::16]] = self.rng.integers(lo, hi, (hkv, d // 16))
        self.upload()

    def upload(self):
        sfi = _sfi()
        self.d_pool = torch.from_numpy(self.pool).cuda()
        # entries behind a request's pages are never followed
        self.kv = sfi.PagedKV4(self.d_pool, dev_i32(self.table), dev_i32(self.lens), self.g_k, self.g_v)

    def rows(self, r):
        return ref.positions(self.pool, self.table[r], self.lens[r], self.d, self.g_k, self.g_v)


def _bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16)


# ---- append and read --------------------------------------------------------------------------------------------

def _hard_rows(rng, n, h, d, g):
    """Rows of all sorts: normal, zero, tiny, huge, halfway values, infinities and NaN."""
    x = rng.standard_normal((n, h, d)) * np.exp(rng.uniform(-6, 6, (n, h, 1)))
    kinds = rng.integers(0, 12, (n, h, d // 16))
    halves = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    for i, j, k in np.argwhere(kinds < 8):
        c, sl = kinds[i, j, k], slice(16 * k, 16 * k + 16)
        if c == 0:
            x[i, j, sl] = 0 if rng.random() < 0.5 else -0.0
        elif c == 1:
            x[i, j, sl] *= 2.0 ** -14 * g
        elif c == 2:
            x[i, j, sl] *= 2.0 ** 14 * g
        elif c in (3, 4):  # a scale of (8..15) 2^e and values halfway between codes
            s = rng.integers(8, 16) * 2.0 ** rng.integers(-6, 3) * g
            x[i, j, sl] = rng.choice(halves, 16) * rng.choice([-1, 1], 16) * s
            x[i, j, 16 * k] = 6 * s
        elif c == 5 and rng.random() < 0.3:
            x[i, j, 16 * k + rng.integers(16)] = rng.choice([np.inf, -np.inf, np.nan])
        elif c == 6:  # amax / 6 halfway between two scales
            x[i, j, sl] = rng.uniform(-1, 1, 16)
            x[i, j, 16 * k + 3] = 6 * (2 * rng.integers(8, 16) + 1) * 2.0 ** -6 * g
    return _bf16(x)


@pytest.mark.parametrize("hkv,d,T,new,ctx,g_k,g_v", [
    (8, 128, 1, [1, 1, 1, 1], [0, 15, 16, 1000], 1.0, 1.0),
    (2, 64, 1, [1, 0, 1], [7, 3, 31], 0.25, 8.0),
    (1, 128, 40, [40, 17, 0, 1, 33], [5, 0, 9, 31, 15], 1.0, 0.5),
    (3, 64, 65, [64, 65, 2], [0, 15, 14], 2.0, 1.0),
])
def test_append_and_read_to_the_bit(hkv, d, T, new, ctx, g_k, g_v):
    sfi = _sfi()
    rng = np.random.default_rng(d + T)
    B = len(new)
    lens = [c + n for c, n in zip(ctx, new)]
    c = Cache(3, lens, hkv, d, g_k, g_v)
    k, v = (_hard_rows(rng, B * T, hkv, d, g).view(B, T, hkv, d) for g in (g_k, g_v))
    want = c.pool.copy()
    for r in range(B):
        for t in range(new[r]):
            pos = ctx[r] + t
            for h in range(hkv):
                blk = want[c.table[r, pos // 16], h]
                for which, (x, g) in enumerate(((k, g_k), (v, g_v))):
                    code, scale = ref.quantise(x[r, t, h].double().numpy()[None], g)
                    ref.write_rows(blk, which, [pos % 16], code, scale)
    st, shape = _status(), sfi.AttnShape(hkv, hkv, d)
    sfi.sfi_kv4_append(shape, c.kv, k.cuda(), v.cuda(), new_lens=dev_i32(new), dev_status=st)
    torch.cuda.synchronize()
    got = c.d_pool.cpu().numpy()
    bad = np.argwhere(got != want)
    assert len(bad) == 0 and st.item() == 0, (len(bad), bad[:5], got[tuple(bad[0])], want[tuple(bad[0])])
    # read back the new rows and what lies around them
    c.pool = want
    first = [max(0, x - 3) for x in ctx]
    n = T + 5
    ko, vo = (torch.full((B, n, hkv, d), 777.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    sfi.sfi_kv4_read(shape, c.kv, ko, vo, first=dev_i32(first), dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    for r in range(B):
        m = min(n, lens[r] - first[r])
        for got, x in zip((ko, vo), c.rows(r)):
            w = x[:, first[r]:first[r] + m].swapaxes(0, 1)
            assert np.array_equal(got[r, :m].double().cpu().numpy(), w, equal_nan=True)
            assert (got[r, max(m, 0):] == 777.0).all()


def test_append_without_new_lens_and_subset():
    sfi = _sfi()
    c = Cache(4, [20, 33, 18], 2, 64)
    k, v = (_bf16(np.random.default_rng(i).standard_normal((3, 18, 2, 64))) for i in (1, 2))
    shape, before = sfi.AttnShape(2, 2, 64), c.pool.copy()
    sfi.sfi_kv4_append(shape, c.kv, k.cuda(), v.cuda(), req_ids=dev_i32([2, 1]))
    c.pool = c.d_pool.cpu().numpy()
    for r in (1, 2):
        for x, src in zip(c.rows(r), (k, v)):
            code, scale = ref.quantise(src[r].double().numpy(), 1.0)
            assert np.array_equal(x[:, -18:].swapaxes(0, 1), ref.values(code, scale, 1.0))
    assert np.array_equal(c.pool[c.table[0, :2]], before[c.table[0, :2]])


# ---- attention --------------------------------------------------------------------------------------------------

def _check_attention(c, q, out, lse, T, G, scale, sets, scores=None, sink=0, recent=0, rows=None):
    """sets(r, h, t) -> (K, V, seen) as the token sees them."""
    q, out, lse = (x.double().cpu().numpy() for x in (q, out, lse))
    sc = None if scores is None else scores.double().cpu().numpy()
    for r in range(len(c.lens)) if rows is None else rows:
        for h in range(c.hkv):
            total, slack = 0.0, 0.0
            for t in range(T):
                k, v, seen = sets(r, h, t)
                hs = slice(h * G, (h + 1) * G)
                o, e, x, bound, dx, eps = ref.attend(q[r, t, hs], k, v, seen, scale)
                err = np.abs(out[r, t, hs] - o)
                assert np.isfinite(out[r, t, hs]).all() and (err <= bound).all(), ("out", r, h, t, (err / bound).max())
                if np.isfinite(e).all():
                    el = np.abs(lse[r, t, hs] - e)
                    assert (el <= eps + 2.0 ** -22 * np.abs(e) + 2.0 ** -22).all(), ("lse", r, h, t, el)
                else:
                    assert (lse[r, t, hs] == e).all()
                if sc is not None:
                    total = total + np.where(seen, x.sum(0), 0.0)
                    slack = slack + np.where(seen, dx.sum(0), 0.0)
            if sc is not None:
                L = c.lens[r]
                pos = np.arange(L)
                cand = (pos >= sink) & (pos < L - recent)
                got = sc[r, h, :L]
                assert (got[~cand] == -np.inf).all()
                assert (np.abs(got - total)[cand] <= (slack + T * G * 2.0 ** -23 * np.abs(total) + 1e-30)[cand]).all()
                assert (sc[r, h, L:] == np.float32(SENTINEL)).all()


def _dense_sets(c, T):
    cache = {}

    def sets(r, h, t):
        if r not in cache:
            cache.clear()
            cache[r] = c.rows(r)
        k, v = cache[r]
        return k[h], v[h], np.arange(c.lens[r]) < c.lens[r] - T + 1 + t
    return sets


def _dense(c, G, T, sink=4, recent=32, scores=False, seed=0, scale=0.0, **kw):
    sfi = _sfi()
    B, hq = len(c.lens), c.hkv * G
    shape = sfi.AttnShape(hq, c.hkv, c.d, softmax_scale=scale)
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(B, T, hq, c.d, generator=g).to(torch.bfloat16).cuda()
    out = torch.full((B, T, hq, c.d), SENTINEL, device="cuda")
    lse = torch.full((B, T, hq), SENTINEL, device="cuda")
    sc = torch.full((B, c.hkv, max(c.lens) + 5), SENTINEL, device="cuda") if scores else None
    ws = sfi.alloc_kv4_workspace(shape, B, T)
    st = _status()
    sfi.sfi_kv4_dense_attn(shape, c.kv, sink, recent, q, out, lse=lse, scores=sc, workspace=ws, dev_status=st, **kw)
    torch.cuda.synchronize()
    n = 512 * c.hkv * 4
    assert not ws[:n].any(), "the counters are left zero"
    return shape, q, out, lse, sc, ws, st


@pytest.mark.parametrize("d,hkv,G,T,lens,scores", [
    (128, 8, 2, 1, [1, 2, 15, 16, 17, 300], True),
    (128, 2, 1, 1, [1], False),
    (128, 1, 8, 1, [5000], True),
    (64, 2, 4, 1, [1000, 33], True),
    (64, 1, 1, 1, [16], True),
    (128, 2, 4, 4, [4, 5, 16, 19, 700], True),
    (128, 8, 2, 8, [2000, 8, 31], True),
    (64, 2, 1, 16, [16, 17, 1500], True),
    (64, 2, 8, 2, [2, 3, 444], False),
    (128, 1, 4, 3, [3, 50, 1234], True),
    (64, 4, 2, 5, [97], True),
    (128, 4, 1, 9, [9, 40], False),
])
def test_dense_attention(d, hkv, G, T, lens, scores):
    c = Cache(10 * hkv + T, lens, hkv, d, 2.0, 0.5)
    shape, q, out, lse, sc, _, st = _dense(c, G, T, scores=scores, seed=T)
    assert st.item() == 0
    _check_attention(c, q, out, lse, T, G, 1 / math.sqrt(d), _dense_sets(c, T), sc, 4, 32)


def test_large_logits_and_softmax_scale():
    """Logits of several hundred: the running maximum moves often, most probabilities vanish."""
    c = Cache(77, [900, 64], 2, 64, 64.0, 2.0 ** -9)
    shape, q, out, lse, sc, _, st = _dense(c, 4, 2, scores=True, scale=0.3)
    assert st.item() == 0
    _check_attention(c, q, out, lse, 2, 4, 0.3, _dense_sets(c, 2), sc, 4, 32)


@pytest.mark.parametrize("factor", [2.0 ** -126, 2.0 ** -60, 2.0 ** 100, 0.0])
def test_query_magnitudes(factor):
    """Queries far from 1: the power of two that brings a row into fp16 loses nothing."""
    sfi = _sfi()
    c = Cache(78, [130], 2, 128)
    shape = sfi.AttnShape(4, 2, 128, softmax_scale=0.05 / factor if 2.0 ** -100 < factor else 1.0)
    q = (torch.randn(1, 1, 4, 128, generator=torch.Generator().manual_seed(2)) * factor).to(torch.bfloat16).cuda()
    out, lse = torch.empty(1, 1, 4, 128, device="cuda"), torch.empty(1, 1, 4, device="cuda")
    sfi.sfi_kv4_dense_attn(shape, c.kv, 0, 0, q, out, lse=lse, workspace=sfi.alloc_kv4_workspace(shape, 1))
    _check_attention(c, q, out, lse, 1, 2, shape.softmax_scale, _dense_sets(c, 1))


def test_many_requests_ragged_and_subset():
    """More requests than one launch takes, most of them short, a few long; then a subset."""
    sfi = _sfi()
    rng = np.random.default_rng(8)
    lens = [int(x) for x in rng.integers(1, 40, 700)]
    lens[3], lens[600] = 2500, 1300
    c = Cache(9, lens, 1, 64)
    shape, q, out, lse, _, ws, st = _dense(c, 2, 1)
    assert st.item() == 0
    _check_attention(c, q, out, lse, 1, 2, 0.125, _dense_sets(c, 1))
    o2, l2 = torch.full_like(out, SENTINEL), torch.full_like(lse, SENTINEL)
    ids = [600, 5, 3]
    sfi.sfi_kv4_dense_attn(shape, c.kv, 4, 32, q, o2, lse=l2, workspace=ws, req_ids=dev_i32(ids))
    _check_attention(c, q, o2, l2, 1, 2, 0.125, _dense_sets(c, 1), rows=ids)
    rest = [r for r in range(700) if r not in ids]
    assert (o2[rest] == SENTINEL).all() and (l2[rest] == SENTINEL).all()


def test_a_run_repeats_to_the_bit():
    c = Cache(12, [9000, 100, 3000], 2, 128)
    a, b = _dense(c, 4, 2, scores=True), _dense(c, 4, 2, scores=True)
    for x, y in zip(a[2:5], b[2:5]):
        assert torch.equal(x, y)


def test_graph_replays_on_new_inputs_and_a_side_stream():
    sfi = _sfi()
    c = Cache(13, [700, 50], 2, 64)
    shape, q, out, lse, _, ws, _ = _dense(c, 2, 1)
    graph = torch.cuda.CUDAGraph()
    o2 = torch.empty_like(out)
    with torch.cuda.graph(graph):
        sfi.sfi_kv4_dense_attn(shape, c.kv, 4, 32, q, o2, workspace=ws)
    q.mul_(-0.5)
    c.lens = [333, 17]
    c.kv.seq_lens.copy_(dev_i32(c.lens))
    graph.replay()
    graph.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    sfi.sfi_kv4_dense_attn(shape, c.kv, 4, 32, q, out, lse=lse, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(out, o2)
    _check_attention(c, q, out, lse, 1, 2, 0.125, _dense_sets(c, 1))


def test_nan_of_the_newest_token_reaches_only_the_rows_that_see_it():
    """K and V of the last position hold NaN: with T tokens only the last token's rows are NaN."""
    T, G = 4, 2
    c = Cache(14, [300, 4], 2, 128)
    sk, sv = (o[2] for o in ref.offsets(128))
    for which in (0, 1):
        for r, L in enumerate(c.lens):
            blk = c.pool[c.table[r, (L - 1) // 16]]
            blk[:, (sk, sv)[which][(L - 1) % 16, 16 * 3]] = 127
        c.upload()
        _, q, out, lse, _, _, _ = _dense(c, G, T)
        o = out.view(2, T, -1, 128)
        if which == 0:
            assert torch.isnan(o[:, T - 1]).all() and torch.isnan(lse[:, T - 1]).all()
        else:  # group 3 of V alone
            assert torch.isnan(o[:, T - 1, :, 48:64]).all()
        assert torch.isfinite(o[:, :T - 1]).all() and torch.isfinite(lse[:, :T - 1]).all()
        sets = _dense_sets(c, T)
        qn, on = q.double().cpu().numpy(), out.double().cpu().numpy()
        for r in range(2):
            for h in range(c.hkv):
                for t in range(T - 1):
                    k, v, seen = sets(r, h, t)
                    hs = slice(h * G, (h + 1) * G)
                    w, _, _, bound, _, _ = ref.attend(qn[r, t, hs], np.nan_to_num(k), np.nan_to_num(v), seen,
                                                      1 / math.sqrt(128))
                    assert (np.abs(on[r, t, hs] - w) <= bound).all()
        for r, L in enumerate(c.lens):
            blk = c.pool[c.table[r, (L - 1) // 16]]
            blk[:, (sk, sv)[which][(L - 1) % 16, 16 * 3]] = 40


# ---- compaction and the sparse state ----------------------------------------------------------------------------

def _selection(rng, lens, hkv, sink, recent, T, k_cap, counts):
    idx = np.zeros((len(lens), hkv, max(1, k_cap)), np.int32)
    for r, L in enumerate(lens):
        hi = max(sink, L - T - recent)
        for h in range(hkv):
            idx[r, h, :counts[r]] = np.sort(rng.choice(np.arange(sink, hi), counts[r], replace=False)) if counts[r] else []
    return idx


def _fast_sets(c, T, sink, recent, idx, counts):
    def sets(r, h, t):
        k, v = c.rows(r)
        Lt = c.lens[r] - T + 1 + t
        at = np.concatenate([np.arange(min(sink, Lt)), idx[r, h, :counts[r]],
                             np.arange(max(sink, Lt - recent), Lt)]).astype(int)
        return k[h][at], v[h][at], np.ones(len(at), bool)
    return sets


@pytest.mark.parametrize("d,hkv,G,T,sink,recent,lens,counts", [
    (128, 8, 2, 1, 64, 256, [2000, 322, 500], [700, 1, 33]),
    (128, 2, 4, 4, 4, 32, [300, 100, 42, 8, 5], [200, 60, 2, 0, 0]),
    (64, 2, 4, 1, 0, 100, [150, 101, 3], [16, 0, 0]),
    (64, 1, 8, 2, 17, 1, [400, 21, 19], [15, 1, 0]),
    (128, 1, 1, 16, 5, 7, [64, 44], [30, 16]),
    (64, 3, 2, 1, 0, 0, [50, 40, 9], [20, 0, 5]),
    (128, 1, 4, 2, 3, 300, [3, 200, 2], [0, 0, 0]),
])
def test_compaction_and_fast_attention(d, hkv, G, T, sink, recent, lens, counts):
    sfi = _sfi()
    rng = np.random.default_rng(sum(lens))
    c = Cache(21, lens, hkv, d, 0.5, 4.0)
    B, k_cap = len(lens), max(counts)
    idx = _selection(rng, lens, hkv, sink, recent, T, k_cap, counts)
    shape = sfi.AttnShape(hkv * G, hkv, d)
    comp = sfi.alloc_kv4_compact(shape, [sink + n for n in counts])
    comp.pool.fill_(0x5A)
    comp.count = dev_i32(counts)
    st = _status()
    sfi.sfi_kv4_compact_gather(shape, c.kv, dev_i32(idx), comp.count, sink, comp, dev_status=st)
    got, off, cap = comp.pool.cpu().numpy(), comp.page_offset.tolist(), comp.capacity.tolist()
    want = np.full_like(got, 0x5A)
    for r, L in enumerate(lens):
        for h in range(hkv):
            pos = list(range(min(sink, L))) + list(idx[r, h, :counts[r]])
            for i in range(-(-len(pos) // 16)):
                blk = np.zeros(18 * d, np.uint8)
                for row, p in enumerate(pos[16 * i:16 * i + 16]):
                    src = c.pool[c.table[r, p // 16], h]
                    for which, (byte, shift, at) in enumerate(ref.offsets(d)):
                        ref.write_rows(blk, which, [row], (src[byte[p % 16]] >> shift[p % 16] & 15)[None],
                                       src[at[p % 16, ::16]][None])
                want[off[r] + h * cap[r] + i] = blk
    assert np.array_equal(got, want) and st.item() == 0
    q = torch.randn(B, T, hkv * G, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    out, lse = torch.full((B, T, hkv * G, d), SENTINEL, device="cuda"), torch.full((B, T, hkv * G), SENTINEL, device="cuda")
    sfi.sfi_kv4_fast_attn(shape, c.kv, comp, sink, recent, q, out, lse=lse, dev_status=st,
                          workspace=sfi.alloc_kv4_workspace(shape, B, T))
    assert st.item() == 0
    _check_attention(c, q, out, lse, T, G, 1 / math.sqrt(d), _fast_sets(c, T, sink, recent, idx, counts))


def test_a_full_selection_equals_dense():
    """Sink, every candidate and the recent window: the fast step is the dense one."""
    sfi = _sfi()
    c = Cache(23, [333], 2, 128)
    shape, q, out, lse, _, ws, _ = _dense(c, 2, 1)
    idx = np.broadcast_to(np.arange(4, 301, dtype=np.int32), (1, 2, 297))
    comp = sfi.alloc_kv4_compact(shape, [301])
    comp.count = dev_i32([297])
    sfi.sfi_kv4_compact_gather(shape, c.kv, dev_i32(idx), comp.count, 4, comp)
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    sfi.sfi_kv4_fast_attn(shape, c.kv, comp, 4, 32, q, o2, lse=l2, workspace=ws)
    assert torch.allclose(out, o2, rtol=0, atol=2e-5 * float(out.abs().max()))
    assert torch.allclose(lse, l2, rtol=0, atol=1e-5)


def test_selector_and_both_steps_together():
    """One cycle as it is used: append, slow step with scores, Selector, compaction, append, fast
    step; the selection is the Selector's on the scores the 4-bit slow step wrote."""
    sfi = _sfi()
    hkv, G, d, sink, recent, k = 2, 4, 128, 4, 32, 64
    lens = [500, 261]
    c = Cache(31, lens, hkv, d)
    shape = sfi.AttnShape(hkv * G, hkv, d)
    ws, st = sfi.alloc_kv4_workspace(shape, 2), _status()
    new = lambda s: _bf16(np.random.default_rng(s).standard_normal((2, 1, hkv, d))).cuda()  # noqa: E731
    q = _bf16(np.random.default_rng(40).standard_normal((2, 1, hkv * G, d))).cuda()
    out, lse = torch.empty(2, 1, hkv * G, d, device="cuda"), torch.empty(2, 1, hkv * G, device="cuda")
    scores = torch.full((2, hkv, 512), SENTINEL, device="cuda")
    sfi.sfi_kv4_append(shape, c.kv, new(1), new(2), dev_status=st)
    sfi.sfi_kv4_dense_attn(shape, c.kv, sink, recent, q, out, lse=lse, scores=scores, workspace=ws, dev_status=st)
    comp = sfi.alloc_kv4_compact(shape, [sink + k] * 2)
    idx = torch.zeros(2, hkv, k, dtype=torch.int32, device="cuda")
    sfi.sfi_select_topk(scores, hkv, c.kv.seq_lens, sink, recent, dev_i32([k, k]), idx, comp.count, dev_status=st)
    sfi.sfi_kv4_compact_gather(shape, c.kv, idx, comp.count, sink, comp, dev_status=st)
    c.pool = c.d_pool.cpu().numpy()
    _check_attention(c, q, out, lse, 1, G, 1 / math.sqrt(d), _dense_sets(c, 1), scores, sink, recent)
    c.lens = [n + 1 for n in lens]
    c.kv.seq_lens.copy_(dev_i32(c.lens))
    sfi.sfi_kv4_append(shape, c.kv, new(3), new(4), dev_status=st)
    sfi.sfi_kv4_fast_attn(shape, c.kv, comp, sink, recent, q, out, lse=lse, workspace=ws, dev_status=st)
    c.pool = c.d_pool.cpu().numpy()
    assert st.item() == 0 and comp.count.tolist() == [k, k]
    _check_attention(c, q, out, lse, 1, G, 1 / math.sqrt(d),
                     _fast_sets(c, 1, sink, recent, idx.cpu().numpy(), [k, k]))


def test_a_decode_step_from_the_projection_to_the_output_as_one_graph():
    """Head norm and rotation of a fused projection, the 4-bit append of its K and V, and the slow
    step over them: captured once and replayed on new inputs and lengths, against the same calls
    and against the formulas."""
    sfi = _sfi()
    hkv, G, d, sink, recent = 2, 4, 128, 4, 32
    hq = hkv * G
    c = Cache(61, [500, 37], hkv, d)
    shape, ws, st = sfi.AttnShape(hq, hkv, d), None, _status()
    ws = sfi.alloc_kv4_workspace(shape, 2)
    inv = [float(1e6 ** (-i / 64)) for i in range(64)]
    rope = sfi.Rope(sfi.rope_turns(inv))
    g = torch.Generator().manual_seed(4)
    rand = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    x, qw, kw = rand(2, 1, (hq + 2 * hkv) * d), rand(d), rand(d)
    q, k, v = (t.unflatten(-1, (-1, d)) for t in x.split([hq * d, hkv * d, hkv * d], -1))
    qn, kn = torch.empty(2, 1, hq, d, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 1, hkv, d, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty(2, 1, hq, d, device="cuda"), torch.empty(2, 1, hq, device="cuda")
    scores = torch.full((2, hkv, 505), SENTINEL, device="cuda")

    def step():
        sfi.sfi_qk_norm_rope(shape, rope, q, k, v, qn, q_weight=qw, k_weight=kw, seq_lens=c.kv.seq_lens, k_out=kn,
                             dev_status=st)
        sfi.sfi_kv4_append(shape, c.kv, kn, v, dev_status=st)
        sfi.sfi_kv4_dense_attn(shape, c.kv, sink, recent, qn, out, lse=lse, scores=scores, workspace=ws, dev_status=st)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in (1, 2):
        c.lens = [500 + n, 37 + n]
        if c.lens[0] > 16 * c.table.shape[1]:
            break
        c.kv.seq_lens.copy_(dev_i32(c.lens))
        x.copy_(rand(2, 1, (hq + 2 * hkv) * d))
        graph.replay()
        torch.cuda.synchronize()
        c.pool = c.d_pool.cpu().numpy()
        _check_attention(c, qn, out, lse, 1, G, 1 / math.sqrt(d), _dense_sets(c, 1), scores, sink, recent)
        for r, L in enumerate(c.lens):
            # what the cache holds for the newest token is the quantised rotated key
            key = kn[r, 0].double().cpu().numpy()
            want = ref.values(*ref.quantise(key, 1.0), 1.0)
            assert np.array_equal(c.rows(r)[0][:, L - 1], want)
            t = k[r, 0].double().cpu().numpy()
            t = t / np.sqrt((t * t).mean(-1, keepdims=True) + 1e-6) * kw.double().cpu().numpy()
            a = (L - 1) * np.array(inv)
            y = np.concatenate([t[:, :64] * np.cos(a) - t[:, 64:] * np.sin(a), t[:, 64:] * np.cos(a) + t[:, :64] * np.sin(a)], 1)
            r2 = np.tile(np.hypot(t[:, :64], t[:, 64:]), (1, 2))
            assert (np.abs(key - y) <= 2.0 ** -8 * np.abs(y) + 2.0 ** -17 * r2).all()
        eager = out.clone()
        step()
        assert torch.equal(out, eager)
    assert st.item() == 0


# ---- refusals ---------------------------------------------------------------------------------------------------

def test_bad_requests_are_left_out_whole():
    """A page id out of range anywhere in a request's row drops that request (scores included);
    lengths that are too short or beyond the table drop theirs; the others are complete."""
    from sparse_kv_long_sfi_gb300 import _abi
    c = Cache(50, [3000, 200, 40, 100], 2, 64)
    c.table[1, 12] = c.pool.shape[0]
    c.table[2, 0] = -5
    c.upload()
    _, q, out, lse, sc, _, st = _dense(c, 2, 2, scores=True)
    assert st.item() == _abi.SFI_DEV_BAD_PAGE
    for x in (out, lse, sc):
        assert (x[1:3] == SENTINEL).all()
    _check_attention(c, q, out, lse, 2, 2, 0.125, _dense_sets(c, 2), sc, 4, 32, rows=[0, 3])
    c.table[1, 12], c.table[2, 0] = 0, 0
    c.upload()
    real, c.lens = c.lens, [3000, 1, c.table.shape[1] * 16 + 1, 0]
    c.kv.seq_lens.copy_(dev_i32(c.lens))
    c.lens = real
    _, q, out, lse, sc, _, st = _dense(c, 2, 2, scores=True)
    assert st.item() == _abi.SFI_DEV_BAD_LEN
    for x in (out, lse, sc):
        assert (x[1:] == SENTINEL).all()
    _check_attention(c, q, out, lse, 2, 2, 0.125, _dense_sets(c, 2), sc, 4, 32, rows=[0])


def test_copy_errors_skip_what_they_concern():
    from sparse_kv_long_sfi_gb300 import _abi
    sfi = _sfi()
    c = Cache(51, [40, 40, 5, 40], 1, 64)
    c.table[1, 1] = 1000
    c.upload()
    shape, st = sfi.AttnShape(1, 1, 64), _status()
    x = _bf16(np.random.default_rng(0).standard_normal((4, 30, 1, 64))).cuda()
    sfi.sfi_kv4_append(shape, c.kv, x, x, new_lens=dev_i32([-1, 30, 9, 31]), dev_status=st)
    assert st.item() == _abi.SFI_DEV_BAD_LEN | _abi.SFI_DEV_BAD_PAGE
    got = c.d_pool.cpu().numpy()
    for r in (0, 2, 3):
        p = c.table[r, :-(-c.lens[r] // 16)]
        assert np.array_equal(got[p], c.pool[p])
    assert not np.array_equal(got[c.table[1, 0]], c.pool[c.table[1, 0]])  # the rows on good pages are written
    st.zero_()
    o = torch.full((4, 50, 1, 64), 777.0, dtype=torch.bfloat16, device="cuda")
    sfi.sfi_kv4_read(shape, c.kv, o, o.clone(), first=dev_i32([-1, 0, 5, 60]), dev_status=st)
    assert st.item() == _abi.SFI_DEV_BAD_LEN | _abi.SFI_DEV_BAD_PAGE
    assert (o[[0, 2, 3]] == 777.0).all() and (o[1, 16:32] == 777.0).all() and (o[1, 32:40] != 777.0).any()
    # compaction and the sparse state
    c = Cache(52, [200, 200, 200, 7, 200], 1, 64)  # request 3 is shorter than the sink
    comp = sfi.alloc_kv4_compact(shape, [40] * 5)
    idx = np.tile(np.arange(8, 40, dtype=np.int32), (5, 1, 1))
    idx[2, 0, 3] = 200
    count = dev_i32([33, 32, 32, 1, 32])
    comp.count = count
    comp.page_offset[4] = 99
    comp.pool.fill_(1)
    st.zero_()
    sfi.sfi_kv4_compact_gather(shape, c.kv, dev_i32(idx), count, 8, comp, dev_status=st)
    assert st.item() == _abi.SFI_DEV_K_OVERFLOW | _abi.SFI_DEV_BAD_INDEX | _abi.SFI_DEV_BAD_COMPACT
    assert (comp.pool[:3] == 1).all() and (comp.pool[9:] == 1).all()
    st.zero_()
    q = _bf16(np.random.default_rng(1).standard_normal((5, 1, 1, 64))).cuda()
    out = torch.full((5, 1, 1, 64), SENTINEL, device="cuda")
    comp.count[0] = 41
    sfi.sfi_kv4_fast_attn(shape, c.kv, comp, 8, 32, q, out, dev_status=st, workspace=sfi.alloc_kv4_workspace(shape, 5))
    assert st.item() == _abi.SFI_DEV_K_OVERFLOW | _abi.SFI_DEV_BAD_COMPACT
    assert (out[[0, 3, 4]] == SENTINEL).all() and (out[1:3] != SENTINEL).all()


def test_binding_refusals():
    sfi = _sfi()
    c = Cache(60, [20], 2, 64)
    shape = sfi.AttnShape(4, 2, 64)
    q, out = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 1, 4, 64, device="cuda")
    ws = sfi.alloc_kv4_workspace(shape, 1)
    with pytest.raises(sfi.SFIError):
        sfi.sfi_kv4_dense_attn(shape, c.kv, 0, 0, q, out, workspace=ws[:-256])
    with pytest.raises(sfi.SFIError):
        sfi.sfi_kv4_dense_attn(shape, c.kv, 0, 0, q, out)
    with pytest.raises(ValueError):
        sfi.sfi_kv4_dense_attn(shape, c.kv, 0, 0, q[..., :32], out, workspace=ws)
    with pytest.raises(ValueError):
        sfi.sfi_kv4_dense_attn(sfi.AttnShape(4, 2, 128), c.kv, 0, 0, q, out, workspace=ws)
    c.kv.k_scale = 3.0
    with pytest.raises(sfi.SFIError):
        sfi.sfi_kv4_dense_attn(shape, c.kv, 0, 0, q, out, workspace=ws)
