"""Window attention and attention weights where they can go wrong: NaN in hidden places, views, subsets of requests,
bad pages and lengths, guard bands, far pages, two streams, captured graphs."""
import numpy as np
import pytest
import torch

from tests import window_reference as ref
from tests.test_gpu_attn_mass import _expected

pytestmark = pytest.mark.gpu

PROMPT, STEP = 70, 2  # query tokens: the two kernels at G = 4
HEADS = (8, 2, 64)
WIDE = 1 << 20


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


class Call:
    """One problem, its two calls and the fp64 answer of single tokens."""

    def __init__(self, seed, lens, t, new=None, heads=HEADS, sink=3, recent=40, fill=None):
        self.c = ref.Cache(seed, lens, *heads, fill=fill)
        self.q = ref.queries(seed + 1, len(lens), t, heads[0], heads[2])
        self.new = [t] * len(lens) if new is None else new
        self.sink, self.recent = sink, recent

    def device(self):
        self.shape, self.kv = self.c.device()
        self.dq, self.dnew, self.st = self.q.cuda(), _i32(self.new), _i32([0])
        self.out = torch.full(self.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full(self.q.shape[:3], 7.0, device="cuda")
        self.mass = torch.full((len(self.new), self.c.hkv, max(self.c.lens)), 0.25, device="cuda")
        return self

    def attend(self, **kw):
        _sfi().sfi_window_attn(self.shape, self.kv, self.sink, self.recent, self.dq, self.out, lse=self.lse,
                               new_lens=self.dnew, dev_status=self.st, **kw)

    def weigh(self, **kw):
        _sfi().sfi_attn_mass(self.shape, self.kv, self.sink, self.recent, self.dq, self.lse, self.mass, decay=0.5,
                             new_lens=self.dnew, dev_status=self.st, **kw)

    def check(self, r, i, out=None, lse=None):
        out, lse = self.out if out is None else out, self.lse if lse is None else lse
        p = self.c.lens[r] - self.new[r] + i
        for h in range(self.c.hq):
            o, x, _, mag, smag = ref.token(self.c, r, h, self.q[r, i, h], p, self.sink, self.recent)
            err = np.abs(out[r, i, h].double().cpu().numpy() - o)
            assert (err <= ref.out_bound(o, mag, self.c.d)).all(), (r, i, h, err.max())
            assert abs(float(lse[r, i, h]) - x) <= ref.lse_bound(x, smag, self.c.d), (r, i, h)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("t,heads", [(PROMPT, HEADS), (3, HEADS), (PROMPT, (16, 8, 128)), (4, (16, 8, 128))])
def test_values_that_later_tokens_see(t, heads, bad):
    """A V row that is not finite, at the newest positions and behind the window: tokens that do not see it keep their
    rows, the others get what the arithmetic gives."""
    c = Call(31, [200, 150 + t], t, heads=heads)
    at = [c.c.lens[0] - 2, c.c.lens[1] - t - 40 - 5]  # seen by the last two tokens; by none
    for r, j in enumerate(at):
        c.c.v[c.c.table[r, j // 16], :, j % 16, 5] = bad
    c.device().attend()
    assert c.st.item() == 0
    for i in range(t - 2):
        c.check(0, i)
    assert (~torch.isfinite(c.out[0, t - 2:, :, 5])).all() and torch.isfinite(c.out[0, t - 2:, :, :5]).all()
    for i in range(0, t, 7):
        c.check(1, i)
    assert torch.isfinite(c.out[1]).all()


@pytest.mark.parametrize("t", [PROMPT, STEP])
def test_views_subsets_and_requests_without_tokens(t):
    """q as a view of a fused projection, out with 16-byte alignment only, requests by id, some with no new token."""
    c = Call(33, [90, 200, t, 130, 300], t, new=[t, 0, t, 1, t]).device()
    hq, hkv, d = HEADS
    fused = torch.full((5, t, hq + 2 * hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    fused[:, :, :hq] = c.dq
    c.dq = fused[:, :, :hq]
    room = torch.full((c.out.numel() + 8,), 7.0, dtype=torch.bfloat16, device="cuda")
    c.out = room[8:].view(c.q.shape)
    assert c.out.data_ptr() % 32 == 16
    c.attend(req_ids=_i32([4, 1, 0, 3]))
    assert c.st.item() == 0 and (c.out[2] == 7).all() and (c.lse[2] == 7).all() and (c.out[1] == 7).all()
    assert (c.out[3, 1:] == 7).all() and (room[:8] == 7).all()
    for r, i in ((0, 0), (0, t - 1), (3, 0), (4, 0), (4, t - 1)):
        c.check(r, i)
    before = c.mass.clone()
    c.weigh(req_ids=_i32([4, 3]))
    for r in (0, 1, 2):
        assert torch.equal(c.mass[r], before[r])
    want, bound = _expected(c.c, c.q, c.lse.cpu(), c.new, 3, 40, before.cpu(), 0.5)
    for r in (3, 4):
        n = c.c.lens[r]
        assert (np.abs(c.mass[r, :, :n].double().cpu().numpy() - want[r, :, :n]) <= bound[r, :, :n]).all()


@pytest.mark.parametrize("t", [PROMPT, STEP])
def test_refused_requests(t):
    """Lengths and request ids out of range: the request is skipped, the others are computed."""
    for lens, new, bit in (([90, t - 1], [t, t], 2), ([90, 400], [t, t], 2), ([90, 90], [t, t + 1], 2),
                           ([90, 90], [t, -1], 2), ([90, -5], [t, 0], 2)):
        c = Call(35, [90, 90], t).device()
        c.kv.seq_lens = _i32(lens)
        c.dnew = _i32(new)
        c.attend()
        assert c.st.item() == bit and (c.out[1] == 7).all() and (c.lse[1] == 7).all(), (lens, new)
        c.check(0, t - 1)
        c.st.zero_()
        c.lse[1] = 0
        before = c.mass.clone()
        c.weigh()
        assert c.st.item() == bit and torch.equal(c.mass[1], before[1]) and not torch.equal(c.mass[0], before[0])
    c = Call(35, [90, 90], t).device()
    for call in (c.attend, c.weigh):
        c.st.zero_()
        call(req_ids=_i32([0, 2]))
        assert c.st.item() == 8
    c.st.zero_()
    call(req_ids=_i32([-1]))
    assert c.st.item() == 8


@pytest.mark.parametrize("t", [PROMPT, STEP])
@pytest.mark.parametrize("page", [-1, 1 << 20])
def test_bad_pages(t, page):
    """An id out of range that the new tokens read: none of that block's rows is written."""
    c = Call(37, [120, 120], t, recent=WIDE)
    c.c.table[1, 2] = page
    c.device().attend()
    assert c.st.item() == 1 and (c.out[1] == 7).all() and (c.lse[1] == 7).all()
    c.check(0, 0)
    c.check(0, t - 1)
    c.st.zero_()
    c.lse[1] = 1.0
    c.weigh()
    assert c.st.item() == 1 and (c.mass[1] == 0.25).all() and not (c.mass[0] == 0.25).any()
    # hidden behind the window it is not read
    c.recent, c.sink = 5, 0
    c.st.zero_()
    c.attend()
    assert c.st.item() == 0 or t == PROMPT
    assert (c.out[1, -1] != 7).any()


@pytest.mark.parametrize("t", [1, 3, PROMPT, 130])
def test_guard_bands(t):
    """Nothing is written before, behind or between what the calls write."""
    c = Call(39, [300, 257], t, new=[t, max(1, t - 1)]).device()
    rooms = {}
    for name in ("out", "lse", "mass"):
        x = getattr(c, name)
        pad = 64
        room = torch.full((x.numel() + 2 * pad,), 7.0, dtype=x.dtype, device="cuda")
        view = room[pad:pad + x.numel()].view(x.shape)
        if name == "mass":
            view.fill_(0.25)
        rooms[name] = room
        setattr(c, name, view)
    pools = c.kv.k_pool.clone(), c.kv.v_pool.clone()
    c.attend()
    c.weigh()
    assert c.st.item() == 0
    for name, room in rooms.items():
        assert (room[:64] == 7).all() and (room[-64:] == 7).all(), name
    assert torch.equal(pools[0], c.kv.k_pool) and torch.equal(pools[1], c.kv.v_pool)
    assert (c.mass[1, :, 257:] == 0.25).all()


def test_pages_far_behind():
    """Pools past 2^32 bytes, the pages in use at their end."""
    c = Call(41, [150], PROMPT, heads=(16, 8, 128))
    far = 140000
    shape, kv = c.c.device()
    for name in ("k_pool", "v_pool"):
        big = torch.empty((far + c.c.pages, 8, 16, 128), dtype=torch.bfloat16, device="cuda")
        big[far:] = getattr(kv, name)
        setattr(kv, name, big)
    kv.page_table += far
    c.device()
    c.kv = kv
    c.attend()
    assert c.st.item() == 0
    for i in (0, 33, PROMPT - 1):
        c.check(0, i)
    before = c.mass.cpu().clone()
    c.weigh()
    want, bound = _expected(c.c, c.q, c.lse.cpu(), c.new, 3, 40, before, 0.5)
    assert (np.abs(c.mass.double().cpu().numpy() - want) <= bound).all()
    step = Call(43, [150], 1, heads=(16, 8, 128))
    step.c, step.q = c.c, c.q[:, -1:].contiguous()
    step.device()
    step.kv = kv
    step.attend()
    step.check(0, 0)
    # and an eviction there
    new, count, idx = _i32([0]), _i32([0]), torch.zeros(1, 8, 20, dtype=torch.int32, device="cuda")
    mass = torch.rand(1, 8, 150, device="cuda")
    _sfi().sfi_kv_evict(shape, kv, mass, 3, 40, _i32([20]), idx, count, new)
    kept, _ = ref.keep(mass[0, 5].double().tolist(), 150, 3, 40, 20)
    for i, j in enumerate(kept):
        assert torch.equal(kv.v_pool[far + int(c.c.table[0, i // 16]), 5, i % 16].cpu(), c.c.v[c.c.table[0, j // 16], 5, j % 16])


@pytest.mark.parametrize("t", [PROMPT, STEP])
def test_two_streams_and_repeated_calls(t):
    """Calls on two streams at once, and again: bit for bit what one call gives."""
    a, b = Call(45, [300] * 6, t).device(), Call(47, [333] * 6, t).device()
    a.attend(), a.weigh(), b.attend(), b.weigh()
    torch.cuda.synchronize()
    want = [x.clone() for x in (a.out, a.lse, a.mass, b.out, b.lse, b.mass)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for c in (a, b):
            c.out.fill_(7), c.lse.fill_(7), c.mass.fill_(0.25)
        torch.cuda.synchronize()
        for c, s in zip((a, b), streams):
            c.attend(stream=s)
            c.weigh(stream=s)
        torch.cuda.synchronize()
        for x, y in zip((a.out, a.lse, a.mass, b.out, b.lse, b.mass), want):
            assert torch.equal(x, y)


@pytest.mark.parametrize("t", [PROMPT, STEP])
def test_captured_and_replayed(t):
    """A captured run reads lengths, pages and queries of its replay."""
    c = Call(49, [300, 257], t).device()
    c.attend(), c.weigh()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.attend()
        c.weigh()
    c.c.lens = [290, 130]
    c.kv.seq_lens.copy_(_i32(c.c.lens))
    c.q = ref.queries(51, 2, t, HEADS[0], HEADS[2])
    c.dq.copy_(c.q)
    for _ in range(2):
        c.out.fill_(7), c.lse.fill_(7), c.mass.fill_(0.25)
        g.replay()
        torch.cuda.synchronize()
        assert c.st.item() == 0
        for r in range(2):
            c.check(r, 0)
            c.check(r, t - 1)
        want, bound = _expected(c.c, c.q, c.lse.cpu(), c.new, 3, 40, torch.full(c.mass.shape, 0.25), 0.5)
        for r in range(2):
            n = c.c.lens[r]
            assert (np.abs(c.mass[r, :, :n].double().cpu().numpy() - want[r, :, :n]) <= bound[r, :, :n]).all()


def test_many_small_items():
    """More blocks of query rows than the GPU has SMs, of one and two tiles, in turn on the same CTAs."""
    lens = [5 + 7 * i % 140 for i in range(300)]
    new = [min(n, 1 + 13 * i % 70) for i, n in enumerate(lens)]
    c = Call(53, lens, 70, new=new, heads=(2, 2, 64), sink=2, recent=30).device()
    c.attend()
    assert c.st.item() == 0
    for r in range(0, 300, 17):
        for i in (0, new[r] // 2, new[r] - 1):
            c.check(r, i)
        assert (c.out[r, new[r]:] == 7).all()
    g8 = Call(55, [n + 40 for n in lens], 40, new=[min(n, 40) for n in new], heads=(8, 1, 128), sink=0, recent=WIDE).device()
    g8.attend()
    for r in range(0, 300, 37):
        for i in (0, g8.new[r] - 1):
            g8.check(r, i)
