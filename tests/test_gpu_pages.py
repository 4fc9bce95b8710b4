"""The page operators against a model on the host: random histories of forks, reservations,
frees and compactions (tables, lengths, holder counts and every byte of the pools equal
after each step), their refusals, and the attention over a forked cache."""
import numpy as np
import pytest
import torch

from tests.gpu_harness import dev_i32

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


def _pages(n):
    return -(-n // 16)


class Model:
    """The operators' rules on host arrays."""

    def __init__(self, reqs, maxp, pages, pools, page_bytes, seed):
        rng = np.random.default_rng(seed)
        self.table = rng.integers(0, pages, (reqs, maxp)).astype(np.int32)
        self.lens = np.zeros(reqs, np.int32)
        self.ref = np.zeros(pages, np.int32)
        self.pools = [rng.integers(0, 256, (pages, page_bytes)).astype(np.uint8) for _ in range(pools)]

    def fork(self, src, dst, lens=None):
        for i, (a, z) in enumerate(zip(src, dst)):
            n = int(self.lens[a]) if lens is None else int(lens[i])
            held = self.table[a, :_pages(n)].copy()
            self.table[z, :len(held)] = held
            np.add.at(self.ref, held, 1)
            self.lens[z] = n

    def free(self, reqs):
        for r in reqs:
            np.subtract.at(self.ref, self.table[r, :_pages(self.lens[r])], 1)
            self.lens[r] = 0

    def reserve(self, new, reqs):
        free = list(np.flatnonzero(self.ref == 0))
        ref0 = self.ref.copy()
        need, seen = [], {}
        for r, n in zip(reqs, new):
            copy = False
            if n > self.lens[r] and self.lens[r] % 16:
                last = int(self.table[r, self.lens[r] // 16])
                copy = ref0[last] - seen.get(last, 0) > 1
                seen[last] = seen.get(last, 0) + 1
            need.append((copy, _pages(n) - _pages(self.lens[r]) + copy))
        if sum(k for _, k in need) > len(free):
            return False
        for (copy, k), r, n in zip(need, reqs, new):
            ids, at = [free.pop(0) for _ in range(k)], _pages(n) - k
            if copy:
                last = self.table[r, at]
                self.ref[last] -= 1
                for p in self.pools:
                    p[ids[0]] = p[last]
            self.table[r, at:at + k] = ids
            self.ref[ids] = 1
            self.lens[r] = n
        return True

    def compact(self):
        live = int((self.ref > 0).sum())
        movers = [i for i in range(live, len(self.ref)) if self.ref[i] > 0]
        holes = [i for i in range(live) if self.ref[i] <= 0]
        for a, z in zip(movers, holes):
            for p in self.pools:
                p[z] = p[a]
            self.ref[z], self.ref[a] = self.ref[a], 0
            for r in range(len(self.lens)):
                row = self.table[r, :_pages(self.lens[r])]
                row[row == a] = z
        return live


class Device:
    def __init__(self, m):
        sfi = _sfi()
        self.pools = [torch.from_numpy(p.copy()).cuda() for p in m.pools]
        self.map = sfi.PageMap(dev_i32(m.table), dev_i32(m.lens), dev_i32(m.ref))
        self.pp = sfi.PagePools(self.pools)
        self.ws = sfi.alloc_page_workspace(self.map)
        self.ws.fill_(0xA5)  # no initial contents are needed
        self.st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def same(self, m, what):
        assert np.array_equal(self.map.page_table.cpu().numpy(), m.table), what
        assert np.array_equal(self.map.seq_lens.cpu().numpy(), m.lens), what
        assert np.array_equal(self.map.ref_count.cpu().numpy(), m.ref), what
        for i, (a, b) in enumerate(zip(self.pools, m.pools)):
            assert np.array_equal(a.cpu().numpy(), b), (what, "pool", i)


@pytest.mark.parametrize("reqs,maxp,pages,pools,page_bytes,seed", [
    (6, 4, 30, 1, 16, 0),
    (40, 9, 150, 3, 4608, 1),
    (200, 20, 1500, 2, 8208, 2),   # a page of one 8 KB chunk and 16 bytes
    (1030, 3, 5000, 1, 32, 3),
])
def test_random_histories(reqs, maxp, pages, pools, page_bytes, seed):
    sfi = _sfi()
    rng = np.random.default_rng(100 + seed)
    m = Model(reqs, maxp, pages, pools, page_bytes, seed)
    d = Device(m)
    refused = 0
    for step in range(40):
        op = rng.choice(["reserve", "reserve", "fork", "free", "compact"])
        if op == "reserve":
            n = int(rng.integers(1, min(reqs, 1024) + 1))
            ids = rng.permutation(reqs)[:n].astype(np.int32)
            if rng.random() < 0.2:
                n = min(reqs, 1024)
                ids = np.arange(n, dtype=np.int32)
            new = np.minimum(m.lens[ids] + rng.integers(0, 40, n) * (rng.random(n) < 0.7), maxp * 16).astype(np.int32)
            d.st.zero_()
            given = None if np.array_equal(ids, np.arange(n)) and rng.random() < 0.5 else dev_i32(ids)
            sfi.sfi_page_reserve(d.map, d.pp, dev_i32(new), given, workspace=d.ws, dev_status=d.st)
            ok = m.reserve(new, ids)
            refused += not ok
            assert d.st.item() == (0 if ok else 64)
        elif op == "fork":
            empty, full = np.flatnonzero(m.lens == 0), np.flatnonzero(m.lens > 0)
            if not len(empty) or not len(full):
                continue
            k = int(rng.integers(1, len(empty) + 1))
            src, dst = rng.choice(full, k), rng.permutation(empty)[:k]
            lens = rng.integers(0, m.lens[src] + 1) if rng.random() < 0.5 else None
            sfi.sfi_page_fork(d.map, dev_i32(src), dev_i32(dst), None if lens is None else dev_i32(lens), dev_status=d.st)
            m.fork(src, dst, lens)
        elif op == "free":
            ids = rng.permutation(reqs)[:int(rng.integers(1, reqs // 2 + 1))]
            sfi.sfi_page_free(d.map, dev_i32(np.concatenate([ids, ids[:1]])), dev_status=d.st)  # the first one twice
            m.free(ids)
        else:
            table, ref = torch.empty_like(d.map.page_table), torch.empty_like(d.map.ref_count)
            live = torch.empty(1, dtype=torch.int32, device="cuda")
            sfi.sfi_page_compact(d.map, d.pp, table, ref, live, workspace=d.ws, dev_status=d.st)
            assert np.array_equal(d.map.page_table.cpu().numpy(), m.table), "the old table stays as it was"
            assert live.item() == m.compact()
            d.map = sfi.PageMap(table, d.map.seq_lens, ref)
        d.same(m, (step, op))
    assert d.st.item() in (0, 64)
    assert refused < 40


def test_copy_on_write_order_and_last_holder():
    """Three holders of one part-filled page and nobody else: the first two in the list copy it
    (lowest free pages first), the last keeps it; a holder outside the list makes all copy."""
    sfi = _sfi()
    m = Model(5, 3, 12, 2, 64, 7)
    m.table[0, :2] = [9, 4]
    m.ref[[9, 4]] = 1
    m.lens[0] = 20
    m.fork([0, 0], [2, 3])
    d = Device(m)
    sfi.sfi_page_reserve(d.map, d.pp, dev_i32([21, 48, 30]), dev_i32([3, 0, 2]), workspace=d.ws, dev_status=d.st)
    assert m.reserve([21, 48, 30], [3, 0, 2])
    d.same(m, "copy on write")
    assert m.table[2, 1] == 4 and m.ref[4] == 1 and m.table[3, 1] == 0 and list(m.table[0, 1:3]) == [1, 2]
    m = Model(5, 3, 12, 2, 64, 8)
    m.table[0, :2] = [9, 4]
    m.ref[[9, 4]] = 1
    m.lens[0] = 20
    m.fork([0, 0, 0], [2, 3, 4])
    d = Device(m)
    sfi.sfi_page_reserve(d.map, d.pp, dev_i32([21, 21, 21, 20]), dev_i32([3, 0, 2, 4]), workspace=d.ws, dev_status=d.st)
    assert m.reserve([21, 21, 21, 20], [3, 0, 2, 4])  # request 4 does not grow: it goes on holding the page
    d.same(m, "a holder that does not grow")
    assert list(m.table[[3, 0, 2, 4], 1]) == [0, 1, 2, 4] and m.ref[4] == 1


def test_copy_pages():
    sfi = _sfi()
    for page_bytes in (16, 4608, 32768 + 16):
        m = Model(1, 1, 40, 3, page_bytes, 1)
        d = Device(m)
        src, dst = [3, 3, 7, 39], [0, 20, 21, 38]
        sfi.sfi_page_copy(d.pp, dev_i32(src), dev_i32(dst), dev_status=d.st)
        for p in m.pools:
            p[dst] = p[src]
        d.same(m, page_bytes)
        assert d.st.item() == 0
        sfi.sfi_page_copy(d.pp, dev_i32([-1, 40, 2, 5]), dev_i32([1, 4, 40, 6]), dev_status=d.st)
        for p in m.pools:
            p[6] = p[5]
        d.same(m, "bad ids are skipped")
        assert d.st.item() == 1


def test_refusals_change_nothing():
    from sparse_kv_long_sfi_gb300 import _abi
    sfi = _sfi()
    m = Model(6, 3, 12, 1, 16, 3)
    assert m.reserve([20, 16, 40], [0, 1, 2])
    m.lens[5] = 49                       # beyond the table: only device data can say so
    m.fork([0], [3])
    d = Device(m)

    def reserve(new, reqs, expect, pools=d.pp):
        d.st.zero_()
        sfi.sfi_page_reserve(d.map, pools, dev_i32(new), dev_i32(reqs), workspace=d.ws, dev_status=d.st)
        assert d.st.item() == expect
        d.same(m, (new, reqs))

    reserve([30, 17], [1, 6], _abi.SFI_DEV_BAD_INDEX)
    reserve([30, 17], [-1, 1], _abi.SFI_DEV_BAD_INDEX)
    reserve([30, 30], [1, 1], _abi.SFI_DEV_BAD_INDEX)       # the same request twice
    reserve([15], [1], _abi.SFI_DEV_BAD_LEN)                # shorter than it is
    reserve([49], [1], _abi.SFI_DEV_BAD_LEN)                # beyond the table
    reserve([21], [0], _abi.SFI_DEV_BAD_PAGE, pools=None)   # a shared page, and nowhere to copy it
    reserve([48, 48, 48, 48], [0, 1, 3, 4], _abi.SFI_DEV_NO_PAGE)
    d.map.page_table[0, 1] = 99
    m.table[0, 1] = 99
    reserve([21], [0], _abi.SFI_DEV_BAD_PAGE)
    for src, dst, expect in (([0], [4], 1), ([2], [2], 8), ([7], [4], 8), ([2], [-1], 8), ([5], [4], 2)):
        d.st.zero_()
        sfi.sfi_page_fork(d.map, dev_i32(src), dev_i32(dst), dev_status=d.st)
        assert d.st.item() == expect
        d.same(m, (src, dst))
    for lens, expect in (([41], 2), ([-1], 2)):
        d.st.zero_()
        sfi.sfi_page_fork(d.map, dev_i32([2]), dev_i32([4]), dev_i32(lens), dev_status=d.st)
        assert d.st.item() == expect
        d.same(m, lens)
    for reqs, expect in (([5], 2), ([9], 8)):
        d.st.zero_()
        sfi.sfi_page_free(d.map, dev_i32(reqs), dev_status=d.st)
        assert d.st.item() == expect
        d.same(m, reqs)
    # a bad id and a page without holders: the rest of the request is let go
    d.st.zero_()
    d.map.ref_count[int(m.table[2, 1])] = 0
    sfi.sfi_page_free(d.map, dev_i32([0, 2]), dev_status=d.st)
    assert d.st.item() == 1
    m.ref[m.table[0, 0]] -= 1
    m.ref[m.table[2, [0, 2]]] -= 1
    m.ref[m.table[2, 1]] = 0
    m.lens[[0, 2]] = 0
    d.same(m, "partial free")


def test_branches_read_what_they_share_and_write_their_own():
    """A request forks twice, the branches append different tokens to their 4-bit cache and attend:
    each sees the common prefix and its own token; then a compaction changes nothing they see."""
    sfi = _sfi()
    hkv, d, L = 2, 64, 37
    shape = sfi.AttnShape(4, hkv, d)
    pool = sfi.alloc_kv4_pool(shape, 30)
    table = torch.zeros(4, 4, dtype=torch.int32, device="cuda")
    lens, ref = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (4, 30))
    ref[[0, 1, 2, 5]] = 1  # pages of someone else, not in this table
    pm = sfi.PageMap(table, lens, ref)
    pp, ws = sfi.PagePools([pool]), sfi.alloc_page_workspace(pm)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    kv = sfi.PagedKV4(pool, table, lens)
    prompt = rand(4, L, hkv, d), rand(4, L, hkv, d)
    sfi.sfi_page_reserve(pm, pp, dev_i32([L]), dev_i32([1]), workspace=ws, dev_status=st)
    sfi.sfi_kv4_append(shape, kv, *prompt, new_lens=dev_i32([0, L, 0, 0]), req_ids=dev_i32([1]), dev_status=st)
    sfi.sfi_page_fork(pm, dev_i32([1, 1]), dev_i32([0, 3]), dev_status=st)
    sfi.sfi_page_reserve(pm, pp, dev_i32([L + 1] * 3), dev_i32([0, 1, 3]), workspace=ws, dev_status=st)
    own = rand(4, 1, hkv, d), rand(4, 1, hkv, d)
    sfi.sfi_kv4_append(shape, kv, *own, req_ids=dev_i32([0, 1, 3]), dev_status=st)
    assert (table[[0, 1, 3], :2] == table[1, :2]).all() and len(set(table[[0, 1, 3], 2].tolist())) == 3
    q = rand(4, 1, 4, d)
    ids, aws = dev_i32([0, 1, 3]), sfi.alloc_kv4_workspace(shape, 4)
    out = torch.empty(4, 1, 4, d, device="cuda")
    sfi.sfi_kv4_dense_attn(shape, kv, 0, 0, q, out, req_ids=ids, workspace=aws, dev_status=st)
    # the same three sequences, each written on its own
    solo_pool = sfi.alloc_kv4_pool(shape, 12)
    solo = sfi.PagedKV4(solo_pool, torch.arange(12, dtype=torch.int32, device="cuda").view(4, 3), dev_i32([L + 1] * 4))
    k, v = (torch.cat([p[1:2].expand(4, -1, -1, -1), o], 1).contiguous() for p, o in zip(prompt, own))
    sfi.sfi_kv4_append(shape, solo, k, v, dev_status=st)
    want = torch.empty_like(out)
    sfi.sfi_kv4_dense_attn(shape, solo, 0, 0, q, want, req_ids=ids, workspace=aws, dev_status=st)
    assert torch.equal(out[[0, 1, 3]], want[[0, 1, 3]])
    # compaction
    ref[[0, 2]] = 0
    t2, r2, live = torch.empty_like(table), torch.empty_like(ref), torch.empty(1, dtype=torch.int32, device="cuda")
    sfi.sfi_page_compact(pm, pp, t2, r2, live, workspace=ws, dev_status=st)
    assert live.item() == 7 and r2[:7].min().item() > 0 and r2[7:].max().item() == 0
    for tab in (table, t2):  # the old table goes on being valid
        kv.page_table = tab
        sfi.sfi_kv4_dense_attn(shape, kv, 0, 0, q, out.zero_(), req_ids=ids, workspace=aws, dev_status=st)
        assert torch.equal(out[[0, 1, 3]], want[[0, 1, 3]])
    assert st.item() == 0
