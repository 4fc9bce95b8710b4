"""The 4-bit fast step for few and for many (request, KV head) units. Few units take a cluster
of CTAs each; many units share the grid in runs, and so do few units of a compact pool that
is large: a pool with room to spare (`roomy`) brings a small call to the second way.
Inputs, reference and tolerances are those of test_gpu_kv4 (the merges' part of its bound,
64 2^-23, covers the at most 8 + 8 steps of a cluster's)."""
import math

import numpy as np
import pytest
import torch

from tests.gpu_harness import dev_i32, dev_i64
from tests.test_gpu_kv4 import SENTINEL, Cache, _check_attention, _fast_sets, _lib, _selection, _sfi, _status  # noqa: F401

pytestmark = pytest.mark.gpu


class Step:
    """Ragged requests, their selection compacted, and a fast step over them."""

    def __init__(self, seed, B, hkv, G, d, T, sink, recent, longest, ragged=False, roomy=False):
        sfi = _sfi()
        self.rng = rng = np.random.default_rng(seed)
        self.T, self.G, self.sink, self.recent = T, G, sink, recent
        lens = [int(x) for x in rng.integers(T, longest + 1, B)]
        lens[-1], lens[0] = T, 16000 if ragged else longest  # (in this order: one request has the longest)
        self.c = Cache(seed, lens, hkv, d, 0.5, 2.0)
        self.counts = [int(rng.integers(0, max(0, L - T - recent - sink) + 1)) for L in lens]
        if ragged:
            self.counts[0] = lens[0] - T - recent - sink
        self.idx = _selection(rng, lens, hkv, sink, recent, T, max(self.counts), self.counts)
        self.shape = sfi.AttnShape(hkv * G, hkv, d)
        self.comp = sfi.alloc_kv4_compact(self.shape, [sink + n + (32000 if roomy else 0) for n in self.counts])
        self.comp.count = dev_i32(self.counts)
        self.st = _status()
        sfi.sfi_kv4_compact_gather(self.shape, self.c.kv, dev_i32(self.idx), self.comp.count, sink, self.comp,
                                   dev_status=self.st)
        self.q = torch.randn(B, T, hkv * G, d, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()
        self.out = torch.full((B, T, hkv * G, d), SENTINEL, device="cuda")
        self.lse = torch.full((B, T, hkv * G), SENTINEL, device="cuda")
        self.ws = sfi.alloc_kv4_workspace(self.shape, B, T)

    def run(self, **kw):
        _sfi().sfi_kv4_fast_attn(self.shape, self.c.kv, self.comp, self.sink, self.recent, self.q, self.out, lse=self.lse,
                                 dev_status=self.st, workspace=self.ws, **kw)

    def check(self, rows=None):
        plain, cache = self.c.rows, {}

        def cached(r):
            if r not in cache:
                cache.clear()
                cache[r] = plain(r)
            return cache[r]
        self.c.rows = cached
        _check_attention(self.c, self.q, self.out, self.lse, self.T, self.G, 1 / math.sqrt(self.c.d),
                         _fast_sets(self.c, self.T, self.sink, self.recent, self.idx, self.counts), rows=rows)
        self.c.rows = plain


@pytest.mark.parametrize("B,hkv,G,d,T,sink,recent,longest", [
    (1, 1, 1, 128, 1, 4, 32, 2000),    # one unit of many blocks
    (1, 1, 8, 64, 2, 0, 0, 900),       # sixteen rows; no sink, no window
    (2, 3, 2, 128, 3, 7, 20, 260),     # six rows, three tokens
    (5, 2, 1, 64, 5, 3, 40, 300),
    (13, 4, 4, 128, 1, 16, 16, 150),   # 52 units: five or fewer CTAs each
    (9, 5, 2, 64, 8, 2, 9, 120),       # 45 units of sixteen rows
    (24, 4, 2, 128, 1, 1, 50, 100),    # 96 units
    (50, 4, 1, 64, 2, 4, 8, 90),       # 200 units
    (64, 8, 2, 128, 1, 4, 32, 70),     # 512 units
    (64, 4, 8, 64, 2, 4, 32, 70),      # 256 units of sixteen rows
])
def test_fast_attention_by_units(B, hkv, G, d, T, sink, recent, longest):
    s = Step(B * hkv + T, B, hkv, G, d, T, sink, recent, longest)
    s.run()
    assert s.st.item() == 0
    s.check(rows=None if B < 10 else sorted({0, 1, B // 2, B - 2, B - 1}))
    assert (s.out != SENTINEL).all() and (s.lse != SENTINEL).all()


@pytest.mark.parametrize("roomy", [False, True])
@pytest.mark.parametrize("B,hkv,G,d,T,sink,recent,longest", [
    (1, 1, 1, 128, 1, 4, 32, 2000),
    (2, 3, 2, 128, 3, 7, 20, 260),
    (3, 2, 4, 64, 4, 2, 9, 120),
])
def test_a_long_unit_among_short_ones(B, hkv, G, d, T, sink, recent, longest, roomy):
    s = Step(B * hkv + T, B, hkv, G, d, T, sink, recent, longest, True, roomy)
    s.run()
    assert s.st.item() == 0
    s.check()


@pytest.mark.parametrize("roomy", [False, True])
@pytest.mark.parametrize("B,hkv,G,d,T", [(6, 2, 2, 128, 1), (6, 1, 8, 64, 2), (6, 3, 1, 64, 1)])
def test_bad_requests_are_left_out_whole(B, hkv, G, d, T, roomy):
    """A page id out of range in the recent window, a count beyond the capacity, a compact offset
    beyond the pool and a length beyond the table: none of that request's rows is written."""
    from sparse_kv_long_sfi_gb300 import _abi
    s = Step(40 + hkv, B, hkv, G, d, T, 4, 100, 400, roomy=roomy)
    lens = s.c.lens
    bad = [r for r in range(1, B) if lens[r] > 40][:3]
    good = [r for r in range(B) if r not in bad]
    s.c.table[bad[0], (lens[bad[0]] - 1) // 16] = s.c.pool.shape[0]
    s.c.upload()
    s.run()
    assert s.st.item() == _abi.SFI_DEV_BAD_PAGE
    for x in (s.out, s.lse):
        assert (x[bad[0]] == SENTINEL).all()
    s.check(rows=[r for r in range(B) if r != bad[0]])
    # and the rest
    count, off = s.comp.count.clone(), s.comp.page_offset.clone()
    s.comp.count[bad[1]] = int(s.comp.capacity[bad[1]]) * 16 + 1
    s.comp.page_offset[bad[2]] = s.comp.pool.shape[0] - hkv * int(s.comp.capacity[bad[2]]) + 1
    s.st.zero_()
    s.out.fill_(SENTINEL)
    s.lse.fill_(SENTINEL)
    s.run()
    assert s.st.item() == _abi.SFI_DEV_BAD_PAGE | _abi.SFI_DEV_K_OVERFLOW | _abi.SFI_DEV_BAD_COMPACT
    for x in (s.out, s.lse):
        assert (x[bad] == SENTINEL).all()
    s.check(rows=good)
    # put right, all but a length
    s.comp.count, s.comp.page_offset = count, off
    s.c.table[bad[0], (lens[bad[0]] - 1) // 16] = 0
    s.c.kv.page_table.copy_(dev_i32(s.c.table))
    for wrong in (T - 1, s.c.table.shape[1] * 16 + 1):
        s.c.kv.seq_lens.copy_(dev_i32([wrong if r == bad[1] else n for r, n in enumerate(lens)]))
        s.st.zero_()
        s.out.fill_(SENTINEL)
        s.lse.fill_(SENTINEL)
        s.run()
        assert s.st.item() == _abi.SFI_DEV_BAD_LEN
        for x in (s.out, s.lse):
            assert (x[bad[1]] == SENTINEL).all() and (x[good] != SENTINEL).all()


@pytest.mark.parametrize("roomy", [False, True])
def test_subsets_repeats_and_graphs(roomy):
    """Requests out of order, rows of the others left as they are; a run repeats to the bit, eagerly and from a graph that is replayed on new inputs."""
    s = Step(77, 5, 2, 4, 128, 2, 4, 40, 330, roomy=roomy)
    ids = dev_i32([3, 0])
    s.run(req_ids=ids, batch=2)
    assert s.st.item() == 0
    for x in (s.out, s.lse):
        assert (x[[1, 2, 4]] == SENTINEL).all()
    s.check(rows=[0, 3])
    first = s.out.clone(), s.lse.clone()
    for _ in range(5):
        s.run(req_ids=ids, batch=2)
        assert torch.equal(s.out, first[0]) and torch.equal(s.lse, first[1])
    s.run()
    s.check()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        s.run()
        s.run()
    torch.cuda.current_stream().wait_stream(stream)
    for seed in (1, 2):
        s.q.copy_(torch.randn(s.q.shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16))
        s.out.fill_(SENTINEL)
        graph.replay()
        s.check()


def test_two_streams_of_clusters():
    """Two fast steps at once, with buffers of their own, give what they give alone."""
    steps = [Step(90 + i, 4 + i, 2, 2, 128, 1, 4, 40, 500 + 100 * i) for i in range(2)]
    alone = []
    for s in steps:
        s.run()
        alone.append(s.out.clone())
        s.check()
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for _ in range(30):
        for s, stream in zip(steps, streams):
            with torch.cuda.stream(stream):
                s.run()
    torch.cuda.synchronize()
    for s, a in zip(steps, alone):
        assert torch.equal(s.out, a)
