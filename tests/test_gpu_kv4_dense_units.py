"""Dense attention over the 4-bit cache in both of its ways: narrow page tables let few units
take a cluster of CTAs each, a wide table (the same requests, more columns) brings them to
runs that the grid shares. Inputs, reference and tolerances are those of test_gpu_kv4 (the
merges' part of its bound, 64 2^-23, covers the at most 8 + 8 steps of a cluster's)."""
import math

import numpy as np
import pytest
import torch

from tests.gpu_harness import dev_i32
from tests.test_gpu_kv4 import SENTINEL, Cache, _check_attention, _dense, _dense_sets, _lib, _sfi, _status  # noqa: F401

pytestmark = pytest.mark.gpu

WIDE = 5000


def _cache(seed, lens, hkv, d, wide):
    c = Cache(seed, lens, hkv, d, 0.5, 2.0)
    if wide:
        c.table = np.pad(c.table, ((0, 0), (0, WIDE)), constant_values=-1)
        c.upload()
    return c


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("B,hkv,G,d,T,longest,scores", [
    (1, 1, 1, 128, 1, 1, True),        # one token: all warps but one are without blocks
    (1, 2, 8, 64, 2, 1700, False),
    (2, 3, 2, 128, 3, 500, True),
    (5, 8, 2, 64, 1, 333, True),
    (13, 4, 4, 128, 1, 150, True),     # 52 units
    (9, 5, 2, 64, 8, 120, False),      # 45 units of sixteen rows
    (24, 4, 2, 128, 1, 100, True),     # 96 units
    (50, 4, 1, 64, 2, 90, False),      # 200 units
    (64, 8, 2, 128, 1, 70, True),      # 512 units
])
def test_dense_attention_by_units(B, hkv, G, d, T, longest, scores, wide):
    rng = np.random.default_rng(B * hkv + T)
    lens = [int(x) for x in rng.integers(T, longest + 1, B)]
    lens[-1], lens[0] = T, longest
    c = _cache(B + hkv, lens, hkv, d, wide)
    _, q, out, lse, sc, _, st = _dense(c, G, T, scores=scores)
    assert st.item() == 0
    rows = None if B < 10 else sorted({0, 1, B // 2, B - 2, B - 1})
    _check_attention(c, q, out, lse, T, G, 1 / math.sqrt(d), _dense_sets(c, T), sc, 4, 32, rows=rows)
    assert (out != SENTINEL).all() and (lse != SENTINEL).all()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("d,hkv,G,T", [(128, 2, 2, 1), (64, 3, 4, 4)])
def test_bad_requests_are_left_out_whole(d, hkv, G, T, wide):
    from sparse_kv_long_sfi_gb300 import _abi
    c = _cache(60, [700, 200, 40, 100], hkv, d, wide)
    c.table[1, 12] = c.pool.shape[0]  # its last page
    c.table[2, 0] = -5                # its first
    c.upload()
    _, q, out, lse, sc, _, st = _dense(c, G, T, scores=True)
    assert st.item() == _abi.SFI_DEV_BAD_PAGE
    for x in (out, lse, sc):
        assert (x[1:3] == SENTINEL).all()
    check = lambda rows: _check_attention(c, q, out, lse, T, G, 1 / math.sqrt(d), _dense_sets(c, T), sc, 4, 32, rows=rows)
    check([0, 3])
    c.table[1, 12], c.table[2, 0] = 0, 0
    c.upload()
    real, c.lens = c.lens, [700, T - 1, c.table.shape[1] * 16 + 1, 0]
    c.kv.seq_lens.copy_(dev_i32(c.lens))
    c.lens = real
    _, q, out, lse, sc, _, st = _dense(c, G, T, scores=True)
    assert st.item() == _abi.SFI_DEV_BAD_LEN
    for x in (out, lse, sc):
        assert (x[1:] == SENTINEL).all()
    check([0])


@pytest.mark.parametrize("wide", [False, True])
def test_subsets_repeats_and_graphs(wide):
    """Requests out of order, rows of the others left as they are; a run repeats to the bit; a graph
    follows lengths that change between its replays."""
    sfi = _sfi()
    T, G = 1, 2
    c = _cache(70, [335, 90, 32, 256, 16], 2, 128, wide)  # (positions up to these hold values)
    shape, q, out, lse, sc, ws, st = _dense(c, G, T, scores=True, req_ids=dev_i32([3, 0]), batch=2)
    for x in (out, lse, sc):
        assert (x[[1, 2, 4]] == SENTINEL).all()
    check = lambda rows: _check_attention(c, q, out, lse, T, G, 1 / math.sqrt(128), _dense_sets(c, T), sc, 4, 32, rows=rows)
    check([0, 3])
    first = out.clone()

    def run(**kw):
        sfi.sfi_kv4_dense_attn(shape, c.kv, 4, 32, q, out, lse=lse, scores=sc, workspace=ws, dev_status=st, **kw)
    for _ in range(5):
        run(req_ids=dev_i32([3, 0]), batch=2)
        assert torch.equal(out, first)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        run()
        run()
    torch.cuda.current_stream().wait_stream(stream)
    for lens in ([330, 90, 17, 256, 1], [335, 81, 32, 241, 16]):
        c.lens = lens
        c.kv.seq_lens.copy_(dev_i32(lens))
        sc.fill_(SENTINEL)
        graph.replay()
        check(None)
    assert st.item() == 0
