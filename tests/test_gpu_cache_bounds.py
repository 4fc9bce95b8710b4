"""Where the cache-side operators write, and where they reach: guard bands around every
output, pools and score arrays beyond 2^32 bytes, calls at once on two streams, and the
wrappers' checks of sizes."""
import numpy as np
import pytest
import torch

from tests.gpu_harness import dev_i32
from tests.test_gpu_guard_bands import BF16, F32, Guarded, _workspace
from tests.test_gpu_kv4 import Cache, _bf16

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


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("hkv,G,d,T", [(8, 2, 128, 1), (2, 4, 64, 2), (1, 4, 128, 4), (2, 8, 128, 1)])
def test_guard_bands_of_the_4bit_calls(hkv, G, d, T):
    sfi = _sfi()
    lens, sink, recent, k = [T, 17 + T, 300, 1500], 4, 32, 100
    c = Cache(3, lens, hkv, d)
    B, shape, st = len(lens), sfi.AttnShape(hkv * G, hkv, d), _status()
    pool = Guarded(c.pool.shape, torch.uint8, 0xA5)
    pool.v.copy_(c.d_pool)
    kv = sfi.PagedKV4(pool.v, c.kv.page_table, c.kv.seq_lens)
    rng = np.random.default_rng(1)
    new = [_bf16(rng.standard_normal((B, T, hkv, d))).cuda() for _ in range(2)]
    q = _bf16(rng.standard_normal((B, T, hkv * G, d))).cuda()
    checks = [("pool", pool)]
    sfi.sfi_kv4_append(shape, kv, *new, dev_status=st)
    # only the pages of the newest tokens changed
    touched = set()
    for r, n in enumerate(lens):
        touched |= {int(c.table[r, p]) for p in range((n - T) // 16, (n - 1) // 16 + 1)}
    rest = [i for i in range(len(c.pool)) if i not in touched]
    assert np.array_equal(pool.v.cpu().numpy()[rest], c.pool[rest])
    ko, vo = (Guarded((B, 21, hkv, d), torch.bfloat16, BF16) for _ in range(2))
    sfi.sfi_kv4_read(shape, kv, ko.v, vo.v, dev_status=st)
    checks += [("k_out", ko), ("v_out", vo)]
    stored = float(torch.tensor(BF16, dtype=torch.bfloat16).float())
    for r, n in enumerate(lens):
        assert (ko.v[r, min(n, 21):].float() == stored).all() and (vo.v[r, min(n, 21):].float() == stored).all()
    out, lse = Guarded((B, T, hkv * G, d), torch.float32, F32), Guarded((B, T, hkv * G), torch.float32, F32)
    scores = Guarded((B, hkv, max(lens) + 3), torch.float32, F32)
    ws = _workspace(sfi.sfi_kv4_workspace_size(shape, B, T))
    sfi.sfi_kv4_dense_attn(shape, kv, sink, recent, q, out.v, lse=lse.v, scores=scores.v, workspace=ws.v, dev_status=st)
    for r, n in enumerate(lens):
        assert (scores.v[r, :, n:] == F32).all()
    checks += [("out", out), ("lse", lse), ("scores", scores), ("workspace", ws)]
    counts = [0, 0, k, 7]
    idx = torch.arange(sink, sink + k, dtype=torch.int32, device="cuda").expand(B, hkv, k).contiguous()
    comp = sfi.alloc_kv4_compact(shape, [sink + n for n in counts])
    blocks = Guarded(tuple(comp.pool.shape), torch.uint8, 0xA5)
    comp.pool, comp.count = blocks.v, dev_i32(counts)
    sfi.sfi_kv4_compact_gather(shape, kv, idx, comp.count, sink, comp, dev_status=st)
    fout, flse = Guarded((B, T, hkv * G, d), torch.float32, F32), Guarded((B, T, hkv * G), torch.float32, F32)
    sfi.sfi_kv4_fast_attn(shape, kv, comp, sink, recent, q, fout.v, lse=flse.v, workspace=ws.v, dev_status=st)
    checks += [("blocks", blocks), ("fast out", fout), ("fast lse", flse)]
    torch.cuda.synchronize()
    assert st.item() == 0
    for name, g in checks:
        assert g.margins_intact(), name
    assert not ws.v[:512 * hkv * 4].any()


def test_guard_bands_of_the_norm_and_the_pages():
    sfi = _sfi()
    hq, hkv, d, T, B = 8, 2, 128, 5, 3
    shape, st = sfi.AttnShape(hq, hkv, d), _status()
    g = torch.Generator().manual_seed(0)
    x = torch.randn(B, T, (hq + 2 * hkv) * d, generator=g).to(torch.bfloat16).cuda()
    q, k, v = (t.unflatten(-1, (-1, d)) for t in x.split([hq * d, hkv * d, hkv * d], -1))
    kp, vp = (Guarded((7, hkv, 16, d), torch.bfloat16, BF16) for _ in range(2))
    qo, ko = Guarded((B, T, hq, d), torch.bfloat16, BF16), Guarded((B, T, hkv, d), torch.bfloat16, BF16)
    kv = sfi.PagedKV(kp.v, vp.v, dev_i32([[0, 6], [1, 2], [3, 4]]), dev_i32([32, 18, 5]))
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    sfi.sfi_qk_norm_rope(shape, sfi.Rope(sfi.rope_turns([0.5 ** i for i in range(64)])), q, k, v, qo.v, q_weight=w,
                         k_weight=w, k_out=ko.v, kv=kv, dev_status=st)
    pools = [Guarded((7, 24), torch.int64, -7) for _ in range(3)]
    for p in pools:
        p.v.copy_(torch.arange(168, device="cuda").view(7, 24))
    sfi.sfi_page_copy(sfi.PagePools([p.v for p in pools]), dev_i32([0, 6]), dev_i32([5, 1]), dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    for g in [kp, vp, qo, ko] + pools:
        assert g.margins_intact()


def test_pools_and_scores_beyond_32_bit_offsets():
    """Pages at the far end of a 4-bit pool of 6 GB, a bf16 pool of 5 GB and page pools of 6 GB; score
    rows that begin past 2^32 bytes."""
    sfi = _sfi()
    hkv, d = 8, 128
    shape, st = sfi.AttnShape(16, hkv, d), _status()
    pages = 330000
    big = torch.zeros(pages, hkv, 18 * d, dtype=torch.uint8, device="cuda")
    far = [pages - 1, pages - 7, pages - 100]
    lens = dev_i32([40, 40])
    near_pool = sfi.alloc_kv4_pool(shape, 3)
    kv = sfi.PagedKV4(big, dev_i32([[0, 0, 0], far]), lens)
    near = sfi.PagedKV4(near_pool, dev_i32([[0, 1, 2], [0, 1, 2]]), lens)
    g = torch.Generator().manual_seed(0)
    k, v = (torch.randn(2, 40, hkv, d, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    q = torch.randn(2, 1, 16, d, generator=g).to(torch.bfloat16).cuda()
    one, ws = dev_i32([1]), sfi.alloc_kv4_workspace(shape, 2)
    stride = 1 << 28  # request 1's rows begin 8 GB into the array
    outs = []
    for c, s in ((kv, torch.empty(2, hkv, stride, device="cuda")), (near, torch.empty(2, hkv, 64, device="cuda"))):
        sfi.sfi_kv4_append(shape, c, k, v, req_ids=one, dev_status=st)
        out, lse = torch.zeros(2, 1, 16, d, device="cuda"), torch.zeros(2, 1, 16, device="cuda")
        sfi.sfi_kv4_dense_attn(shape, c, 2, 3, q, out, lse=lse, scores=s, workspace=ws, req_ids=one, dev_status=st)
        ko, vo = torch.zeros_like(k), torch.zeros_like(v)
        sfi.sfi_kv4_read(shape, c, ko, vo, req_ids=one, dev_status=st)
        outs.append([out, lse, s[1, :, :40].clone(), ko, vo])
        del s
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    ids = torch.tensor([[5, 6, 7], far], dtype=torch.int64)
    sfi.sfi_page_copy(sfi.PagePools([big]), dev_i32(ids[1]), dev_i32(ids[0]), dev_status=st)
    assert torch.equal(big[5:8], big[far])
    del big, kv
    torch.cuda.empty_cache()
    kp = torch.zeros(170000, hkv, 16, d, dtype=torch.bfloat16, device="cuda")
    pkv = sfi.PagedKV(kp, torch.zeros_like(kp), dev_i32([[169999, 169990, 3]]), dev_i32([40]))
    x = torch.randn(1, 40, 16, d, generator=g).to(torch.bfloat16).cuda()
    ko = torch.empty_like(k[:1])
    sfi.sfi_qk_norm_rope(shape, None, x, k[:1], v[:1], torch.empty_like(x), k_out=ko, kv=pkv, dev_status=st)
    assert torch.equal(ko, k[:1])  # neither norm nor rotation: a copy
    for pool, src in ((pkv.k_pool, k), (pkv.v_pool, v)):
        got = pool[[169999, 169990, 3]].transpose(1, 2).reshape(48, hkv, d)
        assert torch.equal(got[:40], src[0])
    assert st.item() == 0


def test_two_streams_at_once():
    """The same calls from two streams, each with its own workspace and outputs, many times over."""
    sfi = _sfi()
    hkv, G, d = 2, 4, 128
    shape = sfi.AttnShape(hkv * G, hkv, d)
    caches = [Cache(70 + i, [3000, 40, 700], hkv, d) for i in range(2)]
    q = torch.randn(3, 1, hkv * G, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    want, streams, state = [], [torch.cuda.Stream() for _ in range(2)], []
    for c in caches:
        ws, out = sfi.alloc_kv4_workspace(shape, 3), torch.empty(3, 1, hkv * G, d, device="cuda")
        sfi.sfi_kv4_dense_attn(shape, c.kv, 4, 32, q, out, workspace=ws)
        want.append(out.clone())
        state.append((c, ws, out))
    torch.cuda.synchronize()
    for _ in range(30):
        for s, (c, ws, out) in zip(streams, state):
            with torch.cuda.stream(s):  # the current stream, and the argument, name the stream
                sfi.sfi_kv4_dense_attn(shape, c.kv, 4, 32, q, out, workspace=ws)
            sfi.sfi_kv4_dense_attn(shape, c.kv, 4, 32, q, out, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for w, (_, _, out) in zip(want, state):
        assert torch.equal(w, out)


def test_wrappers_check_sizes():
    sfi = _sfi()
    shape = sfi.AttnShape(4, 2, 64)
    c = Cache(80, [20, 30], 2, 64)
    kv = c.kv
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    f = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    ws = sfi.alloc_kv4_workspace(shape, 2)
    comp = sfi.alloc_kv4_compact(shape, [10])  # one request's layout for a batch of two
    pm = sfi.PageMap(kv.page_table, kv.seq_lens, torch.zeros(9, dtype=torch.int32, device="cuda"))
    bad = [
        lambda: sfi.sfi_kv4_append(shape, kv, bf(1, 1, 2, 64), bf(1, 1, 2, 64)),
        lambda: sfi.sfi_kv4_append(shape, kv, bf(2, 1, 2, 64), bf(2, 2, 2, 64)),
        lambda: sfi.sfi_kv4_append(shape, kv, bf(2, 1, 2, 64), bf(2, 1, 2, 64), new_lens=dev_i32([1])),
        lambda: sfi.sfi_kv4_append(shape, kv, bf(2, 1, 2, 64), bf(2, 1, 2, 64), batch=3),
        lambda: sfi.sfi_kv4_append(shape, kv, bf(2, 1, 2, 64), bf(2, 1, 2, 64), req_ids=dev_i32([0]), batch=2),
        lambda: sfi.sfi_kv4_append(shape, kv, bf(2, 1, 2, 64).float(), bf(2, 1, 2, 64)),
        lambda: sfi.sfi_kv4_append(shape, kv, bf(2, 2, 3, 64).transpose(1, 2), bf(2, 3, 2, 64)),
        lambda: sfi.sfi_kv4_append(shape, kv, bf(3, 2, 2, 64).transpose(0, 1)[:, :2], bf(2, 2, 2, 64)),
        lambda: sfi.sfi_kv4_read(shape, kv, bf(2, 1, 2, 64), bf(2, 1, 2, 64), first=dev_i32([0])),
        lambda: sfi.sfi_kv4_dense_attn(shape, kv, 0, 0, bf(1, 1, 4, 64), f(1, 1, 4, 64), workspace=ws),
        lambda: sfi.sfi_kv4_dense_attn(shape, kv, 0, 0, bf(2, 1, 4, 64), f(2, 1, 4, 32), workspace=ws),
        lambda: sfi.sfi_kv4_dense_attn(shape, kv, 0, 0, bf(2, 1, 4, 64), f(2, 1, 4, 64), scores=f(2, 64), workspace=ws),
        lambda: sfi.sfi_kv4_fast_attn(shape, kv, comp, 4, 8, bf(2, 1, 4, 64), f(2, 1, 4, 64), workspace=ws),
        lambda: sfi.sfi_kv4_compact_gather(shape, kv, dev_i32(np.zeros((2, 1, 4))), dev_i32([1, 1]), 4, comp),
        lambda: sfi.sfi_qk_norm_rope(shape, None, bf(2, 1, 4, 64), bf(2, 1, 2, 64), None, bf(2, 1, 4, 32)),
        lambda: sfi.sfi_qk_norm_rope(shape, None, bf(2, 1, 64, 4).transpose(2, 3), bf(2, 1, 2, 64), None, bf(2, 1, 4, 64)),
        lambda: sfi.sfi_qk_norm_rope(shape, None, bf(2, 1, 4, 64), bf(2, 1, 2, 64), None, bf(2, 1, 4, 64),
                                     k_out=bf(2, 1, 2, 64), batch=3),
        lambda: sfi.sfi_page_copy(sfi.PagePools([bf(4, 8)]), dev_i32([1]), dev_i32([1, 2])),
        lambda: sfi.PagePools([bf(4, 8), bf(5, 8)]),
        lambda: sfi.PagePools([]),
        lambda: sfi.sfi_page_reserve(pm, None, dev_i32([1]), dev_i32([0, 1])),
        lambda: sfi.sfi_page_compact(pm, sfi.PagePools([bf(9, 8)]), dev_i32([[0]]), pm.ref_count, dev_i32([0])),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    with pytest.raises(sfi.SFIError):  # neither pages nor k_out
        sfi.sfi_qk_norm_rope(shape, None, bf(2, 1, 4, 64), bf(2, 1, 2, 64), None, bf(2, 1, 4, 64))
    with pytest.raises(sfi.SFIError):  # the map's own counts as the new ones
        sfi.sfi_page_compact(pm, sfi.PagePools([bf(9, 8)]), torch.empty_like(pm.page_table), pm.ref_count, dev_i32([0]),
                             workspace=sfi.alloc_page_workspace(pm))
