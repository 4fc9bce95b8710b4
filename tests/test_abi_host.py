"""The C-ABI library builds, loads and exports every entry point include/sfi.h
declares; host-side argument validation answers without touching a GPU."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "sfi.h")


@pytest.fixture(scope="module")
def libsfi():
    from sparse_kv_long_sfi_gb300 import _abi, build
    build.build()
    return _abi.lib()


def declared_functions():
    text = open(HEADER).read()
    return re.findall(r"^SFI_API\s+[\w\s\*]+?\b(sfi_\w+)\s*\(", text, flags=re.M)


def test_header_declares_the_five_hot_path_calls():
    names = declared_functions()
    for n in ["sfi_paged_kv_append", "sfi_fast_decode_attn", "sfi_slow_dense_attn_with_scores", "sfi_select_topk",
              "sfi_compact_gather"]:
        assert n in names


def test_library_exports_every_declared_symbol(libsfi):
    from sparse_kv_long_sfi_gb300 import _abi
    names = declared_functions()
    assert set(names) == set(_abi.PROTOTYPES)
    for n in names:
        assert hasattr(libsfi, n), n


def test_library_exports_nothing_else(libsfi):
    import subprocess
    from sparse_kv_long_sfi_gb300 import build
    out = subprocess.run(["nm", "-D", "--defined-only", build.LIB], capture_output=True, text=True).stdout
    exported = {l.split()[-1] for l in out.splitlines() if l.strip()}
    assert exported == set(declared_functions())


def test_version_and_status_strings(libsfi):
    assert libsfi.sfi_version() == 1
    assert libsfi.sfi_status_string(0) == b"SFI_OK"
    assert libsfi.sfi_status_string(3) == b"SFI_ERR_WORKSPACE"
    assert libsfi.sfi_status_string(99) == b"SFI_ERR_UNKNOWN"


def _shape(hq=16, hkv=8, d=128, p=16):
    from sparse_kv_long_sfi_gb300 import _abi
    return _abi.sfi_attn_shape(hq, hkv, d, p, 0.0)


def _paged(npages=4, maxp=4):
    from sparse_kv_long_sfi_gb300 import _abi
    # dummy, 16-byte aligned host addresses: validation never dereferences them
    return _abi.sfi_paged_kv(4096, 8192, npages, maxp, 12288, 16384)


@pytest.mark.parametrize("shape_args,expect", [
    ((16, 8, 96, 16), 2),    # head_dim 96 unsupported
    ((16, 8, 128, 32), 2),   # page size 32 unsupported
    ((48, 4, 128, 16), 2),   # G = 12 unsupported
    ((16, 5, 128, 16), 1),   # Hq not a multiple of Hkv
    ((0, 8, 128, 16), 1),
])
def test_shape_validation_before_launch(libsfi, shape_args, expect):
    sh = _shape(*shape_args)
    kv = _paged()
    st = libsfi.sfi_slow_dense_attn_with_scores(ctypes.byref(sh), ctypes.byref(kv), 4, 32, 4096, None, None, 8192,
                                                None, None, 0, None, 1, 0, 0, 0, None, 0, None, None)
    assert st == expect


def test_null_and_negative_arguments(libsfi):
    from sparse_kv_long_sfi_gb300 import _abi
    sh, kv = _shape(), _paged()
    assert libsfi.sfi_paged_kv_append(None, ctypes.byref(kv), 4096, 4096, None, 1, None, None) == 1
    assert libsfi.sfi_paged_kv_append(ctypes.byref(sh), None, 4096, 4096, None, 1, None, None) == 1
    assert libsfi.sfi_paged_kv_append(ctypes.byref(sh), ctypes.byref(kv), None, 4096, None, 1, None, None) == 1
    assert libsfi.sfi_paged_kv_append(ctypes.byref(sh), ctypes.byref(kv), 4097, 4096, None, 1, None, None) == 1
    comp = _abi.sfi_compact_kv(4096, 4096, 100, 4096, 4096, 4096)
    assert libsfi.sfi_fast_decode_attn(ctypes.byref(sh), ctypes.byref(kv), ctypes.byref(comp), -1, 32, 4096, None,
                                       None, 4096, None, None, 1, 0, 0, 0, None, 0, None, None) == 1
    assert libsfi.sfi_fast_decode_attn(ctypes.byref(sh), ctypes.byref(kv), None, 4, 32, 4096, None, None, 4096,
                                       None, None, 1, 0, 0, 0, None, 0, None, None) == 1
    # k_new without v_new
    assert libsfi.sfi_fast_decode_attn(ctypes.byref(sh), ctypes.byref(kv), ctypes.byref(comp), 4, 32, 4096, 4096,
                                       None, 4096, None, None, 1, 0, 0, 0, None, 0, None, None) == 1
    assert libsfi.sfi_select_topk(None, 16, 8, 4096, 4, 32, 4096, 8, 4096, 4096, None, 1, None, None) == 1
    assert libsfi.sfi_select_topk(4096, 0, 8, 4096, 4, 32, 4096, 8, 4096, 4096, None, 1, None, None) == 1
    assert libsfi.sfi_compact_gather(ctypes.byref(sh), ctypes.byref(kv), 4096, 4096, -1, 4, ctypes.byref(comp),
                                     None, 1, None, None) == 1
    bad_pages = _abi.sfi_paged_kv(4096, 8192, 0, 4, 12288, 16384)
    assert libsfi.sfi_paged_kv_append(ctypes.byref(sh), ctypes.byref(bad_pages), 4096, 4096, None, 1, None,
                                      None) == 1


def test_empty_batch_is_a_no_op(libsfi):
    sh, kv = _shape(), _paged()
    assert libsfi.sfi_paged_kv_append(ctypes.byref(sh), ctypes.byref(kv), 4096, 4096, None, 0, None, None) == 0
    assert libsfi.sfi_select_topk(4096, 16, 8, 4096, 4, 32, 4096, 8, 4096, 4096, None, 0, None, None) == 0


def test_workspace_size_rejects_bad_shapes(libsfi):
    sh = _shape(16, 8, 96)
    assert libsfi.sfi_workspace_size(ctypes.byref(sh), 4, 1024, 0) == 0
    assert libsfi.sfi_plan_splits(ctypes.byref(sh), 4, 1024, 0) == 0
    assert libsfi.sfi_plan_splits(ctypes.byref(_shape()), 4, 0, 0) == 1  # no token bound: one split
    assert libsfi.sfi_plan_splits(ctypes.byref(_shape()), 4, 4096, 3) == 3  # explicit request honoured
    for bad in (0, -1, 9, 16):
        assert libsfi.sfi_attn_cluster_capacity(bad) == 0


def test_cluster_capacity_needs_a_device(libsfi):
    """The capacity query answers 0 for every valid size when there is no CUDA device
    (so automatic plans keep the slot-count rule), and a positive count with one."""
    import torch
    caps = [libsfi.sfi_attn_cluster_capacity(c) for c in range(1, 9)]
    if torch.cuda.is_available():
        assert all(c > 0 for c in caps)
    else:
        assert caps == [0] * 8
        assert libsfi.sfi_plan_splits(ctypes.byref(_shape()), 4, 4096, 3) == 3  # plans still answer


def test_multi_token_calls_validate_on_the_host(libsfi):
    from sparse_kv_long_sfi_gb300 import _abi
    sh, kv = _shape(), _paged()  # G = 2: at most 8 tokens
    comp = _abi.sfi_compact_kv(4096, 4096, 100, 4096, 4096, 4096)

    def verify(T, batch=1, scores=None, stride=0):
        return libsfi.sfi_dense_verify_attn(ctypes.byref(sh), ctypes.byref(kv), 4, 32, 4096, T, None, None, 8192, None,
                                            scores, stride, None, batch, 0, 0, 0, None, 0, None, None)

    def draft(T, c=comp, batch=1):
        return libsfi.sfi_sparse_draft_attn(ctypes.byref(sh), ctypes.byref(kv), c and ctypes.byref(c), 4, 32, 4096,
                                            T, None, None, 8192, None, None, batch, 0, 0, 0, None, 0, None, None)

    assert verify(0) == 1 and verify(17) == 1
    assert verify(9) == 2                      # 9 tokens x G = 2 > 16 rows
    assert verify(8, batch=0) == 0             # empty batch: nothing to do
    assert verify(4, scores=4096, stride=0) == 1
    assert draft(0) == 1 and draft(9) == 2 and draft(4, c=None) == 1
    assert draft(8, batch=0) == 0
    sh8 = _shape(32, 4)                        # G = 8: two tokens
    assert libsfi.sfi_dense_verify_attn(ctypes.byref(sh8), ctypes.byref(kv), 4, 32, 4096, 3, None, None, 8192, None,
                                        None, 0, None, 1, 0, 0, 0, None, 0, None, None) == 2
    # k_new without v_new
    assert libsfi.sfi_dense_verify_attn(ctypes.byref(sh), ctypes.byref(kv), 4, 32, 4096, 2, 4096, None, 8192, None,
                                        None, 0, None, 1, 0, 0, 0, None, 0, None, None) == 1
    assert libsfi.sfi_paged_kv_append_tokens(ctypes.byref(sh), ctypes.byref(kv), 4096, 4096, 0, None, 1, None,
                                             None) == 1
    assert libsfi.sfi_paged_kv_append_tokens(ctypes.byref(sh), ctypes.byref(kv), 4096, 4096, 5, None, 0, None,
                                             None) == 0
    assert libsfi.sfi_multi_workspace_size(ctypes.byref(sh), 4, 0, 1024, 0) == 0


def test_select_compact_validates_on_the_host(libsfi):
    from sparse_kv_long_sfi_gb300 import _abi
    sh, kv = _shape(), _paged()
    comp = _abi.sfi_compact_kv(4096, 4096, 100, 4096, 4096, 4096)

    def call(scores=4096, stride=16, k=4096, idx=4096, cnt=4096, c=comp, batch=1, sink=4):
        return libsfi.sfi_select_compact(ctypes.byref(sh), ctypes.byref(kv), scores, stride, sink, 32, k, 8, idx, cnt,
                                         c and ctypes.byref(c), None, batch, None, None)

    assert call(scores=None) == 1 and call(stride=0) == 1 and call(k=None) == 1 and call(idx=None) == 1
    assert call(cnt=None) == 1 and call(c=None) == 1 and call(sink=-1) == 1
    assert call(c=_abi.sfi_compact_kv(4097, 4096, 100, 4096, 4096, 4096)) == 1  # unaligned compact K
    assert call(batch=0) == 0


def test_binding_constants_match_the_header():
    """Every numeric #define and status enumerator of include/sfi.h has the same value
    in the Python binding."""
    from sparse_kv_long_sfi_gb300 import _abi
    text = open(os.path.join(os.path.dirname(__file__), "..", "include", "sfi.h")).read()
    defines = {m.group(1): int(m.group(2)) for m in re.finditer(r"^#define (SFI_(?:DEV|ATTN|MAX)_\w+) (\d+)u?\b", text, re.M)}
    enums = {m.group(1): int(m.group(2)) for m in re.finditer(r"^\s+(SFI_(?:OK|ERR_\w+)) = (\d+)", text, re.M)}
    assert len(defines) >= 10 and len(enums) == 5
    for name, value in {**defines, **enums}.items():
        assert getattr(_abi, name) == value, name


def test_qk_norm_rope_validates_on_the_host(libsfi):
    from sparse_kv_long_sfi_gb300 import _abi
    rope = _abi.sfi_rope(4096, None, 128, 1, 0)

    def call(sh=_shape(), rope=rope, q=4096, qs=2048, k=4096, ks=1024, v=4096, vs=1024, qw=None, eps=1e-6, pos=None,
             axis_stride=0, T=1, lens=None, q_out=4096, k_out=4096, kv=_paged(), batch=1):
        return libsfi.sfi_qk_norm_rope(ctypes.byref(sh), rope and ctypes.byref(rope), q, qs, k, ks, v, vs, qw, None, eps,
                                       pos, axis_stride, T, None, lens, q_out, k_out, kv and ctypes.byref(kv), None,
                                       batch, None, None)

    assert call(batch=0) == 0
    assert call(sh=_shape(16, 8, 96)) == 2 and call(sh=_shape(16, 5)) == 1
    assert call(q=None) == 1 and call(k=None) == 1 and call(v=None) == 1 and call(q_out=None) == 1
    assert call(k_out=None, kv=None) == 1          # nowhere to put K
    assert call(q=4104) == 1 and call(k_out=4100) == 1 and call(qw=4098) == 1
    assert call(qs=2040) == 1 and call(qs=2052) == 1 and call(ks=1020) == 1 and call(vs=1016) == 1
    assert call(T=0) == 1 and call(batch=-1) == 1 and call(eps=-1.0) == 1 and call(eps=float("nan")) == 1
    for rot, expect in ((-16, 2), (24, 2), (144, 2), (0, 0), (16, 0)):
        assert call(rope=_abi.sfi_rope(4096, None, rot, 1, 0), batch=0) == expect
    assert call(rope=_abi.sfi_rope(None, None, 64, 1, 0)) == 1
    assert call(rope=_abi.sfi_rope(4096, None, 64, 0, 0)) == 1 and call(rope=_abi.sfi_rope(4096, None, 64, 9, 0)) == 1
    assert call(rope=_abi.sfi_rope(4096, None, 64, 1, 2)) == 1
    assert call(kv=None) == 1                      # rotation by neither slot nor position
    assert call(kv=None, lens=4096, batch=0) == 0
    assert call(rope=_abi.sfi_rope(4096, None, 64, 3, 0), pos=4096, axis_stride=4, T=5) == 1
    assert call(rope=None, kv=None, v=None, batch=0) == 0


def test_rope_turns_are_exact_modulo_one_turn():
    """turns[i] is inv_freq / (2 pi) in 2^-64 turns: close to the fp64 quotient, and wrapped
    for more than half a turn."""
    import math
    import sparse_kv_long_sfi_gb300 as sfi
    f = [1.0, 1e-6, 0.37, 4.0, 2 * math.pi * 1.75]
    got = sfi.rope_turns(f, device="cpu").tolist()
    for x, t in zip(f, got):
        turn = x / (2 * math.pi) % 1.0
        assert abs((t % 2 ** 64) / 2 ** 64 - turn) <= 2.0 ** -51, x


def _kv4(k_scale=1.0, v_scale=1.0, pool=4096, npages=4, maxp=4):
    from sparse_kv_long_sfi_gb300 import _abi
    return _abi.sfi_paged_kv4(pool, npages, maxp, 12288, 16384, k_scale, v_scale)


def test_kv4_calls_validate_on_the_host(libsfi):
    from sparse_kv_long_sfi_gb300 import _abi
    comp = _abi.sfi_compact_kv4(4096, 8, 4096, 4096, 4096)
    ref = lambda x: x and ctypes.byref(x)  # noqa: E731

    def append(sh=_shape(), kv=_kv4(), k=4096, v=4096, T=1, batch=1, ks=1024, vs=1024):
        return libsfi.sfi_kv4_append(ref(sh), ref(kv), k, ks, v, vs, T, None, None, batch, None, None)

    def read(sh=_shape(), kv=_kv4(), k=4096, v=4096, T=1, batch=1):
        return libsfi.sfi_kv4_read(ref(sh), ref(kv), k, v, T, None, None, batch, None, None)

    def gather(kv=_kv4(), idx=4096, count=4096, k_cap=8, sink=4, c=comp, batch=1):
        return libsfi.sfi_kv4_compact_gather(ref(_shape()), ref(kv), idx, count, k_cap, sink, ref(c), None, batch, None,
                                             None)

    def dense(sh=_shape(), kv=_kv4(), sink=4, recent=32, q=4096, T=1, out=4096, scores=None, stride=0, batch=1, ws=None,
              ws_bytes=0):
        return libsfi.sfi_kv4_dense_attn(ref(sh), ref(kv), sink, recent, q, T, out, None, scores, stride, None, batch, ws,
                                         ws_bytes, None, None)

    def fast(kv=_kv4(), c=comp, q=4096, T=1, out=4096, batch=1):
        return libsfi.sfi_kv4_fast_attn(ref(_shape()), ref(kv), ref(c), 4, 32, q, T, out, None, None, batch, None, 0, None,
                                        None)

    for call in (append, read):
        assert call(batch=0) == 0
        assert call(sh=_shape(16, 8, 96)) == 2 and call(k=None) == 1 and call(v=4097) == 1
        assert call(T=0) == 1 and call(batch=-1) == 1
    assert append(ks=1016) == 1 and append(vs=1023) == 1 and append(vs=1028) == 1 and append(ks=2048, batch=0) == 0
    for call in (append, read, gather, dense, fast):
        assert call(kv=None) == 1
        assert call(kv=_kv4(pool=4097)) == 1 and call(kv=_kv4(npages=0)) == 1 and call(kv=_kv4(maxp=0)) == 1
        assert call(kv=_kv4(maxp=1 << 28)) == 2
        for bad in (0.0, -1.0, 3.0, float("inf"), float("nan"), 2.0 ** -100, 2.0 ** 90):
            assert call(kv=_kv4(k_scale=bad)) == 1 and call(kv=_kv4(v_scale=bad)) == 1
        assert call(kv=_kv4(2.0 ** -20, 2.0 ** 20), batch=0) == 0
    assert gather(idx=None) == 1 and gather(k_cap=-1) == 1 and gather(sink=-1) == 1 and gather(c=None) == 1
    assert gather(k_cap=0, sink=0) == 0
    assert gather(c=_abi.sfi_compact_kv4(4096, 0, 4096, 4096, 4096)) == 1
    assert fast(c=None) == 1 and fast(c=_abi.sfi_compact_kv4(4104, 8, 4096, 4096, 4096)) == 1
    assert dense(q=None) == 1 and dense(out=4100) == 1 and dense(sink=-1) == 1 and dense(recent=-1) == 1
    assert dense(T=0) == 1 and dense(T=17) == 1 and dense(T=9) == 2 and dense(T=8, batch=0) == 0
    assert dense(scores=4096, stride=0) == 1
    assert dense() == 3 and fast() == 3                   # no workspace
    assert dense(ws=4096, ws_bytes=16) == 3 and dense(ws=4100, ws_bytes=1 << 40) == 3
    sh = _shape()
    assert libsfi.sfi_kv4_workspace_size(ref(sh), 4, 8) > 0 and libsfi.sfi_kv4_workspace_size(ref(sh), 4, 9) == 0
    assert libsfi.sfi_kv4_workspace_size(ref(_shape(16, 8, 96)), 4, 1) == 0


def test_page_calls_validate_on_the_host(libsfi):
    from sparse_kv_long_sfi_gb300 import _abi
    ref = lambda x: x and ctypes.byref(x)  # noqa: E731
    mp = lambda **k: _abi.sfi_page_map(**{**dict(page_table=4096, seq_lens=4096, ref_count=4096, num_reqs=4,  # noqa: E731
                                                max_pages_per_req=8, num_pages=32, page_size=16), **k})
    pl = lambda **k: _abi.sfi_page_pools(**{**dict(pools=4096, num_pools=2, page_bytes=4608, num_pages=32), **k})  # noqa: E731

    def copy(q=pl(), src=4096, dst=4096, n=1):
        return libsfi.sfi_page_copy(ref(q), src, dst, n, None, None)

    def fork(m=mp(), src=4096, dst=4096, n=1):
        return libsfi.sfi_page_fork(ref(m), src, dst, None, n, None, None)

    def reserve(m=mp(), q=pl(), new=4096, reqs=4096, n=1, ws=4096, size=1 << 20):
        return libsfi.sfi_page_reserve(ref(m), ref(q), new, reqs, n, ws, size, None, None)

    def free(m=mp(), reqs=4096, n=1):
        return libsfi.sfi_page_free(ref(m), reqs, n, None, None)

    def compact(m=mp(), q=pl(), table=8192, ref_out=8192, live=8192, ws=4096, size=1 << 20):
        return libsfi.sfi_page_compact(ref(m), ref(q), table, ref_out, live, ws, size, None, None)

    for call in (fork, reserve, free, compact):
        assert call(m=None) == 1 and call(m=mp(page_table=None)) == 1 and call(m=mp(seq_lens=None)) == 1
        assert call(m=mp(ref_count=None)) == 1 and call(m=mp(num_reqs=0)) == 1 and call(m=mp(num_pages=0)) == 1
        assert call(m=mp(max_pages_per_req=0)) == 1 and call(m=mp(page_size=32)) == 2
        assert call(m=mp(max_pages_per_req=1 << 28)) == 2
    for call in (copy, reserve, compact):
        assert call(q=pl(pools=None)) == 1 and call(q=pl(num_pools=0)) == 1 and call(q=pl(page_bytes=24)) == 1
        assert call(q=pl(page_bytes=0)) == 1 and call(q=pl(num_pages=0)) == 1
    assert copy(q=None) == 1 and copy(src=None) == 1 and copy(dst=None) == 1 and copy(n=-1) == 1 and copy(n=0) == 0
    assert fork(src=None) == 1 and fork(dst=None) == 1 and fork(n=-1) == 1 and fork(n=0) == 0
    assert free(reqs=None) == 1 and free(n=-1) == 1 and free(n=0) == 0
    assert reserve(new=None) == 1 and reserve(n=-1) == 1 and reserve(n=1025) == 2 and reserve(n=0) == 0
    assert reserve(reqs=None, n=5) == 1 and reserve(q=pl(num_pages=31)) == 1
    assert reserve(ws=None) == 3 and reserve(ws=4100) == 3 and reserve(size=16) == 3
    assert compact(q=None) == 1 and compact(table=None) == 1 and compact(ref_out=None) == 1 and compact(live=None) == 1
    assert compact(table=4096) == 1 and compact(ref_out=4096) == 1 and compact(q=pl(num_pages=31)) == 1
    assert compact(ws=None) == 3 and compact(size=16) == 3
    m = mp()
    assert libsfi.sfi_page_workspace_size(ref(m)) >= 3 * 32 * 4 and libsfi.sfi_page_workspace_size(None) == 0
