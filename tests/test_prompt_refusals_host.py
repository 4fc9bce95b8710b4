"""What the calls around prompts, evicted caches and drafts refuse before anything is launched."""
import ctypes

import pytest
import torch

import sparse_kv_long_sfi_gb300 as sfi
from sparse_kv_long_sfi_gb300 import _abi, api

INVALID, UNSUPPORTED = 1, 2
A = 4096  # an aligned address; nothing is read


@pytest.fixture(scope="module")
def lib():
    from sparse_kv_long_sfi_gb300 import build
    build.build()
    return _abi.lib()


def _shape(hq=16, hkv=8, d=128, p=16):
    return ctypes.byref(_abi.sfi_attn_shape(hq, hkv, d, p, 0.0))


def _paged(k=A, v=2 * A, pages=4, maxp=4, table=3 * A, lens=4 * A):
    return ctypes.byref(_abi.sfi_paged_kv(k, v, pages, maxp, table, lens))


WINDOW = dict(shape=_shape(), kv=_paged(), sink=4, recent=32, q=A, q_stride=2048, num_reqs=3, num_tokens=5, new_lens=None,
              out=A, lse=A, req_ids=None, batch=0, dev_status=None, stream=None)
MASS = dict(shape=_shape(), kv=_paged(), sink=4, recent=32, q=A, q_stride=2048, num_reqs=3, num_tokens=5, new_lens=None,
            lse=A, mass=A, mass_stride=64, decay=1.0, req_ids=None, batch=0, dev_status=None, stream=None)
EVICT = dict(shape=_shape(), kv=_paged(), mass=A, mass_stride=64, sink=4, recent=32, k_per_req=A, k_cap=8, idx_out=A,
             count_out=A, mass_out=None, new_lens=A, req_ids=None, batch=0, dev_status=None, stream=None)
VERIFY = dict(target=A, target_stride=100, draft=A, draft_stride=100, tokens=A, u=A, vocab=100, num_drafts=3,
              draft_lens=None, seq_lens=None, out_tokens=A, accepted=A, new_lens=None, req_ids=None, batch=0,
              dev_status=None, stream=None)
TRIM = dict(map=ctypes.byref(_abi.sfi_page_map(A, A, A, 3, 4, 9, 16)), new_lens=A, reqs=None, n=0, dev_status=None,
            stream=None)


def test_no_requests_is_no_error(lib):
    for name, args in (("window_attn", WINDOW), ("attn_mass", MASS), ("kv_evict", EVICT), ("verify_tokens", VERIFY),
                       ("page_trim", TRIM)):
        assert getattr(lib, "sfi_" + name)(*args.values()) == 0, name


@pytest.mark.parametrize("change,status", [
    (dict(shape=_shape(d=96)), UNSUPPORTED), (dict(shape=_shape(p=32)), UNSUPPORTED), (dict(shape=_shape(48, 4)), UNSUPPORTED),
    (dict(shape=_shape(16, 5)), INVALID), (dict(shape=None), INVALID), (dict(kv=None), INVALID),
    (dict(kv=_paged(k=None)), INVALID), (dict(kv=_paged(k=A + 8)), INVALID), (dict(kv=_paged(pages=0)), INVALID),
    (dict(kv=_paged(pages=1 << 24)), UNSUPPORTED), (dict(kv=_paged(maxp=1 << 27)), UNSUPPORTED),
    (dict(sink=-1), INVALID), (dict(recent=-1), INVALID), (dict(q=None), INVALID), (dict(q=A + 8), INVALID),
    (dict(q_stride=2047), INVALID), (dict(q_stride=2040), INVALID), (dict(q_stride=2052), INVALID),
    (dict(q_stride=1 << 38), UNSUPPORTED), (dict(num_tokens=0), INVALID), (dict(num_reqs=-1), INVALID),
    (dict(batch=-1), INVALID), (dict(batch=65536), UNSUPPORTED),
    (dict(num_reqs=1 << 16, num_tokens=1 << 15), UNSUPPORTED),
])
def test_attention_and_weights(lib, change, status):
    assert lib.sfi_window_attn(*{**WINDOW, **change}.values()) == status
    assert lib.sfi_attn_mass(*{**MASS, **change}.values()) == status


@pytest.mark.parametrize("change", [dict(out=None), dict(out=A + 8)])
def test_attention(lib, change):
    assert lib.sfi_window_attn(*{**WINDOW, **change}.values()) == INVALID


@pytest.mark.parametrize("change", [dict(lse=None), dict(mass=None), dict(mass_stride=0), dict(decay=float("nan")),
                                    dict(decay=float("inf"))])
def test_weights(lib, change):
    assert lib.sfi_attn_mass(*{**MASS, **change}.values()) == INVALID


@pytest.mark.parametrize("change,status", [
    (dict(shape=_shape(d=96)), UNSUPPORTED), (dict(kv=None), INVALID), (dict(mass=None), INVALID),
    (dict(k_per_req=None), INVALID), (dict(idx_out=None), INVALID), (dict(count_out=None), INVALID),
    (dict(new_lens=None), INVALID), (dict(new_lens=4 * A), INVALID), (dict(mass_out=A), INVALID),
    (dict(mass_stride=0), INVALID), (dict(sink=-1), INVALID), (dict(recent=-1), INVALID), (dict(k_cap=-1), INVALID),
    (dict(batch=-1), INVALID), (dict(batch=65536), UNSUPPORTED),
])
def test_eviction(lib, change, status):
    assert lib.sfi_kv_evict(*{**EVICT, **change}.values()) == status


@pytest.mark.parametrize("change,status", [
    (dict(target=None), INVALID), (dict(tokens=None), INVALID), (dict(u=None), INVALID), (dict(out_tokens=None), INVALID),
    (dict(accepted=None), INVALID), (dict(seq_lens=A), INVALID), (dict(new_lens=A), INVALID), (dict(vocab=0), INVALID),
    (dict(num_drafts=0), INVALID), (dict(target_stride=99), INVALID), (dict(draft_stride=99), INVALID),
    (dict(batch=-1), INVALID), (dict(vocab=1 << 21, target_stride=1 << 21, draft_stride=1 << 21), UNSUPPORTED),
])
def test_verification(lib, change, status):
    assert lib.sfi_verify_tokens(*{**VERIFY, **change}.values()) == status


def test_trim(lib):
    for change, status in ((dict(map=None), INVALID), (dict(new_lens=None), INVALID), (dict(n=-1), INVALID),
                           (dict(n=4), INVALID),
                           (dict(map=ctypes.byref(_abi.sfi_page_map(A, A, A, 3, 4, 9, 32))), UNSUPPORTED)):
        assert lib.sfi_page_trim(*{**TRIM, **change}.values()) == status, change


# ---- the binding's own checks ---------------------------------------------------------------------------------------


@pytest.fixture
def host(monkeypatch):
    """Tensors of host memory pass for those of the current device; nothing is launched."""
    real = api._need

    def need(t, dtype, name):
        if t is not None and t.dtype == dtype and t.is_contiguous():
            return
        real(t, dtype, name)

    monkeypatch.setattr(api, "_need", need)
    monkeypatch.setattr(api, "_on_current_device", lambda t, name: None)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: -1, raising=False)
    monkeypatch.setattr(api, "_stream_here", lambda stream, dev: None)
    calls = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: calls.append((name, a)) or 0

    monkeypatch.setattr(api._abi, "lib", lambda: Lib())
    return calls


def _bf16(*dims):
    return torch.zeros(*dims, dtype=torch.bfloat16)


def _i32(*dims):
    return torch.zeros(*dims, dtype=torch.int32)


def _attn():
    shape = sfi.AttnShape(8, 2, 64)
    kv = sfi.PagedKV(_bf16(5, 2, 16, 64), _bf16(5, 2, 16, 64), _i32(3, 4), _i32(3))
    return shape, kv, dict(q=_bf16(3, 6, 8, 64), out=_bf16(3, 6, 8, 64), lse=torch.zeros(3, 6, 8),
                           mass=torch.zeros(3, 2, 64), mass_out=torch.zeros(3, 2, 64), new_lens=_i32(3), k_per_req=_i32(3),
                           idx_out=_i32(3, 2, 7), count_out=_i32(3))


def _window(shape, kv, a, **kw):
    sfi.sfi_window_attn(shape, kv, 4, 32, a["q"], a["out"], lse=a["lse"], new_lens=a["new_lens"], **kw)


def _mass(shape, kv, a, **kw):
    sfi.sfi_attn_mass(shape, kv, 4, 32, a["q"], a["lse"], a["mass"], new_lens=a["new_lens"], **kw)


def _evict(shape, kv, a, **kw):
    sfi.sfi_kv_evict(shape, kv, a["mass"], 4, 32, a["k_per_req"], a["idx_out"], a["count_out"], a["new_lens"],
                     mass_out=a["mass_out"], **kw)


@pytest.mark.parametrize("call,wrong", [
    (_window, dict(q=_bf16(2, 6, 8, 64))), (_window, dict(q=_bf16(3, 6, 4, 64))), (_window, dict(q=torch.zeros(3, 6, 8, 64))),
    (_window, dict(out=_bf16(3, 5, 8, 64))), (_window, dict(out=torch.zeros(3, 6, 8, 64))), (_window, dict(lse=torch.zeros(3, 6))),
    (_window, dict(new_lens=_i32(2))), (_window, dict(q=_bf16(3, 6, 64, 8).transpose(2, 3))),
    (_mass, dict(q=_bf16(2, 6, 8, 64))), (_mass, dict(lse=torch.zeros(3, 5, 8))), (_mass, dict(mass=torch.zeros(3, 64))),
    (_mass, dict(mass=torch.zeros(2, 2, 64))), (_mass, dict(mass=_bf16(3, 2, 64))), (_mass, dict(new_lens=_i32(4))),
    (_evict, dict(mass=torch.zeros(3, 8, 64))), (_evict, dict(mass_out=torch.zeros(3, 2, 63))), (_evict, dict(idx_out=_i32(3, 7))),
    (_evict, dict(k_per_req=_i32(2))), (_evict, dict(count_out=_i32(4))), (_evict, dict(new_lens=torch.zeros(3))),
])
def test_shapes(host, call, wrong):
    shape, kv, a = _attn()
    call(shape, kv, a)
    assert len(host) == 1
    with pytest.raises(ValueError):
        call(shape, kv, {**a, **wrong})
    with pytest.raises(ValueError):
        call(shape, kv, a, batch=4)
    with pytest.raises(ValueError):
        call(sfi.AttnShape(8, 2, 128), kv, a)
    assert len(host) == 1


def test_queries_of_a_fused_projection(host):
    shape, kv, a = _attn()
    fused = _bf16(3, 6, 12, 64)
    _window(shape, kv, {**a, "q": fused[:, :, :8]})
    assert host[-1][1][5] == 12 * 64 and host[-1][1][6:8] == (3, 6)


def _verify(a):
    sfi.sfi_verify_tokens(a["target"], a["draft"], a["tokens"], a["u"], a["out_tokens"], a["accepted"],
                          draft_lens=a.get("draft_lens"))


@pytest.mark.parametrize("wrong", [
    dict(target=torch.zeros(2, 4, 50, dtype=torch.float64)), dict(target=torch.zeros(2, 200)), dict(draft=torch.zeros(2, 3, 49)),
    dict(draft=torch.zeros(2, 4, 50)), dict(draft=torch.zeros(3, 3, 50)), dict(tokens=_i32(2, 4)), dict(u=torch.zeros(2, 3)),
    dict(out_tokens=_i32(2, 3)), dict(accepted=_i32(3)), dict(tokens=torch.zeros(2, 3, dtype=torch.int64)),
    dict(target=torch.zeros(2, 4, 100)[..., ::2]), dict(target=torch.zeros(4, 2, 50).transpose(0, 1)), dict(draft_lens=_i32(3)),
])
def test_verification_shapes(host, wrong):
    a = dict(target=torch.zeros(2, 4, 50), draft=torch.zeros(2, 3, 50), tokens=_i32(2, 3), u=torch.zeros(2, 4),
             out_tokens=_i32(2, 4), accepted=_i32(2))
    _verify(a)
    _verify({**a, "draft": None})
    _verify({**a, "target": torch.zeros(2, 4, 64)[..., :50]})
    assert host[-1][1][1] == 64
    with pytest.raises(ValueError):
        _verify({**a, **wrong})
    assert len(host) == 3


def test_more_work_than_a_launch_can_name(lib):
    heads = 65535
    many = dict(shape=_shape(heads, heads), q_stride=heads * 128, num_reqs=1, batch=65535)
    assert lib.sfi_window_attn(*{**WINDOW, **many, "num_tokens": 257}.values()) == UNSUPPORTED
    assert lib.sfi_attn_mass(*{**MASS, **many}.values()) == UNSUPPORTED
    more = dict(shape=_shape(65536, 65536), q_stride=65536 * 128)
    assert lib.sfi_window_attn(*{**WINDOW, **more}.values()) == UNSUPPORTED
    assert lib.sfi_attn_mass(*{**MASS, **more}.values()) == UNSUPPORTED
    assert lib.sfi_kv_evict(*{**EVICT, "shape": _shape(65536, 65536)}.values()) == UNSUPPORTED
    assert lib.sfi_verify_tokens(*{**VERIFY, "batch": (1 << 24) + 1}.values()) == UNSUPPORTED
