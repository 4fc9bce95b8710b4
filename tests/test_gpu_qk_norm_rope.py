"""sfi_qk_norm_rope against the formula in 64 bits: head layouts, rotated widths, split and
adjacent pairs, several position axes, far and negative positions, ragged and strided
inputs, request subsets, and what must stay untouched.

Tolerance: the result is rounded once to bf16, at most 2^-8 |y|. The fp32 work before it is
off by at most 2^-18 of the pair's length (a norm of up to 128 terms: 64 ulp at the very
worst, the angle's 2^-24 turns of the two sides, two products), so
|gpu - ref| <= 2^-8 |y| + 2^-17 r, r the length of the rotated pair (|y| unrotated)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

SENTINEL = 777.0  # no output of these inputs


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from sparse_kv_long_sfi_gb300 import build
    build.build()


def _sfi():
    import sparse_kv_long_sfi_gb300 as sfi
    return sfi


def _reference(x, w, pos, inv_freq, interleaved, eps):
    """x [N][heads][D] fp64, pos [N][pairs] -> y and the length of each value's pair."""
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    y, r = x.copy(), np.abs(x)
    h = len(inv_freq)
    if h:
        a = (pos.astype(np.float64) * inv_freq)[:, None]
        i, j = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if interleaved else (slice(0, h), slice(h, 2 * h))
        y[..., i] = x[..., i] * np.cos(a) - x[..., j] * np.sin(a)
        y[..., j] = x[..., j] * np.cos(a) + x[..., i] * np.sin(a)
        r[..., i] = r[..., j] = np.hypot(x[..., i], x[..., j])
    return y, r


def _close(got, ref, what):
    y, r = ref
    err = np.abs(got.double().cpu().numpy() - y)
    bound = 2.0 ** -8 * np.abs(y) + 2.0 ** -17 * r
    assert (err <= bound).all(), (what, (err - bound).max())


CASES = [
    # hq, hkv, d, rot, T, new_lens, ctx, interleaved, axes, weights, fused
    (16, 8, 128, 128, 1, [1] * 5, [0, 15, 16, 1000, 40000], False, 1, True, True),
    (16, 8, 128, 128, 37, [37, 1, 0, 20], [5, 0, 9, 31], False, 1, True, True),
    (8, 2, 64, 64, 9, [9, 4], [100, 3], True, 1, True, False),
    (8, 2, 64, 32, 9, [9, 4], [100, 3], False, 3, True, True),
    (4, 1, 128, 16, 3, [3], [14], True, 2, False, True),
    (1, 1, 64, 48, 5, [5, 5, 2], [0, 0, 0], False, 1, True, False),
    (32, 4, 128, 96, 2, [2, 1], [30, 64], True, 1, True, True),
    (8, 8, 64, 0, 4, [4], [2], False, 1, True, True),
    (24, 3, 128, 128, 300, [300, 211], [0, 77], False, 1, True, True),
]


@pytest.mark.parametrize("case", CASES)
def test_formula(case):
    sfi = _sfi()
    hq, hkv, d, rot, T, new, ctx, interleaved, axes, weights, fused = case
    B = len(new)
    g = torch.Generator().manual_seed(hq * 1000 + rot + T)
    lens = [c + n for c, n in zip(ctx, new)]
    maxp = max(1, max(-(-n // 16) for n in lens))
    npages = B * maxp + 3
    table = torch.randperm(npages, generator=g)[:B * maxp].view(B, maxp).to(torch.int32)
    if fused:
        x = torch.randn(B, T, (hq + 2 * hkv) * d + 8, generator=g).to(torch.bfloat16).cuda()
        q, k, v, _ = x.split([hq * d, hkv * d, hkv * d, 8], -1)
        q, k, v = (t.unflatten(-1, (-1, d)) for t in (q, k, v))
    else:
        q, k, v = (torch.randn(B, T, h, d, generator=g).to(torch.bfloat16).cuda() for h in (hq, hkv, hkv))
    qw, kw = ((torch.randn(d, generator=g) * 0.3 + 1).to(torch.bfloat16) for _ in range(2)) if weights else (None, None)
    inv = 1e6 ** (-np.arange(0, rot, 2, dtype=np.float64) / max(rot, 1))
    rope, pos, axis = None, None, None
    if rot:
        if axes > 1:
            pos = torch.randint(-50, 70000, (axes, B, T), generator=g, dtype=torch.int32)
            axis = torch.arange(rot // 2) % axes
        rope = sfi.Rope(sfi.rope_turns(inv), axis=None if axis is None else axis.to(torch.uint8).cuda(), num_axes=axes,
                        interleaved=interleaved)
    kp = torch.full((npages, hkv, 16, d), SENTINEL, dtype=torch.bfloat16, device="cuda")
    vp = torch.full_like(kp, SENTINEL)
    kv = sfi.PagedKV(kp, vp, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"))
    qo = torch.full((B, T, hq, d), SENTINEL, dtype=torch.bfloat16, device="cuda")
    ko = torch.full((B, T, hkv, d), SENTINEL, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    sfi.sfi_qk_norm_rope(sfi.AttnShape(hq, hkv, d), rope, q, k, v, qo, q_weight=None if qw is None else qw.cuda(),
                         k_weight=None if kw is None else kw.cuda(), eps=1e-5,
                         positions=None if pos is None else pos.cuda(),
                         new_lens=torch.tensor(new, dtype=torch.int32, device="cuda"), k_out=ko, kv=kv, dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    touched = torch.zeros(npages, 16, dtype=torch.bool)
    for r in range(B):
        n = new[r]
        assert (qo[r, n:] == SENTINEL).all() and (ko[r, n:] == SENTINEL).all()
        if n == 0:
            continue
        slot = ctx[r] + np.arange(n)
        if pos is None:
            p = np.repeat(slot[:, None], max(rot // 2, 1), 1)[:, :rot // 2]
        else:
            p = pos[:, r, :n].numpy()[axis.numpy()].T
        f = lambda t: t[r, :n].double().cpu().numpy()  # noqa: E731
        w = lambda t: None if t is None else t.double().numpy()  # noqa: E731
        _close(qo[r, :n], _reference(f(q), w(qw), p, inv, interleaved, 1e-5), f"q of request {r}")
        kref = _reference(f(k), w(kw), p, inv, interleaved, 1e-5)
        _close(ko[r, :n], kref, f"k of request {r}")
        page, off = table[r, slot // 16].long(), torch.from_numpy(slot % 16)
        touched[page, off] = True
        assert torch.equal(kp.cpu()[page, :, off], ko[r, :n].cpu()), "the pages hold what k_out holds"
        assert torch.equal(vp.cpu()[page, :, off], v[r, :n].cpu())
    rest = ~touched[:, None, :, None].expand(npages, hkv, 16, d)
    assert (kp.cpu()[rest] == SENTINEL).all() and (vp.cpu()[rest] == SENTINEL).all()


def test_far_positions_keep_the_angle():
    """At positions near 2^31 the angle of every pair is that of exact arithmetic."""
    from fractions import Fraction
    sfi = _sfi()
    d, pos = 64, [2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, 987654321]
    inv = [float(1e4 ** (-i / 32)) for i in range(32)]
    two_pi = Fraction(62831853071795864769252867665590057683943, 10 ** 40)
    q = torch.zeros(1, len(pos), 1, d, dtype=torch.bfloat16, device="cuda")
    q[..., :32] = 1.0
    qo, ko = torch.empty_like(q), torch.empty_like(q)
    sfi.sfi_qk_norm_rope(sfi.AttnShape(1, 1, d), sfi.Rope(sfi.rope_turns(inv)), q, q.clone(), None, qo, k_out=ko,
                         positions=torch.tensor([pos], dtype=torch.int32, device="cuda"))
    for t, p in enumerate(pos):
        for i, f in enumerate(inv):
            turn = Fraction(f) * p / two_pi
            a = 2 * np.pi * float(turn - turn.__floor__())
            for got, ref in ((qo[0, t, 0, i], np.cos(a)), (qo[0, t, 0, 32 + i], np.sin(a))):
                assert abs(float(got) - ref) <= 2.0 ** -8 * abs(ref) + 2.0 ** -17, (p, i)


def test_request_subset_side_stream_and_graph():
    """req_ids picks requests, the rest keeps its contents; the call runs on the given stream
    and replays from a captured graph on new inputs."""
    sfi = _sfi()
    hq, hkv, d, T = 8, 2, 64, 3
    shape = sfi.AttnShape(hq, hkv, d)
    g = torch.Generator().manual_seed(5)
    x = torch.randn(4, T, hq + hkv, d, generator=g).to(torch.bfloat16).cuda()
    inv = [float(1e4 ** (-i / 32)) for i in range(32)]
    rope = sfi.Rope(sfi.rope_turns(inv))
    pos = torch.randint(0, 9999, (4, T), generator=g, dtype=torch.int32).cuda()
    ids = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    full_q = torch.empty(4, T, hq, d, dtype=torch.bfloat16, device="cuda")
    full_k = torch.empty(4, T, hkv, d, dtype=torch.bfloat16, device="cuda")
    q, k = x[:, :, :hq], x[:, :, hq:]
    sfi.sfi_qk_norm_rope(shape, rope, q, k, None, full_q, k_out=full_k, positions=pos)
    qo, ko = torch.full_like(full_q, SENTINEL), torch.full_like(full_k, SENTINEL)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    sfi.sfi_qk_norm_rope(shape, rope, q, k, None, qo, k_out=ko, positions=pos, req_ids=ids, stream=side)
    side.synchronize()
    for r in range(4):
        if r in (1, 3):
            assert torch.equal(qo[r], full_q[r]) and torch.equal(ko[r], full_k[r])
        else:
            assert (qo[r] == SENTINEL).all() and (ko[r] == SENTINEL).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sfi.sfi_qk_norm_rope(shape, rope, q, k, None, qo, k_out=ko, positions=pos)
    x.copy_(torch.randn(4, T, hq + hkv, d, generator=g).to(torch.bfloat16))
    graph.replay()
    torch.cuda.synchronize()
    sfi.sfi_qk_norm_rope(shape, rope, q, k, None, full_q, k_out=full_k, positions=pos)
    assert torch.equal(qo, full_q) and torch.equal(ko, full_k)


def test_device_errors_skip_what_they_concern():
    from sparse_kv_long_sfi_gb300 import _abi
    sfi = _sfi()
    shape = sfi.AttnShape(2, 1, 64)
    new, lens = [2, 3, -1, 2, 2], [1, 40, 5, 70, 18]  # L < n; n > T; n < 0; past the table; a bad page
    B, T, maxp = 5, 2, 4
    table = torch.arange(B * maxp, dtype=torch.int32).view(B, maxp).cuda()
    table[4, 1] = 99
    x = torch.ones(B, T, 2, 64, dtype=torch.bfloat16, device="cuda")
    y = torch.ones(B, T, 1, 64, dtype=torch.bfloat16, device="cuda")
    kp = torch.full((B * maxp, 1, 16, 64), SENTINEL, dtype=torch.bfloat16, device="cuda")
    vp = kp.clone()
    kv = sfi.PagedKV(kp, vp, table, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    qo = torch.full_like(x, SENTINEL)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    rope = sfi.Rope(sfi.rope_turns([1.0] * 32), axis=torch.zeros(32, dtype=torch.uint8, device="cuda"))
    sfi.sfi_qk_norm_rope(shape, rope, x, y, y, qo, kv=kv, dev_status=st,
                         new_lens=torch.tensor(new, dtype=torch.int32, device="cuda"))
    assert st.item() == _abi.SFI_DEV_BAD_LEN | _abi.SFI_DEV_BAD_PAGE
    assert (qo[:4] == SENTINEL).all() and (qo[4] != SENTINEL).all()
    assert (kp == SENTINEL).all() and (vp == SENTINEL).all()
    st.zero_()
    rope.axis[3] = 1
    sfi.sfi_qk_norm_rope(shape, rope, x[4:], y[4:], y[4:], qo[4:], k_out=torch.empty_like(y[4:]), dev_status=st,
                         positions=torch.ones(1, T, dtype=torch.int32, device="cuda"))
    assert st.item() == _abi.SFI_DEV_BAD_INDEX
    assert (qo[4, :, :, 3] == 1).all() and (qo[4, :, :, 2] != 1).all()
