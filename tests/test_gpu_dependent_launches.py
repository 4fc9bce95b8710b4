"""Chains of dependent launches across the bf16 and the 4-bit calls: a bf16 step that writes
its token, a call on the 4-bit cache, and a bf16 step that may read ahead of its wait."""
import pytest
import torch

from tests.gpu_harness import Problem
from tests.test_gpu_kv4 import Cache

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


@pytest.mark.parametrize("between", ["dense", "scores", "fast", "append", "read", "compact"])
def test_a_step_that_reads_ahead_sees_the_step_before_the_4bit_call(between):
    """SFI_ATTN_EARLY_KV_PREFETCH asks that the kernel directly before the call writes nothing of
    what it reads. The append two kernels before must have landed all the same: with the flag, bit
    for bit what the step gives without it, over many tokens in a row."""
    sfi = _sfi()
    prob = Problem(seed=5, lens=[9000, 300, 5000, 40], Hq=16, Hkv=8, D=128, S=4, W=32).to_device()
    B, L, reps = prob.B, int(prob.lens.max()) + 16, 24
    c = Cache(6, [70, 33], 2, 128)
    shape, G = sfi.AttnShape(4, 2, 128), 2
    comp = sfi.alloc_kv4_compact(shape, [20, 20])
    comp.count.fill_(16)
    idx = torch.arange(4, 20, dtype=torch.int32, device="cuda").expand(2, 2, 16).contiguous()
    g = torch.Generator().manual_seed(7)
    rand = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    tokens = [(rand(B, 8, 128), rand(B, 8, 128)) for _ in range(reps)]
    q, q4, new4 = rand(B, 16, 128), rand(2, 1, 2 * G, 128), (rand(2, 1, 2, 128), rand(2, 1, 2, 128))
    out4, read4 = torch.empty(2, 1, 2 * G, 128, device="cuda"), (rand(2, 8, 2, 128), rand(2, 8, 2, 128))
    scores4 = torch.empty(2, 2, 80, device="cuda")
    ws4 = sfi.alloc_kv4_workspace(shape, 2)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    sfi.sfi_kv4_compact_gather(shape, c.kv, idx, comp.count, 4, comp, dev_status=st)
    calls = {
        "dense": lambda: sfi.sfi_kv4_dense_attn(shape, c.kv, 4, 8, q4, out4, workspace=ws4, dev_status=st),
        "scores": lambda: sfi.sfi_kv4_dense_attn(shape, c.kv, 4, 8, q4, out4, scores=scores4, workspace=ws4, dev_status=st),
        "fast": lambda: sfi.sfi_kv4_fast_attn(shape, c.kv, comp, 4, 8, q4, out4, workspace=ws4, dev_status=st),
        "append": lambda: sfi.sfi_kv4_append(shape, c.kv, *new4, dev_status=st),
        "read": lambda: sfi.sfi_kv4_read(shape, c.kv, *read4, dev_status=st),
        "compact": lambda: sfi.sfi_kv4_compact_gather(shape, c.kv, idx, comp.count, 4, comp, dev_status=st),
    }
    ws = [sfi.alloc_workspace(prob.shape, B, L) for _ in range(2)]

    def run(flags):
        first = torch.empty(B, 16, 128, device="cuda")
        outs = [torch.full((B, 16, 128), float("nan"), device="cuda") for _ in range(reps)]
        for (k, v), out in zip(tokens, outs):
            sfi.sfi_slow_dense_attn_with_scores(prob.shape, prob.d_kv, 4, 32, prob.d_q, first, max_tokens=L, workspace=ws[0],
                                                dev_status=st, k_new=k, v_new=v)
            calls[between]()
            sfi.sfi_slow_dense_attn_with_scores(prob.shape, prob.d_kv, 4, 32, q, out, max_tokens=L, workspace=ws[1],
                                                dev_status=st, flags=flags)
        torch.cuda.synchronize()
        assert st.item() == 0
        return outs

    plain, ahead = run(0), run(sfi.SFI_ATTN_EARLY_KV_PREFETCH)
    assert not torch.equal(plain[0], plain[1])  # each token counts
    for a, b in zip(plain, ahead):
        assert torch.equal(a, b)
