"""Prompts, eviction by attention weight, drafts and their verification in one run, as a serving loop has them: two
layers over shared pages, every step against the host's fp64, eager and as captured graphs."""
import numpy as np
import pytest
import torch

from tests import window_reference as ref

pytestmark = pytest.mark.gpu

HQ, HKV, D, LAYERS, SINK, RECENT, K, T, V = 8, 2, 64, 2, 4, 24, 40, 3, 501
LENS = [150, 61, 230]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from sparse_kv_long_sfi_gb300 import build
    build.build()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Loop:
    """Device state of the requests, and what the host knows of it."""

    def __init__(self, seed):
        import sparse_kv_long_sfi_gb300 as sfi
        self.sfi, self.g = sfi, torch.Generator().manual_seed(seed)
        b, pages = len(LENS), 60
        self.shape = sfi.AttnShape(HQ, HKV, D)
        self.pools = [[torch.full((pages, HKV, 16, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
                      for _ in range(LAYERS)]
        self.map = sfi.PageMap(_i32(np.zeros((b, 20))), _i32([0] * b), _i32([0] * pages))
        self.kvs = [sfi.PagedKV(k, v, self.map.page_table, self.map.seq_lens) for k, v in self.pools]
        self.pp = sfi.PagePools([p for kv in self.pools for p in kv])
        self.ws = sfi.alloc_page_workspace(self.map)
        self.st = _i32([0])
        self.rows = [[[[] for _ in range(HKV)] for _ in range(b)] for _ in range(LAYERS)]  # (k, v) by slot

    def new(self, *dims):
        return torch.randn(*dims, generator=self.g).to(torch.bfloat16)

    def write(self, tokens, lens):
        """New K and V of every layer: the device's pages, and the host's lists."""
        b = len(LENS)
        for layer, kv in enumerate(self.kvs):
            q, k, v = self.new(b, tokens, HQ, D), self.new(b, tokens, HKV, D), self.new(b, tokens, HKV, D)
            out = torch.empty(b, tokens, HQ, D, dtype=torch.bfloat16, device="cuda")
            self.sfi.sfi_qk_norm_rope(self.shape, None, q.cuda(), k.cuda(), v.cuda(), out, new_lens=_i32(lens), kv=kv,
                                      dev_status=self.st)
            assert torch.equal(out[0, 0].cpu(), q[0, 0])
            for r, n in enumerate(lens):
                for t in range(n):
                    for h in range(HKV):
                        self.rows[layer][r][h].append((k[r, t, h], v[r, t, h]))
            yield layer, kv, q

    def cache(self, layer):
        """The host's rows as a Cache that the reference reads."""
        c = ref.Cache.__new__(ref.Cache)
        c.hq, c.hkv, c.d = HQ, HKV, D
        c.lens = [len(self.rows[layer][r][0]) for r in range(len(LENS))]
        c.k, c.v = 0, 1
        c.rows = lambda which, r, h: torch.stack([x[which] for x in self.rows[layer][r][h]]).double().numpy()
        return c


def _attended(loop, layer, q, out, lse, lens, tokens):
    c = loop.cache(layer)
    for r, n in enumerate(lens):
        for i in sorted({t for t in tokens if t < n} | {n - 1}):
            for h in range(HQ):
                o, x, _, mag, smag = ref.token(c, r, h, q[r, i, h], c.lens[r] - n + i, SINK, RECENT)
                assert (np.abs(out[r, i, h].double().cpu().numpy() - o) <= ref.out_bound(o, mag, D)).all(), (layer, r, i, h)
                assert abs(float(lse[r, i, h]) - x) <= ref.lse_bound(x, smag, D)


@pytest.mark.parametrize("captured", [False, True])
def test_prompt_evict_draft_verify(captured):
    loop = Loop(3)
    sfi, b, m, st = loop.sfi, len(LENS), loop.map, loop.st

    def run(fn):
        """Once eagerly, or captured and replayed."""
        if not captured:
            return fn()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fn()
        g.replay()

    # prompts
    sfi.sfi_page_reserve(m, loop.pp, _i32(LENS), workspace=loop.ws, dev_status=st)
    n = max(LENS)
    masses = [torch.full((b, HKV, 320), float("nan"), device="cuda") for _ in range(LAYERS)]
    spare = [torch.zeros_like(x) for x in masses]
    new_lens = _i32([0] * b)
    for layer, kv, q in loop.write(n, LENS):
        dq, out, lse = q.cuda(), torch.zeros(b, n, HQ, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(b, n, HQ, device="cuda")
        lens = _i32(LENS)

        def prompt():
            sfi.sfi_window_attn(loop.shape, kv, SINK, RECENT, dq, out, lse=lse, new_lens=lens, dev_status=st)
            # (every position is new: what the weights held does not count)
            sfi.sfi_attn_mass(loop.shape, kv, SINK, RECENT, dq, lse, masses[layer], new_lens=lens, dev_status=st)

        run(prompt)
        _attended(loop, layer, q, out, lse, LENS, (0, 5, 60, 100))
        for r, x in enumerate(LENS):
            assert abs(float(masses[layer][r, :, :x].double().sum()) / (x * HQ) - 1) < 1e-5
    # every layer cut to its own heaviest rows
    k_per_req = _i32([K, K, K])
    idx, count = torch.zeros(b, HKV, K, dtype=torch.int32, device="cuda"), _i32([0] * b)
    for layer, kv in enumerate(loop.kvs):
        run(lambda: sfi.sfi_kv_evict(loop.shape, kv, masses[layer], SINK, RECENT, k_per_req, idx, count, new_lens,
                                     mass_out=spare[layer], dev_status=st))
        for r, x in enumerate(LENS):
            for h in range(HKV):
                kept, _ = ref.keep(masses[layer][r, h].double().tolist(), x, SINK, RECENT, K)
                loop.rows[layer][r][h] = [loop.rows[layer][r][h][j] for j in kept]
                assert torch.equal(spare[layer][r, h, :len(kept)], masses[layer][r, h, kept])
    cut = [min(x, SINK + K + RECENT) for x in LENS]
    assert new_lens.tolist() == cut
    run(lambda: sfi.sfi_page_trim(m, new_lens, dev_status=st))
    assert m.seq_lens.tolist() == cut and int(m.ref_count.sum()) == sum(-(-x // 16) for x in cut)
    # drafts: room, K and V, attention over the evicted caches, weights on top of the kept ones
    sfi.sfi_page_reserve(m, loop.pp, _i32([x + T for x in cut]), workspace=loop.ws, dev_status=st)
    for layer, kv, q in loop.write(T, [T] * b):
        dq, out, lse = q.cuda(), torch.zeros(b, T, HQ, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(b, T, HQ, device="cuda")

        def draft():
            sfi.sfi_window_attn(loop.shape, kv, SINK, RECENT, dq, out, lse=lse, dev_status=st)
            sfi.sfi_attn_mass(loop.shape, kv, SINK, RECENT, dq, lse, spare[layer], decay=0.5, dev_status=st)

        run(draft)
        _attended(loop, layer, q, out, lse, [T] * b, range(T))
        assert torch.isfinite(spare[layer][0, :, :cut[0] + T]).all()
    # verification: the last token fed and T - 1 drafts gave T rows of the target
    target = torch.softmax(torch.randn(b, T, V, generator=loop.g) * 2, -1)
    q = torch.softmax(torch.log(target[:, :T - 1]) + torch.randn(b, T - 1, V, generator=loop.g) * 0.3, -1)
    tokens = torch.multinomial(q.view(-1, V), 1, generator=loop.g).view(b, T - 1).to(torch.int32)
    u = torch.rand(b, T, generator=loop.g)
    out_tokens, accepted = _i32(np.zeros((b, T))), _i32([0] * b)
    dt, dd, dx, du = target.cuda(), q.cuda(), tokens.cuda(), u.cuda()
    run(lambda: sfi.sfi_verify_tokens(dt, dd, dx, du, out_tokens, accepted, seq_lens=m.seq_lens, new_lens=new_lens, dev_status=st))
    want = [ref.verify(target[r].numpy(), q[r].numpy(), tokens[r].tolist(), u[r].numpy(), T - 1) for r in range(b)]
    assert accepted.tolist() == [a for a, _ in want]
    assert [out_tokens[r, a].item() for r, (a, _) in enumerate(want)] == [x for _, x in want]
    final = [x + T - (T - 1) + a for x, (a, _) in zip(cut, want)]
    assert new_lens.tolist() == final
    run(lambda: sfi.sfi_page_trim(m, new_lens, dev_status=st))
    assert m.seq_lens.tolist() == final and int(m.ref_count.sum()) == sum(-(-x // 16) for x in final)
    assert st.item() == 0
