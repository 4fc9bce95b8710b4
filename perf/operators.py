"""Cases of the cache-side operators: head norm + position rotation into the cache, the
cache held in 4 bits with its attention, and the page operators.

`run` computes a case with this repository's kernels when `own` is true, and otherwise
in its plain form: elementary torch operations in fp32 (angles in fp64), rounded once at
the end. `exact` computes the same in fp64 from the definitions, written apart.

The 4-bit cache. A token's K (and V) row of one head is quantised in groups of 16 values:
scale s = e4m3(min(amax / (6 g), 448)), codes e2m1(x / (s g)), both to nearest even; s = 0
gives zeros. g is a power of two per cache. The block of one (page of 16 tokens, KV head)
has 18 D bytes:
  [0, 8D)    K codes: byte token * D/2 + d/2, the even d in the low four bits
  [8D, 9D)   K scales: byte token * D/16 + d/16
  [9D, 17D)  V codes: for d = 64 a + 16 b + 8 c + 2 e + f and token = 4 t + 2 h + l the
             byte 512 a + 128 e + 32 t + 16 f + 4 b + 2 h + c, l = 0 in the low four bits
  [17D, 18D) V scales: byte t * D/4 + 4 * (d/16) + token % 4, t = token / 4
"""
import math

import torch

own = False

PAGE = 16
DEV = "cuda"
GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]  # the magnitudes of e2m1


# ---- cases ------------------------------------------------------------------------------------------------------
# Head layouts, sink, recent window and lengths are those of the repository's benchmark and tests (16/8/128, 32/8/128
# and 8/2/64 heads; sink 64 + recent 256 and sink 4 + recent 32; 16K, 32K and 4K-128K contexts), or generic.

def listed():
    return [
        # one decode step of the benchmark's batch: every request's newest token, into the bf16 pages
        dict(name="norm_rope_step_b16", op="norm_rope", batch=16, tokens=1, new_min=1, ctx=16384, hq=16, hkv=8, d=128,
             rot=128, axes=1, interleaved=False),
        # two prompts of 8K tokens, the whole chunk of one layer
        dict(name="norm_rope_prompt_2x8k", op="norm_rope", batch=2, tokens=8192, new_min=8192, ctx=0, hq=32, hkv=8,
             d=128, rot=128, axes=1, interleaved=False),
        # ragged chunks of image tokens (time, height, width), half of each head rotated in adjacent pairs
        dict(name="norm_rope_axes_ragged", op="norm_rope", batch=5, tokens=1001, new_min=77, ctx=333, hq=8, hkv=2, d=64,
             rot=32, axes=3, interleaved=True),
        # one decode step's tokens into the 4-bit pages, and read back
        dict(name="kv4_write_step_b16", op="kv4_write", batch=16, tokens=1, new_min=1, ctx=16384, hkv=8, d=128),
        # ragged prompt chunks into the 4-bit pages at unaligned positions, and read back
        dict(name="kv4_write_chunk_4x4k", op="kv4_write", batch=4, tokens=4096, new_min=1000, ctx=501, hkv=8, d=128),
        # the smallest decode attention: one request, 1000 tokens, small heads
        dict(name="kv4_dense_b1_1k", op="kv4_dense", batch=1, tokens=1, len_min=1000, len_max=1000, hq=8, hkv=2, d=64,
             sink=4, recent=32, scores=True),
        # the slow step of the benchmark's batch: dense attention with the Selector's scores
        dict(name="kv4_slow_b16_16k", op="kv4_dense", batch=16, tokens=1, len_min=16384, len_max=16384, hq=16, hkv=8,
             d=128, sink=64, recent=256, scores=True),
        # verification of 4 drafted tokens in a ragged batch
        dict(name="kv4_verify_ragged_t4", op="kv4_dense", batch=8, tokens=4, len_min=515, len_max=131072, hq=32, hkv=8,
             d=128, sink=64, recent=256, scores=False),
        # refresh (compaction) and one fast step at 6.25% retention of 16K
        dict(name="kv4_fast_b16_k704", op="kv4_fast", batch=16, tokens=1, len_min=16384, len_max=16384, k=704, hq=16,
             hkv=8, d=128, sink=64, recent=256),
        # the same at 32 requests of 32K with two drafted tokens
        dict(name="kv4_fast_b32_k1728_t2", op="kv4_fast", batch=32, tokens=2, len_min=30011, len_max=32768, k=1728,
             hq=32, hkv=8, d=128, sink=64, recent=256),
        # four branches of each of 16 requests: the old branches are freed, new ones forked and given room
        dict(name="pages_branch_16x4", op="pages_branch", batch=16, branches=4, len_min=200, len_max=1500, grow=1,
             pools=56, page_bytes=32768),
        # a fragmented cache: the live pages of 64 requests move to the front of 8 pools
        dict(name="pages_compact_64", op="pages_compact", batch=64, len_min=512, len_max=4096, pools=8,
             page_bytes=32768),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "kv4_write", "kv4_dense", "kv4_fast", "pages_branch", "pages_compact"])
    hq, hkv, d = rng.choice([(16, 8, 128), (32, 8, 128), (8, 2, 64), (8, 8, 64), (16, 2, 128), (4, 1, 128)])
    sink, recent = rng.choice([(64, 256), (4, 32), (0, 100), (17, 1)])
    if op == "norm_rope":
        b, t = _log(rng, 1, 32), _log(rng, 1, 4096)
        t = max(1, min(t, 16384 // b))
        rot = rng.choice([d, d // 2, 16, 48])
        return dict(op=op, batch=b, tokens=t, new_min=rng.randint(1, t), ctx=_log(rng, 1, 30000), hq=hq, hkv=hkv, d=d,
                    rot=rot, axes=rng.choice([1, 1, 2, 3]), interleaved=rng.random() < 0.5)
    if op == "kv4_write":
        b, t = _log(rng, 1, 32), _log(rng, 1, 4096)
        t = max(1, min(t, 16384 // b))
        return dict(op=op, batch=b, tokens=t, new_min=rng.randint(1, t), ctx=_log(rng, 1, 8000), hkv=hkv, d=d)
    tokens = rng.randint(1, 16 // (hq // hkv))
    if op == "kv4_dense":
        b, hi = _log(rng, 1, 64), _log(rng, 40, 60000)
        hi = max(40, min(hi, 250000 // b))
        return dict(op=op, batch=b, tokens=tokens, len_min=rng.randint(20, hi), len_max=hi, hq=hq, hkv=hkv, d=d,
                    sink=sink, recent=recent, scores=rng.random() < 0.5)
    if op == "kv4_fast":
        b, k = _log(rng, 1, 32), _log(rng, 1, 1700)
        lo = sink + recent + k + 20 + rng.randint(0, 2000)
        return dict(op=op, batch=b, tokens=tokens, len_min=lo, len_max=lo + rng.randint(0, 4000), k=k, hq=hq, hkv=hkv,
                    d=d, sink=sink, recent=recent)
    pools, page_bytes = rng.choice([(2, 8192), (8, 4608), (24, 18432), (16, 32768)])
    lo = _log(rng, 1, 1000)
    if op == "pages_branch":
        return dict(op=op, batch=_log(rng, 1, 48), branches=rng.randint(1, 5), len_min=lo, len_max=lo + _log(rng, 1, 2000),
                    grow=rng.randint(1, 40), pools=pools, page_bytes=page_bytes)
    return dict(op=op, batch=_log(rng, 1, 100), len_min=lo, len_max=lo + _log(rng, 1, 2000), pools=pools,
                page_bytes=page_bytes)


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, evenly over their logarithm, the largest first."""
    if n == 1 or lo == hi:
        return [hi] * n
    return [int(round(hi * (lo / hi) ** (i / (n - 1)))) for i in range(n)]


# ---- the 4-bit format in torch ----------------------------------------------------------------------------------

def _e4m3(code):
    return code.contiguous().view(torch.float8_e4m3fn).float()


def _quantise(x, g):
    """bf16 values [..., D] -> e2m1 codes [..., D] and e4m3 scale codes [..., D/16], uint8."""
    xg = x.float().unflatten(-1, (-1, 16))
    amax = xg.abs().amax(-1)
    fine = torch.isfinite(xg).all(-1)
    s8 = torch.where(fine, amax / (6.0 * g), torch.zeros_like(amax)).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = s8.float() * g
    y = torch.where((s > 0)[..., None], xg / s[..., None], torch.zeros_like(xg))
    a = y.abs()
    mag = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = torch.where(fine[..., None], mag + 8 * torch.signbit(y).to(torch.uint8), torch.zeros_like(mag))
    scale = torch.where(fine, s8.view(torch.uint8), torch.full_like(mag[..., 0], 0x7F))
    return code.flatten(-2), scale


def _pack(kc, ks, vc, vs):
    """Codes [n][16][H][D] and scales [n][16][H][D/16] of whole pages -> blocks [n][H][18 D]."""
    n, _, h, d = kc.shape
    kb = kc.permute(0, 2, 1, 3).unflatten(-1, (-1, 2))
    kb = (kb[..., 0] | kb[..., 1] << 4).reshape(n, h, 8 * d)
    ksb = ks.permute(0, 2, 1, 3).reshape(n, h, d)
    # d -> (a, b, c, e, f); token -> (t, h, l)
    v = vc.permute(0, 2, 3, 1).reshape(n, h, d // 64, 4, 2, 4, 2, 4, 2, 2)
    v = (v[..., 0] | v[..., 1] << 4)                                        # n h a b c e f t hh
    v = v.permute(0, 1, 2, 5, 7, 6, 3, 8, 4).reshape(n, h, 8 * d)           # a e t f b hh c
    vsb = vs.permute(0, 2, 1, 3).reshape(n, h, 4, 4, d // 16).transpose(-1, -2).reshape(n, h, d)
    return torch.cat([kb, ksb, v, vsb], -1).contiguous()


def _unpack(blocks, d):
    """Blocks [..., 18 D] -> K codes, K scales, V codes, V scales, each [..., 16][D or D/16], uint8."""
    lead = blocks.shape[:-1]
    kb, ksb, vb, vsb = blocks.split([8 * d, d, 8 * d, d], -1)
    kc = torch.stack([kb & 15, kb >> 4], -1).reshape(*lead, 16, d)
    ks = ksb.reshape(*lead, 16, d // 16)
    v = vb.reshape(-1, d // 64, 4, 4, 2, 4, 2, 2)                           # a e t f b hh c
    v = torch.stack([v & 15, v >> 4], -1)                                   # ... l
    v = v.permute(0, 3, 6, 8, 1, 5, 7, 2, 4).reshape(*lead, 16, d)          # t hh l | a b c e f
    vs = vsb.reshape(*lead, 4, d // 16, 4).transpose(-1, -2).reshape(*lead, 16, d // 16)
    return kc, ks, v, vs


def _values(code, scale, g):
    grid = torch.tensor(GRID + [-x for x in GRID], device=code.device)
    v = grid[code.int()].unflatten(-1, (-1, 16)) * (_e4m3(scale) * g)[..., None]
    return v.flatten(-2)


def _rows(state):
    """The cache's values by position: K, V fp32 [B][Hkv][max pages * 16][D]."""
    c = state["case"]
    kc, ks, vc, vs = _unpack(state["pool"][state["page_table"].long()], c["d"])   # [B][P][H][16][..]
    out = []
    for code, scale, g in ((kc, ks, state["k_scale"]), (vc, vs, state["v_scale"])):
        out.append(_values(code, scale, g).transpose(1, 2).flatten(2, 3))
    return out


# ---- inputs -----------------------------------------------------------------------------------------------------

def _gen(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000003 + sum(map(ord, case["op"])))
    h = torch.Generator()
    h.manual_seed(seed * 7919 + 11)
    return g, h


def _shuffled(values, h):
    return [values[i] for i in torch.randperm(len(values), generator=h).tolist()]


def _table(lens, h, spare=8):
    """A page table whose pages are scattered over a pool with a few spare pages."""
    need = [-(-n // PAGE) for n in lens]
    pages = sum(need) + spare
    ids = torch.randperm(pages, generator=h, dtype=torch.int64).to(torch.int32)
    table = torch.zeros(len(lens), max(need), dtype=torch.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = ids[at:at + n]
        at += n
    return table, pages


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).to(torch.bfloat16)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _outliers(g, heads, d):
    """Channel magnitudes of a cache: most near 1, a few channels several times larger."""
    m = torch.rand(heads, d, generator=g, device=DEV) * 0.5 + 0.5
    return torch.where(torch.rand(heads, d, generator=g, device=DEV) < 0.04, m * 6, m)


def _kv4_pool(g, pages, hkv, d, k_scale, v_scale):
    ko, vo = _outliers(g, hkv, d), _outliers(g, hkv, d)
    pool = torch.empty(pages, hkv, 18 * d, dtype=torch.uint8, device=DEV)
    for i in range(0, pages, 2048):
        n = min(2048, pages - i)
        k = (_normal(g, n, 16, hkv, d).float() * ko).to(torch.bfloat16)
        v = (_normal(g, n, 16, hkv, d).float() * vo).to(torch.bfloat16)
        pool[i:i + n] = _pack(*_quantise(k, k_scale), *_quantise(v, v_scale))
    return pool


def prepare(case, seed):
    g, h = _gen(case, seed)
    c, b = case, case["batch"]
    s = {"case": c}
    if c["op"] in ("norm_rope", "kv4_write"):
        t, hkv, d = c["tokens"], c["hkv"], c["d"]
        new = _shuffled(_spread(c["new_min"], t, b), h)
        lens = [c["ctx"] + n for n in new]
        table, pages = _table(lens, h)
        s.update(new_lens=_i32(new), seq_lens=_i32(lens), page_table=table.to(DEV))
        if c["op"] == "kv4_write":
            s["k_scale"], s["v_scale"] = 1.0, 0.5
            s["pool"] = torch.randint(0, 256, (pages, hkv, 18 * d), generator=g, device=DEV, dtype=torch.uint8)
            s["k_new"] = (_normal(g, b, t, hkv, d).float() * _outliers(g, hkv, d)).to(torch.bfloat16)
            s["v_new"] = _normal(g, b, t, hkv, d)
            s["first"] = s["seq_lens"] - s["new_lens"]
            s["k_out"], s["v_out"] = (torch.zeros(b, t, hkv, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
            return s
        hq, rot = c["hq"], min(c["rot"], d)
        qkv = _normal(g, b, t, (hq + 2 * hkv) * d)  # the projections' output, as one matrix product leaves it
        s["q"], s["k"], s["v"] = (x.unflatten(-1, (-1, d)) for x in qkv.split([hq * d, hkv * d, hkv * d], -1))
        s["q_weight"], s["k_weight"] = ((1 + 0.2 * _normal(g, d).float()).to(torch.bfloat16) for _ in range(2))
        s["inv_freq"] = 1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
        s["k_pool"], s["v_pool"] = _normal(g, pages, hkv, PAGE, d), _normal(g, pages, hkv, PAGE, d)
        s["q_out"] = torch.zeros(b, t, hq, d, dtype=torch.bfloat16, device=DEV)
        s["positions"] = s["axis"] = None
        if c["axes"] > 1:
            p = torch.randint(0, 1 + c["ctx"] + t, (c["axes"], b, t), generator=g, device=DEV, dtype=torch.int32)
            s["positions"] = p
            s["axis"] = (torch.arange(rot // 2, device=DEV) % c["axes"]).to(torch.uint8)
        return s
    if c["op"] in ("kv4_dense", "kv4_fast"):
        hkv, d, t = c["hkv"], c["d"], c["tokens"]
        lens = _shuffled(_spread(c["len_min"], c["len_max"], b), h)
        table, pages = _table(lens, h)
        s["k_scale"], s["v_scale"] = 2.0, 1.0
        s["pool"] = _kv4_pool(g, pages, hkv, d, s["k_scale"], s["v_scale"])
        s.update(seq_lens=_i32(lens), page_table=table.to(DEV))
        s["q"] = _normal(g, b, t, c["hq"], d)
        s["out"] = torch.zeros(b, t, c["hq"], d, device=DEV)
        s["lse"] = torch.zeros(b, t, c["hq"], device=DEV)
        if c["op"] == "kv4_dense":
            s["scores"] = torch.zeros(b, hkv, max(lens), device=DEV) if c["scores"] else None
            return s
        # a selection among the candidates, ascending, as the Selector leaves it (the last one drawn drops out)
        score = torch.rand(b, hkv, max(lens), generator=g, device=DEV)
        pos = torch.arange(max(lens), device=DEV)
        top = (s["seq_lens"].long() - t - c["recent"])[:, None, None]
        score = torch.where((pos >= c["sink"]) & (pos < top), score, torch.full_like(score, -1.0))
        s["idx"] = score.topk(c["k"], -1).indices.sort(-1).values.to(torch.int32)
        s["count"] = _i32(_shuffled(_spread(max(1, c["k"] // 2), c["k"], b), h))
        return s
    lens = _shuffled(_spread(c["len_min"], c["len_max"], b), h)
    if c["op"] == "pages_branch":
        kids = b * c["branches"]
        longest = max(lens) + c["grow"]
        table, used = _table(lens, h, spare=0)
        extra = sum(-(-(n + c["grow"]) // PAGE) - n // PAGE for n in lens) * c["branches"]
        pages = used + extra + 5
        where = torch.randperm(pages, generator=h)[:used].to(torch.int32)
        full = torch.zeros(b + kids, -(-longest // PAGE), dtype=torch.int32)
        full[:b, :table.shape[1]] = where[table.long()]
        parents = [i // c["branches"] for i in range(kids)]
        s["src"], s["dst"] = _i32(_shuffled(parents, h)), _i32(list(range(b, b + kids)))
        s["seq_lens"] = _i32(lens + [0] * kids)
        s["new_lens"] = s["seq_lens"][s["src"].long()] + c["grow"]
    else:
        table, used = _table(lens, h, spare=0)
        pages = 2 * used + 3
        where = torch.randperm(pages, generator=h)[:used].to(torch.int32)
        full = where[table.long()]
        s["seq_lens"] = _i32(lens)
    s["page_table"] = full.to(DEV)
    s["ref_count"] = torch.zeros(pages, dtype=torch.int32, device=DEV)
    s["ref_count"][where.to(DEV).long()] = 1
    s["pool"] = torch.randint(-20000, 20000, (c["pools"], pages, c["page_bytes"] // 2), generator=g, device=DEV,
                              dtype=torch.int16)
    if c["op"] == "pages_compact":
        s["table_out"] = torch.zeros_like(s["page_table"])
        s["ref_out"] = torch.zeros_like(s["ref_count"])
        s["live"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    return s


# ---- one pass ---------------------------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    return (_OWN if own else _PLAIN)[op](state)


def _plain_norm_rope(s):
    c = s["case"]
    b, t, d, rot = c["batch"], c["tokens"], c["d"], min(c["rot"], c["d"])
    step = torch.arange(t, device=DEV)
    valid = step[None] < s["new_lens"][:, None]
    slot = (s["seq_lens"] - s["new_lens"]).long()[:, None] + step
    if s["positions"] is None:
        pos = slot[..., None]
    else:
        pos = s["positions"][s["axis"].long()].permute(1, 2, 0)
    ang = pos.double() * s["inv_freq"].to(DEV)
    cos, sin = (f(ang).float()[:, :, None] for f in (torch.cos, torch.sin))

    def turn(x, w):
        x = x.float()
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
        r, rest = x[..., :rot], x[..., rot:]
        x0, x1 = (r[..., 0::2], r[..., 1::2]) if c["interleaved"] else r.chunk(2, -1)
        y0, y1 = x0 * cos - x1 * sin, x1 * cos + x0 * sin
        r = torch.stack([y0, y1], -1).flatten(-2) if c["interleaved"] else torch.cat([y0, y1], -1)
        return torch.cat([r, rest], -1).to(torch.bfloat16)

    s["q_out"].copy_(torch.where(valid[..., None, None], turn(s["q"], s["q_weight"]), s["q_out"]))
    k = turn(s["k"], s["k_weight"])
    r, j = valid.nonzero(as_tuple=True)
    page, off = s["page_table"][r, slot[r, j] // PAGE].long(), slot[r, j] % PAGE
    s["k_pool"][page, :, off] = k[r, j]
    s["v_pool"][page, :, off] = s["v"][r, j]
    return {"q": s["q_out"], "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def _own_norm_rope(s):
    import sparse_kv_long_sfi_gb300 as sfi
    c = s["case"]
    if "shape" not in s:  # kept by a user's program for all steps
        s["shape"] = sfi.AttnShape(c["hq"], c["hkv"], c["d"])
        s["rope"] = sfi.Rope(sfi.rope_turns(s["inv_freq"]), axis=s["axis"], num_axes=c["axes"],
                             interleaved=c["interleaved"])
        s["kv"] = sfi.PagedKV(s["k_pool"], s["v_pool"], s["page_table"], s["seq_lens"])
    sfi.sfi_qk_norm_rope(s["shape"], s["rope"], s["q"], s["k"], s["v"], s["q_out"], q_weight=s["q_weight"],
                         k_weight=s["k_weight"], eps=1e-6, positions=s["positions"], new_lens=s["new_lens"], kv=s["kv"])
    return {"q": s["q_out"], "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def _plain_kv4_write(s):
    c = s["case"]
    d, t = c["d"], c["tokens"]
    step = torch.arange(t, device=DEV)
    valid = step[None] < s["new_lens"][:, None]
    r, j = valid.nonzero(as_tuple=True)
    pos = s["first"].long()[r] + j
    page, off = s["page_table"][r, pos // PAGE].long(), pos % PAGE
    # whole pages are unpacked, their new rows replaced, and packed again
    ids, inv = torch.unique(page, return_inverse=True)
    kc, ks, vc, vs = (x.transpose(1, 2).contiguous() for x in _unpack(s["pool"][ids], d))
    kc[inv, off], ks[inv, off] = _quantise(s["k_new"][r, j], s["k_scale"])
    vc[inv, off], vs[inv, off] = _quantise(s["v_new"][r, j], s["v_scale"])
    s["pool"][ids] = _pack(kc, ks, vc, vs)
    # and read back
    kc, ks, vc, vs = (x.transpose(1, 2) for x in _unpack(s["pool"][ids], d))
    s["k_out"][r, j] = _values(kc[inv, off], ks[inv, off], s["k_scale"]).to(torch.bfloat16)
    s["v_out"][r, j] = _values(vc[inv, off], vs[inv, off], s["v_scale"]).to(torch.bfloat16)
    return {"k": s["k_out"], "v": s["v_out"]}


def _own_kv4(s):
    import sparse_kv_long_sfi_gb300 as sfi
    c = s["case"]
    if "shape" not in s:
        s["shape"] = sfi.AttnShape(c.get("hq", c["hkv"]), c["hkv"], c["d"])
        s["kv"] = sfi.PagedKV4(s["pool"], s["page_table"], s["seq_lens"], s["k_scale"], s["v_scale"])
        if c["op"] != "kv4_write":
            s["workspace"] = sfi.alloc_kv4_workspace(s["shape"], c["batch"], c["tokens"])
        if c["op"] == "kv4_fast":
            s["compact"] = sfi.alloc_kv4_compact(s["shape"], [c["sink"] + c["k"]] * c["batch"])
            s["compact"].count = s["count"]
    return sfi, c, s["shape"], s["kv"]


def _own_kv4_write(s):
    sfi, c, shape, kv = _own_kv4(s)
    sfi.sfi_kv4_append(shape, kv, s["k_new"], s["v_new"], new_lens=s["new_lens"])
    sfi.sfi_kv4_read(shape, kv, s["k_out"], s["v_out"], first=s["first"])
    return {"k": s["k_out"], "v": s["v_out"]}


def _attend(q, k, v, seen, scale):
    """q [B][T][Hkv][G][D], k/v [B][Hkv][N][D], seen [B][T][1 or Hkv][N] -> out, lse, logits [B][Hkv][T][G][N]."""
    x = torch.einsum("bthgd,bhnd->bhtgn", q, k) * scale
    see = seen.transpose(1, 2)[:, :, :, None]
    z = torch.where(see, x, torch.full_like(x, -math.inf))
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - m)
    n = p.sum(-1, keepdim=True)
    o = torch.einsum("bhtgn,bhnd->bthgd", p / n, v)
    return o.flatten(2, 3), (m + torch.log(n))[..., 0].permute(0, 2, 1, 3).flatten(2), x


def _plain_kv4_dense(s):
    c = s["case"]
    k, v = _rows(s)
    q = s["q"].float().unflatten(2, (c["hkv"], -1))
    n, t = k.shape[2], c["tokens"]
    pos = torch.arange(n, device=DEV)
    end = (s["seq_lens"].long()[:, None] - t + 1 + torch.arange(t, device=DEV))   # L_t
    seen = pos < end[:, :, None, None]                                            # [B][T][1][N]
    o, lse, x = _attend(q, k, v, seen, 1 / math.sqrt(c["d"]))
    s["out"].copy_(o)
    s["lse"].copy_(lse)
    if s["scores"] is not None:
        x = (x * seen.transpose(1, 2)[:, :, :, None]).sum((2, 3))[..., :s["scores"].shape[-1]]
        pos, length = pos[:x.shape[-1]], s["seq_lens"].long()[:, None, None]
        cand = (pos >= c["sink"]) & (pos < length - c["recent"])
        x = torch.where(cand, x, torch.full_like(x, -math.inf))
        s["scores"].copy_(torch.where(pos < length, x, s["scores"]))
    return {"out": s["out"], "lse": s["lse"], "scores": s["scores"]}


def _own_kv4_dense(s):
    sfi, c, shape, kv = _own_kv4(s)
    sfi.sfi_kv4_dense_attn(shape, kv, c["sink"], c["recent"], s["q"], s["out"], lse=s["lse"], scores=s["scores"],
                           workspace=s["workspace"])
    return {"out": s["out"], "lse": s["lse"], "scores": s["scores"]}


def _plain_kv4_fast(s):
    c = s["case"]
    t, sink, recent = c["tokens"], c["sink"], c["recent"]
    b, hkv = c["batch"], c["hkv"]
    length = s["seq_lens"].long()[:, None, None]
    # positions: sink | selected | the recent windows of all tokens
    w = torch.arange(recent + t, device=DEV)
    pos = torch.cat([torch.arange(sink, device=DEV).expand(b, hkv, -1), s["idx"].long(),
                     (length - t + 1 - recent + w).expand(b, hkv, -1)], -1)
    at = pos.clamp(min=0)
    # the values of the listed rows only
    pages = torch.gather(s["page_table"].long()[:, None].expand(-1, hkv, -1), 2,
                         (at // PAGE).clamp(max=s["page_table"].shape[1] - 1))
    blocks = s["pool"][pages, torch.arange(hkv, device=DEV)[:, None]]
    rows = (at % PAGE)[..., None, None]
    kc, ks, vc, vs = (torch.gather(x, 3, rows.expand(-1, -1, -1, 1, x.shape[-1]))[:, :, :, 0]
                      for x in _unpack(blocks, c["d"]))
    k, v = _values(kc, ks, s["k_scale"]), _values(vc, vs, s["v_scale"])
    end = (s["seq_lens"].long()[:, None] - t + 1 + torch.arange(t, device=DEV))[:, :, None, None]   # L_t
    slot = torch.arange(pos.shape[-1], device=DEV)
    part = pos[:, None]
    seen = torch.where(slot < sink, part < end,
                       torch.where(slot < sink + c["k"], slot - sink < s["count"].long()[:, None, None, None],
                                   (part >= sink) & (part >= end - recent) & (part < end)))
    o, lse, _ = _attend(s["q"].float().unflatten(2, (hkv, -1)), k, v, seen, 1 / math.sqrt(c["d"]))
    s["out"].copy_(o)
    s["lse"].copy_(lse)
    return {"out": s["out"], "lse": s["lse"]}


def _own_kv4_fast(s):
    sfi, c, shape, kv = _own_kv4(s)
    sfi.sfi_kv4_compact_gather(shape, kv, s["idx"], s["count"], c["sink"], s["compact"])
    sfi.sfi_kv4_fast_attn(shape, kv, s["compact"], c["sink"], c["recent"], s["q"], s["out"], lse=s["lse"],
                          workspace=s["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


def _pages_answer(s):
    return {"pool": s["pool"], "page_table": s["page_table"], "seq_lens": s["seq_lens"], "ref_count": s["ref_count"]}


def _plain_pages_branch(s):
    table, lens, ref, pool = s["page_table"], s["seq_lens"], s["ref_count"], s["pool"]
    src, dst = s["src"].long(), s["dst"].long()
    col = torch.arange(table.shape[1], device=DEV)

    def count(rows, sign):
        held = col < ((lens[rows] + PAGE - 1) // PAGE)[:, None]
        ids = table[rows][held].long()
        ref.index_add_(0, ids, torch.full_like(ids, sign, dtype=torch.int32))

    # free the old branches
    count(dst, -1)
    lens[dst] = 0
    # fork: the parents' rows, shared
    held = col < ((lens[src] + PAGE - 1) // PAGE)[:, None]
    table[dst] = torch.where(held, table[src], table[dst])
    lens[dst] = lens[src]
    count(dst, 1)
    # room for the branches' growth: a private last page (copied where others hold it), then fresh pages. Each branch's
    # parent keeps the shared page, so every branch with a part-filled last page gets a copy.
    old, new = lens[dst], s["new_lens"]
    have, full = (old + PAGE - 1) // PAGE, old // PAGE
    need = (new + PAGE - 1) // PAGE
    fresh = (col >= full[:, None]) & (col < need[:, None])
    row, at = fresh.nonzero(as_tuple=True)
    free = (ref == 0).nonzero()[:, 0][:row.numel()]
    was = table[dst[row], at].long()
    part = at < have[row]
    pool[:, free[part]] = pool[:, was[part]]
    ref.index_add_(0, was[part], torch.full_like(was[part], -1, dtype=torch.int32))
    ref[free] = 1
    table[dst[row], at] = free.to(torch.int32)
    lens[dst] = new
    return _pages_answer(s)


def _own_pages(s):
    import sparse_kv_long_sfi_gb300 as sfi
    if "map" not in s:
        s["map"] = sfi.PageMap(s["page_table"], s["seq_lens"], s["ref_count"])
        s["pools"] = sfi.PagePools(list(s["pool"]))
        s["workspace"] = sfi.alloc_page_workspace(s["map"])
    return sfi


def _own_pages_branch(s):
    sfi = _own_pages(s)
    sfi.sfi_page_free(s["map"], s["dst"])
    sfi.sfi_page_fork(s["map"], s["src"], s["dst"])
    sfi.sfi_page_reserve(s["map"], s["pools"], s["new_lens"], s["dst"], workspace=s["workspace"])
    return _pages_answer(s)


def _plain_pages_compact(s):
    table, ref, pool = s["page_table"], s["ref_count"], s["pool"]
    pages = ref.numel()
    ids = torch.arange(pages, device=DEV)
    live = ref > 0
    n = live.sum()
    move, hole = (live & (ids >= n)).nonzero()[:, 0], (~live & (ids < n)).nonzero()[:, 0]
    new = ids.clone()
    new[move] = hole
    pool[:, hole] = pool[:, move]
    s["ref_out"].copy_(ref)
    s["ref_out"][move] = 0
    s["ref_out"][hole] = ref[move]
    held = torch.arange(table.shape[1], device=DEV) < ((s["seq_lens"] + PAGE - 1) // PAGE)[:, None]
    s["table_out"].copy_(torch.where(held, new[table.long()].to(torch.int32), table))
    s["live"].copy_(n.to(torch.int32))
    return {"pool": pool, "table": s["table_out"], "ref_count": s["ref_out"], "live": s["live"]}


def _own_pages_compact(s):
    sfi = _own_pages(s)
    sfi.sfi_page_compact(s["map"], s["pools"], s["table_out"], s["ref_out"], s["live"], workspace=s["workspace"])
    return {"pool": s["pool"], "table": s["table_out"], "ref_count": s["ref_out"], "live": s["live"]}


_PLAIN = {"norm_rope": _plain_norm_rope, "kv4_write": _plain_kv4_write, "kv4_dense": _plain_kv4_dense,
          "kv4_fast": _plain_kv4_fast, "pages_branch": _plain_pages_branch, "pages_compact": _plain_pages_compact}
_OWN = {"norm_rope": _own_norm_rope, "kv4_write": _own_kv4_write, "kv4_dense": _own_kv4_dense,
        "kv4_fast": _own_kv4_fast, "pages_branch": _own_pages_branch, "pages_compact": _own_pages_compact}


# ---- what a pass cannot do without ------------------------------------------------------------------------------

def work(case):
    c, op = case, case["op"]
    if op in ("norm_rope", "kv4_write"):
        n = sum(_spread(c["new_min"], c["tokens"], c["batch"]))
        if op == "norm_rope":  # q, k and v rows read once and written once
            heads = c["hq"] + 2 * c["hkv"]
            return {"bytes": 4 * n * heads * c["d"], "flops": 8 * n * (c["hq"] + c["hkv"]) * c["d"]}
        # K and V rows in bf16, written in 4.5 bits, read back and written in bf16
        return {"bytes": n * c["hkv"] * 2 * c["d"] * (2 + 2 * 0.5625 + 2), "flops": 8 * n * c["hkv"] * c["d"]}
    lens = _spread(c["len_min"], c["len_max"], c["batch"])
    if op in ("kv4_dense", "kv4_fast"):
        b, t = c["batch"], c["tokens"]
        io = b * t * c["hq"] * (c["d"] * 6 + 4)
        row = 2 * c["d"] * 0.5625
        if op == "kv4_dense":
            rows = sum(lens)
            io += 4 * c["hkv"] * rows if c["scores"] else 0
        else:  # the selected rows are read and packed, then read again with the recent window
            count = sum(_spread(max(1, c["k"] // 2), c["k"], b))
            packed = count + b * c["sink"]
            rows = packed + b * (c["recent"] + t - 1)
            io += c["hkv"] * (packed * 2 * row + 4 * count)
        return {"bytes": io + rows * c["hkv"] * row, "flops": 4 * rows * t * c["hq"] * c["d"]}
    if op == "pages_branch":
        held = sum(-(-n // PAGE) for n in lens) * c["branches"]
        grown = sum(-(-(n + c["grow"]) // PAGE) - n // PAGE for n in lens) * c["branches"]
        moved = sum(n % PAGE > 0 for n in lens) * c["branches"]
        return {"bytes": 2 * moved * c["pools"] * c["page_bytes"] + 4 * (3 * held + 2 * grown), "flops": 0}
    # of 2 n + 3 pages, n of them in use anywhere: about half of those lie behind the first n
    used = sum(-(-n // PAGE) for n in lens)
    moved = used * (used + 3) // (2 * used + 3)
    return {"bytes": 2 * moved * c["pools"] * c["page_bytes"] + 4 * (2 * used + 2 * (2 * used + 3)), "flops": 0}


# ---- the definitions in 64 bits ---------------------------------------------------------------------------------

def _nearest_even(x, table):
    """Index of the nearest entry of an ascending table; halfway goes to the even index."""
    table = torch.tensor(table, dtype=torch.float64, device=DEV)
    mid = (table[1:] + table[:-1]) / 2
    lo, hi = torch.searchsorted(mid, x.contiguous()), torch.searchsorted(mid, x.contiguous(), right=True)
    return torch.where(lo == hi, lo, torch.where(lo % 2 == 0, lo, hi)), table


def _e4m3_table():
    return [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1]


def _exact_round_trip(x, g):
    x = x.double().unflatten(-1, (-1, 16))
    i, table = _nearest_even((x.abs().amax(-1) / 6 / g).clamp(max=448.0), _e4m3_table())
    s = (table[i] * g)[..., None]
    j, grid = _nearest_even(torch.where(s > 0, x.abs() / s, torch.zeros_like(x)).clamp(max=6.0), GRID)
    return (grid[j] * torch.sign(x) * s).flatten(-2)


def _offsets(d):
    """Byte, shift and scale byte of K[token][dim] and V[token][dim] in a block, by the format's own words."""
    tok, dim = torch.arange(16, device=DEV)[:, None], torch.arange(d, device=DEV)[None]
    k = tok * (d // 2) + dim // 2, (dim % 2 * 4).expand(16, d), 8 * d + tok * (d // 16) + dim // 16
    a, b, cc, e, f = dim // 64, dim // 16 % 4, dim // 8 % 2, dim // 2 % 4, dim % 2
    t, hh, low = tok // 4, tok // 2 % 2, tok % 2
    v = (9 * d + 512 * a + 128 * e + 32 * t + 16 * f + 4 * b + 2 * hh + cc, (low * 4).expand(16, d),
         17 * d + t * (d // 4) + 4 * (dim // 16) + tok % 4)
    return k, v


def _exact_rows(s, r):
    """K and V of request r in 64 bits, [Hkv][positions][D]."""
    d = s["case"]["d"]
    blocks = s["pool"][s["page_table"][r].long()]
    magnitudes = torch.tensor(GRID, dtype=torch.float64, device=DEV)
    scales = torch.tensor(_e4m3_table() + [math.nan], dtype=torch.float64, device=DEV)
    out = []
    for (byte, shift, at), g in zip(_offsets(d), (s["k_scale"], s["v_scale"])):
        code = blocks[..., byte] >> shift.to(torch.uint8) & 15
        x = magnitudes[(code & 7).long()] * scales[blocks[..., at].long()] * g
        out.append(torch.where(code >= 8, -x, x).transpose(0, 1).flatten(1, 2))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op == "norm_rope":
        t, rot = c["tokens"], min(c["rot"], c["d"])
        inv = s["inv_freq"].to(DEV)
        first = (s["seq_lens"] - s["new_lens"]).tolist()
        out = {n: s[m].double() for n, m in (("q", "q_out"), ("k_pool", "k_pool"), ("v_pool", "v_pool"))}
        for r, n in enumerate(s["new_lens"].tolist()):
            slot = first[r] + torch.arange(n, device=DEV)
            pos = slot[:, None] if s["positions"] is None else s["positions"][:, r, :n].T[:, s["axis"].long()]
            unit = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), pos.double() * inv)[:, None]

            def turned(x, w):
                x = x[r, :n].double()
                x = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w.double()
                h = x[..., :rot]
                h = h.unflatten(-1, (-1, 2)) if c["interleaved"] else h.unflatten(-1, (2, -1)).transpose(-1, -2)
                z = torch.view_as_real(torch.view_as_complex(h.contiguous()) * unit)
                h = z.flatten(-2) if c["interleaved"] else z.transpose(-1, -2).flatten(-2)
                return torch.cat([h, x[..., rot:]], -1)

            out["q"][r, :n] = turned(s["q"], s["q_weight"])
            page = s["page_table"][r, slot // PAGE].long()
            out["k_pool"][page, :, slot % PAGE] = turned(s["k"], s["k_weight"])
            out["v_pool"][page, :, slot % PAGE] = s["v"][r, :n].double()
        return out
    if op == "kv4_write":
        out = {}
        for name, x, g in (("k", s["k_new"], s["k_scale"]), ("v", s["v_new"], s["v_scale"])):
            held = torch.arange(c["tokens"], device=DEV) < s["new_lens"][:, None]
            out[name] = _exact_round_trip(x, g) * held[..., None, None]
        return out
    if op in ("kv4_dense", "kv4_fast"):
        t, sink, recent, hkv, d = c["tokens"], c["sink"], c["recent"], c["hkv"], c["d"]
        out = {"out": s["out"].double(), "lse": s["lse"].double()}
        if op == "kv4_dense":
            out["scores"] = None if s["scores"] is None else s["scores"].double()
        for r, length in enumerate(s["seq_lens"].tolist()):
            k, v = _exact_rows(s, r)
            at = torch.arange(length, device=DEV).expand(hkv, -1)
            if op == "kv4_fast":
                sel = s["idx"][r, :, :int(s["count"][r])].long()
                low = max(sink, length - t + 1 - recent)
                at = torch.cat([torch.arange(sink, device=DEV).expand(hkv, -1), sel,
                                torch.arange(low, length, device=DEV).expand(hkv, -1)], 1)
                sparse = torch.arange(at.shape[1], device=DEV)[None] < sink + sel.shape[1]
            total = 0
            for i in range(t):
                end = length - t + 1 + i
                q = s["q"][r, i].double().reshape(hkv, -1, d)
                x = q @ torch.gather(k, 1, at[..., None].expand(-1, -1, d)).transpose(1, 2) / math.sqrt(d)
                see = at < end
                if op == "kv4_fast":
                    see = see & (sparse | (at >= end - recent))
                z = x.masked_fill(~see[:, None], -math.inf)
                out["lse"][r, i] = torch.logsumexp(z, -1).flatten()
                out["out"][r, i] = (torch.softmax(z, -1) @ torch.gather(v, 1, at[..., None].expand(-1, -1, d))).flatten(0, 1)
                total = total + x.masked_fill(~see[:, None], 0).sum(1)
            if out.get("scores") is not None:
                out["scores"][r, :, :length] = -math.inf
                out["scores"][r, :, sink:max(sink, length - recent)] = total[:, sink:max(sink, length - recent)]
        return out
    table, lens, ref = s["page_table"].tolist(), s["seq_lens"].tolist(), s["ref_count"].tolist()
    pages, moves = len(ref), []
    if op == "pages_branch":
        for p, kid in zip(s["src"].tolist(), s["dst"].tolist()):  # the old branches hold nothing yet
            have = -(-lens[p] // PAGE)
            table[kid][:have], lens[kid] = table[p][:have], lens[p]
            for i in table[p][:have]:
                ref[i] += 1
        free = [i for i in range(pages) if ref[i] == 0]
        for kid, new in zip(s["dst"].tolist(), s["new_lens"].tolist()):
            for i in range(lens[kid] // PAGE, -(-new // PAGE)):
                page = free.pop(0)
                if i < -(-lens[kid] // PAGE):
                    moves.append((table[kid][i], page))
                    ref[table[kid][i]] -= 1
                table[kid][i], ref[page] = page, 1
            lens[kid] = new
        out = {"page_table": _i32(table), "seq_lens": _i32(lens), "ref_count": _i32(ref)}
    else:
        live = sum(x > 0 for x in ref)
        moves = list(zip([i for i in range(live, pages) if ref[i]], [i for i in range(live) if not ref[i]]))
        where = dict(moves)
        out = {"table": _i32([[where.get(p, p) if i < -(-n // PAGE) else p for i, p in enumerate(row)]
                              for row, n in zip(table, lens)]), "live": _i32([live])}
        for a, z in moves:
            ref[z], ref[a] = ref[a], 0
        out["ref_count"] = _i32(ref)
    pool = s["pool"].clone()
    if moves:
        a, z = torch.tensor(moves, device=DEV).T
        pool[:, z] = s["pool"][:, a]
    return {**out, "pool": pool}
