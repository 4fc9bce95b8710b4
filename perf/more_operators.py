"""Cases of the operators around a cache that is written by prompts, cut back and drafted on: attention with a sliding
window and sinks (prompts and single steps), accumulated attention weights, eviction by them, verification of drafted
tokens, and the pages of a speculative step.

`run` computes a case with this repository's kernels when `own` is true, and otherwise in its plain form: elementary
torch operations in fp32 (sums of probabilities and their comparisons in fp64), rounded once at the end. `exact` computes
the same in fp64 from the definitions, written apart.

Definitions. Request r has L_r cached tokens, the last n_r of them new (their queries are given); new token t is at
position p = L_r - n_r + t and sees j <= p with j < S or j > p - W (sink S, recent window W; W >= L is causal attention).
  window  out = sum_j exp(x_j - lse) v_j, x_j = q . k_j / sqrt(D), lse = log sum_j exp(x_j)
  mass    mass[h][j] = decay * mass[h][j] (0 for the new positions) + sum over the tokens that see j and the query heads of
          KV head h of exp(x_j - lse)
  evict   keep [0, S), [L - W, L) and the k_r candidates between with the largest mass (equal ones: the lower position); the
          kept rows of K and V move to the front in their order, the mass into a second buffer
  verify  draft x_t is accepted while u_t q_t(x_t) < p_t(x_t); after a accepted drafts the next token is the first i with
          w_0 + ... + w_i > u_T sum(w), where w = max(p_a - q_a, 0) (p_a when all are accepted, or when that is 0 everywhere)
  pages   room for a step's drafts is reserved (free pages, lowest id first), then the requests are cut to what was accepted
"""
import math

import torch

own = False

PAGE = 16
DEV = "cuda"


# ---- cases ------------------------------------------------------------------------------------------------------
# Head layouts, sink and recent window are those of the repository's benchmark and tests (16/8/128, 32/8/128 and 8/2/64
# heads; sink 64 + recent 256 and sink 4 + recent 32), the contexts too (4K to 128K); vocabularies are generic.

def listed():
    return [
        # one decode step of the benchmark's batch with its window and sinks, read in place from the pages
        dict(name="window_step_b16", op="window", batch=16, tokens=1, new_min=1, ctx_min=16383, ctx_max=16383, hq=16,
             hkv=8, d=128, sink=64, recent=256),
        # one decode step with a wide window, ragged lengths
        dict(name="window_step_b32_w4k", op="window", batch=32, tokens=1, new_min=1, ctx_min=5001, ctx_max=30011, hq=32,
             hkv=8, d=128, sink=64, recent=4096),
        # two prompts of 8K tokens through a window of 1024
        dict(name="window_prompt_2x8k_w1k", op="window", batch=2, tokens=8192, new_min=8192, ctx_min=0, ctx_max=0, hq=16,
             hkv=8, d=128, sink=64, recent=1024),
        # ragged chunks of prompts behind cached context, causal (the window is longer than any request)
        dict(name="window_chunk_ragged_causal", op="window", batch=4, tokens=2048, new_min=501, ctx_min=333, ctx_max=6001,
             hq=32, hkv=8, d=128, sink=0, recent=1 << 20),
        # the weights that the last 64 tokens of 16K prompts give to the whole prompt
        dict(name="mass_last64_b8_16k", op="mass", batch=8, tokens=64, new_min=64, ctx_min=16320, ctx_max=16320, hq=16,
             hkv=8, d=128, sink=0, recent=1 << 20, decay=1.0),
        # a whole prompt of 8K tokens, every token's weights
        dict(name="mass_prompt_8k", op="mass", batch=1, tokens=8192, new_min=8192, ctx_min=0, ctx_max=0, hq=16, hkv=8,
             d=128, sink=0, recent=1 << 20, decay=1.0),
        # caches held at 2048 rows that have grown by 64
        dict(name="evict_b16_2112_to_2048", op="evict", batch=16, len_min=2112, len_max=2112, k_min=1728, k_max=1728,
             hkv=8, d=128, sink=64, recent=256),
        # prompts of up to 16K cut to about a thousand rows
        dict(name="evict_prompts_b8_16k", op="evict", batch=8, len_min=7001, len_max=16384, k_min=704, k_max=1024, hkv=8,
             d=128, sink=64, recent=256),
        # one request, four drafts, a small vocabulary
        dict(name="verify_b1_t4", op="verify", batch=1, drafts=4, vocab=32000, greedy=False),
        # a batch with seven drafts each and a large vocabulary
        dict(name="verify_b64_t7", op="verify", batch=64, drafts=7, vocab=150001, greedy=False),
        # a step's pages for a small batch, and for a large one with long requests and long drafts
        dict(name="pages_step_b16", op="pages", batch=16, len_min=3000, len_max=5000, grow=8, spare=100),
        dict(name="pages_step_b512", op="pages", batch=512, len_min=500, len_max=30000, grow=64, spare=5000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["window", "window", "window", "mass", "mass", "evict", "verify", "pages"])
    hq, hkv, d = rng.choice([(16, 8, 128), (32, 8, 128), (8, 2, 64), (8, 8, 64), (16, 2, 128), (4, 1, 128)])
    sink, recent = rng.choice([(64, 256), (4, 32), (0, 100), (17, 1), (64, 1024), (33, 4000), (0, 1 << 20)])
    if op in ("window", "mass"):
        b, t = _log(rng, 1, 32), _log(rng, 1, 4096)
        t = max(1, min(t, 8192 // b))
        ctx = _log(rng, 1, 30000)
        ctx = max(1, min(ctx, 200000 // b, (1 << 25) // (b * t)))
        c = dict(op=op, batch=b, tokens=t, new_min=rng.randint(1, t), ctx_min=rng.randint(0, ctx), ctx_max=ctx, hq=hq,
                 hkv=hkv, d=d, sink=sink, recent=recent)
        return dict(c, decay=rng.choice([1.0, 0.5])) if op == "mass" else c
    if op == "evict":
        hi = _log(rng, 40, 16000)
        b = max(1, min(_log(rng, 1, 32), 130000 // hi))
        k = _log(rng, 1, 2000)
        return dict(op=op, batch=b, len_min=rng.randint(20, hi), len_max=hi, k_min=rng.randint(0, k), k_max=k, hkv=hkv,
                    d=d, sink=sink, recent=min(recent, 1024))
    if op == "verify":
        return dict(op=op, batch=_log(rng, 1, 64), drafts=rng.randint(1, 7), vocab=_log(rng, 300, 150000),
                    greedy=rng.random() < 0.3)
    lo = _log(rng, 1, 10000)
    return dict(op=op, batch=_log(rng, 1, 500), len_min=lo, len_max=lo + _log(rng, 1, 15000), grow=rng.randint(1, 64),
                spare=rng.randint(0, 3000))


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, evenly over their logarithm, the largest first."""
    if n == 1 or lo == hi:
        return [hi] * n
    return [int(round((hi + 1) * ((lo + 1) / (hi + 1)) ** (i / (n - 1)))) - 1 for i in range(n)]


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


def _keys(g, pages, hkv, d):
    """Keys as a model leaves them: a few channels several times larger than the others."""
    m = torch.rand(hkv, 1, d, generator=g, device=DEV) * 0.5 + 0.5
    m = torch.where(torch.rand(hkv, 1, d, generator=g, device=DEV) < 0.04, m * 3, m)
    return (torch.randn(pages, hkv, PAGE, d, generator=g, device=DEV) * m).to(torch.bfloat16)


def prepare(case, seed):
    g, h = _gen(case, seed)
    c, b = case, case["batch"]
    s = {"case": c}
    if c["op"] in ("window", "mass"):
        t, hq, hkv, d = c["tokens"], c["hq"], c["hkv"], c["d"]
        each = _shuffled(list(zip(_spread(c["new_min"], t, b), _spread(c["ctx_min"], c["ctx_max"], b))), h)
        new, lens = [n for n, _ in each], [n + x for n, x in each]
        table, pages = _table(lens, h)
        s.update(new_lens=_i32(new), seq_lens=_i32(lens), page_table=table.to(DEV), max_len=max(lens))
        s["k_pool"], s["v_pool"] = _keys(g, pages, hkv, d), _normal(g, pages, hkv, PAGE, d)
        s["q"] = _normal(g, b, t, hq, d)
        if c["op"] == "window":
            s["out"] = torch.zeros(b, t, hq, d, dtype=torch.bfloat16, device=DEV)
            s["lse"] = torch.zeros(b, t, hq, device=DEV)
            return s
        s["mass"] = torch.rand(b, hkv, max(lens), generator=g, device=DEV)
        # the log-sum-exps that the attention of the same tokens left behind
        lse = torch.zeros(b, t, hq, device=DEV)
        for r in range(b):
            k = s["k_pool"][s["page_table"][r].long()].transpose(0, 1).flatten(1, 2)[:, :lens[r]]
            see = _seen(s["new_lens"][r:r + 1], s["seq_lens"][r:r + 1], torch.arange(lens[r], device=DEV)[None], c)[0]
            for i in range(hkv):
                x = torch.einsum("tgd,nd->gtn", s["q"][r].unflatten(1, (hkv, -1))[:, i].float(), k[i].float())
                x = (x / math.sqrt(d)).masked_fill_(~see, -math.inf)
                lse[r].unflatten(1, (hkv, -1))[:, i] = torch.logsumexp(x, -1).T
        s["lse"] = torch.where(torch.isfinite(lse), lse, torch.zeros_like(lse))
        return s
    if c["op"] == "evict":
        hkv, d = c["hkv"], c["d"]
        lens = _shuffled(_spread(c["len_min"], c["len_max"], b), h)
        table, pages = _table(lens, h)
        s.update(seq_lens=_i32(lens), page_table=table.to(DEV), max_len=max(lens))
        s["k_pool"], s["v_pool"] = _keys(g, pages, hkv, d), _normal(g, pages, hkv, PAGE, d)
        s["k_per_req"] = _i32(_shuffled(_spread(c["k_min"], c["k_max"], b), h))
        # a few heavy positions among many light ones, and some of equal weight
        s["mass"] = torch.rand(b, hkv, max(lens), generator=g, device=DEV).pow(6).mul(4096).ceil().div(64)
        s["idx"] = torch.zeros(b, hkv, max(1, c["k_max"]), dtype=torch.int32, device=DEV)
        s["count"], s["new_lens"] = (torch.zeros(b, dtype=torch.int32, device=DEV) for _ in range(2))
        s["mass_out"] = torch.zeros_like(s["mass"])
        return s
    if c["op"] == "verify":
        t, v = c["drafts"], c["vocab"]
        logits = torch.randn(b, t + 1, v, generator=g, device=DEV) * 2.5
        s["target"] = torch.softmax(logits, -1)
        # the drafting pass is near the target, not equal to it
        s["draft"] = torch.softmax(logits[:, :t] + torch.randn(b, t, v, generator=g, device=DEV) * 0.4, -1)
        pick = s["draft"].cumsum(-1).contiguous()
        x = torch.rand(b, t, 1, generator=g, device=DEV) * pick[..., -1:]
        s["tokens"] = torch.searchsorted(pick, x)[..., 0].clamp(max=v - 1).to(torch.int32)
        if c["greedy"]:
            s["draft"], s["tokens"] = None, s["target"][:, :t].argmax(-1).to(torch.int32)
        s["draft_lens"] = _i32(_shuffled(_spread(max(1, t // 2), t, b), h))
        s["u"] = torch.rand(b, t + 1, generator=g, device=DEV)
        s["out_tokens"] = torch.zeros(b, t + 1, dtype=torch.int32, device=DEV)
        s["accepted"] = torch.zeros(b, dtype=torch.int32, device=DEV)
        return s
    lens = _shuffled(_spread(c["len_min"], c["len_max"], b), h)
    table, used = _table(lens, h, spare=0)
    pages = used + sum(-(-(n + c["grow"]) // PAGE) - -(-n // PAGE) for n in lens) + c["spare"]
    where = torch.randperm(pages, generator=h)[:used].to(torch.int32)
    full = torch.zeros(b, -(-(max(lens) + c["grow"]) // PAGE), dtype=torch.int32)
    full[:, :table.shape[1]] = where[table.long()]
    s["page_table"], s["seq_lens"] = full.to(DEV), _i32(lens)
    s["grown"], s["kept"] = s["seq_lens"] + c["grow"], s["seq_lens"].clone()
    s["ref_count"] = torch.zeros(pages, dtype=torch.int32, device=DEV)
    s["ref_count"][where.to(DEV).long()] = 1
    return s


# ---- one pass ---------------------------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    return (_OWN if own else _PLAIN)[op](state)


def _seen(new_lens, seq_lens, pos, c):
    """Whether token t of request r sees position pos[r][i]: [B][T][N]."""
    p = (seq_lens - new_lens).long()[:, None, None] + torch.arange(c["tokens"], device=DEV)[:, None]
    pos = pos[:, None]
    held = torch.arange(c["tokens"], device=DEV)[:, None] < new_lens[:, None, None]
    return held & (pos <= p) & ((pos < c["sink"]) | (pos > p - c["recent"]))


def _rows(s, pool, pos):
    """Rows at positions pos [B][N] in fp32: [B][Hkv][N][D]."""
    page = torch.gather(s["page_table"].long(), 1, (pos // PAGE).clamp(max=s["page_table"].shape[1] - 1))
    return pool[page, :, pos % PAGE].float().transpose(1, 2)


def _positions(s):
    """The positions that any token of a request sees, [B][N] (some twice, some behind the end)."""
    c, b = s["case"], s["case"]["batch"]
    n = c["sink"] + c["recent"] + c["tokens"] - 1
    if n >= s["max_len"]:
        return torch.arange(s["max_len"], device=DEV).expand(b, -1)
    first = ((s["seq_lens"] - s["new_lens"]).long()[:, None] + 1 - c["recent"]).clamp(min=c["sink"])
    window = first + torch.arange(c["recent"] + c["tokens"] - 1, device=DEV)
    return torch.cat([torch.arange(c["sink"], device=DEV).expand(b, -1), window], 1)


def _logits(s, pos):
    c = s["case"]
    q = s["q"].float().unflatten(2, (c["hkv"], -1))
    return torch.einsum("bthgd,bhnd->bhgtn", q, _rows(s, s["k_pool"], pos)) / math.sqrt(c["d"])


def _plain_window(s):
    c = s["case"]
    pos = _positions(s)
    see = _seen(s["new_lens"], s["seq_lens"], pos, c)
    x = _logits(s, pos).masked_fill_(~see[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    x = x.sub_(m).exp_()
    n = x.sum(-1, keepdim=True)
    o = torch.einsum("bhgtn,bhnd->bhgtd", x, _rows(s, s["v_pool"], pos)) / n
    o, lse = o.permute(0, 3, 1, 2, 4).flatten(2, 3), (m + torch.log(n))[..., 0].permute(0, 3, 1, 2).flatten(2)
    held = torch.arange(c["tokens"], device=DEV) < s["new_lens"][:, None]
    s["out"].copy_(torch.where(held[..., None, None], o.to(torch.bfloat16), s["out"]))
    s["lse"].copy_(torch.where(held[..., None], lse, s["lse"]))
    return {"out": s["out"], "lse": s["lse"]}


def _own_attention(s):
    import sparse_kv_long_sfi_gb300 as sfi
    c = s["case"]
    if "shape" not in s:  # kept by a user's program for all steps
        s["shape"] = sfi.AttnShape(c.get("hq", c["hkv"]), c["hkv"], c["d"])
        s["kv"] = sfi.PagedKV(s["k_pool"], s["v_pool"], s["page_table"], s["seq_lens"])
    return sfi, c, s["shape"], s["kv"]


def _own_window(s):
    sfi, c, shape, kv = _own_attention(s)
    sfi.sfi_window_attn(shape, kv, c["sink"], c["recent"], s["q"], s["out"], lse=s["lse"], new_lens=s["new_lens"])
    return {"out": s["out"], "lse": s["lse"]}


def _plain_mass(s):
    c = s["case"]
    pos = torch.arange(s["max_len"], device=DEV).expand(c["batch"], -1)
    see = _seen(s["new_lens"], s["seq_lens"], pos, c)
    lse = s["lse"].unflatten(2, (c["hkv"], -1)).permute(0, 2, 3, 1)[..., None]
    x = _logits(s, pos).sub_(lse).exp_().masked_fill_(~see[:, None, None], 0.0).sum((2, 3))
    length = s["seq_lens"].long()[:, None, None]
    old = torch.where(pos[:, None] < length - s["new_lens"].long()[:, None, None], s["mass"] * c["decay"],
                      torch.zeros_like(x))
    s["mass"].copy_(torch.where(pos[:, None] < length, old + x, s["mass"]))
    return {"mass": s["mass"]}


def _own_mass(s):
    sfi, c, shape, kv = _own_attention(s)
    sfi.sfi_attn_mass(shape, kv, c["sink"], c["recent"], s["q"], s["lse"], s["mass"], decay=c["decay"],
                      new_lens=s["new_lens"])
    return {"mass": s["mass"]}


def _evicted(s):
    return {"k_pool": s["k_pool"], "v_pool": s["v_pool"], "idx": s["idx"], "count": s["count"],
            "new_lens": s["new_lens"], "mass": s["mass_out"]}


def _plain_evict(s):
    c = s["case"]
    b, hkv, n = c["batch"], c["hkv"], s["max_len"]
    pos = torch.arange(n, device=DEV)
    length, k = s["seq_lens"].long()[:, None, None], s["k_per_req"].long()[:, None, None]
    sink = pos < c["sink"]
    recent = (pos >= length - c["recent"]) & (pos < length)
    cand = ~sink & (pos < length - c["recent"])
    order = torch.sort(torch.where(cand, s["mass"], torch.full_like(s["mass"], -math.inf)), dim=-1,
                       descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, pos.expand(b, hkv, -1))
    chosen = cand & (rank < k)
    s["count"].copy_(torch.minimum(cand.sum(-1)[:, 0], k[:, 0, 0]))
    # positions of the chosen rows and of all kept rows, ascending
    at = torch.where(chosen, pos, n).sort(-1).values[..., :s["idx"].shape[-1]]
    s["idx"][..., :at.shape[-1]] = torch.where(at < n, at.to(torch.int32), s["idx"][..., :at.shape[-1]])
    keep = ((sink & (pos < length)) | recent | chosen)
    src = torch.where(keep, pos, n).sort(-1).values
    s["new_lens"].copy_(keep.sum(-1)[:, 0])
    held = src < n
    src = src.clamp(max=n - 1)
    s["mass_out"].copy_(torch.where(held, torch.gather(s["mass"], -1, src), s["mass_out"]))
    table = s["page_table"].long()[:, None].expand(-1, hkv, -1)
    r, hh, to = held.nonzero(as_tuple=True)
    a, z = table[r, hh, src[r, hh, to] // PAGE], table[r, hh, to // PAGE]
    off = src[r, hh, to] % PAGE
    s["k_pool"][z, hh, to % PAGE] = s["k_pool"][a, hh, off]
    s["v_pool"][z, hh, to % PAGE] = s["v_pool"][a, hh, off]
    return _evicted(s)


def _own_evict(s):
    sfi, c, shape, kv = _own_attention(s)
    sfi.sfi_kv_evict(shape, kv, s["mass"], c["sink"], c["recent"], s["k_per_req"], s["idx"], s["count"],
                     s["new_lens"], mass_out=s["mass_out"])
    return _evicted(s)


def _plain_verify(s):
    c = s["case"]
    b, t = c["batch"], c["drafts"]
    step = torch.arange(t, device=DEV)
    x = s["tokens"].long()[..., None]
    p = torch.gather(s["target"][:, :t], -1, x)[..., 0].double()
    q = torch.ones_like(p) if s["draft"] is None else torch.gather(s["draft"], -1, x)[..., 0].double()
    ok = (s["u"][:, :t].double() * q < p) & (step < s["draft_lens"][:, None])
    a = ok.long().cumprod(-1).sum(-1)
    r = torch.arange(b, device=DEV)
    w = s["target"][r, a].double()
    at = a.clamp(max=t - 1)
    if s["draft"] is None:
        rest = w.scatter(-1, x[r, at], 0.0)
    else:
        rest = (w - s["draft"][r, at].double()).clamp(min=0)
    rest = torch.where((a < s["draft_lens"])[:, None], rest, w)
    w = torch.where(rest.sum(-1, keepdim=True) > 0, rest, w)
    cum = w.cumsum(-1)
    following = (cum > s["u"][:, t:].double() * cum[:, -1:]).long().argmax(-1)
    col = torch.arange(t + 1, device=DEV)
    drafts = torch.cat([s["tokens"].long(), torch.full_like(following[:, None], -1)], 1)
    out = torch.where(col < a[:, None], drafts, torch.where(col == a[:, None], following[:, None], -1))
    s["out_tokens"].copy_(out)
    s["accepted"].copy_(a)
    return {"tokens": s["out_tokens"], "accepted": s["accepted"]}


def _own_verify(s):
    import sparse_kv_long_sfi_gb300 as sfi
    sfi.sfi_verify_tokens(s["target"], s["draft"], s["tokens"], s["u"], s["out_tokens"], s["accepted"],
                          draft_lens=s["draft_lens"])
    return {"tokens": s["out_tokens"], "accepted": s["accepted"]}


def _plain_pages(s):
    table, lens, ref = s["page_table"], s["seq_lens"], s["ref_count"]
    col = torch.arange(table.shape[1], device=DEV)

    def pages(n):
        return ((n + PAGE - 1) // PAGE)[:, None]

    fresh = (col >= pages(lens)) & (col < pages(s["grown"]))
    row, at = fresh.nonzero(as_tuple=True)
    free = (ref == 0).nonzero()[:, 0][:row.numel()]
    ref[free] = 1
    table[row, at] = free.to(torch.int32)
    lens.copy_(s["grown"])
    row, at = ((col >= pages(s["kept"])) & (col < pages(lens))).nonzero(as_tuple=True)
    back = table[row, at].long()
    ref.index_add_(0, back, torch.full_like(back, -1, dtype=torch.int32))
    lens.copy_(s["kept"])
    return {"page_table": table, "seq_lens": lens, "ref_count": ref}


def _own_pages(s):
    import sparse_kv_long_sfi_gb300 as sfi
    if "map" not in s:
        s["map"] = sfi.PageMap(s["page_table"], s["seq_lens"], s["ref_count"])
        s["workspace"] = sfi.alloc_page_workspace(s["map"])
    sfi.sfi_page_reserve(s["map"], None, s["grown"], workspace=s["workspace"])
    sfi.sfi_page_trim(s["map"], s["kept"])
    return {"page_table": s["page_table"], "seq_lens": s["seq_lens"], "ref_count": s["ref_count"]}


_PLAIN = {"window": _plain_window, "mass": _plain_mass, "evict": _plain_evict, "verify": _plain_verify,
          "pages": _plain_pages}
_OWN = {"window": _own_window, "mass": _own_mass, "evict": _own_evict, "verify": _own_verify, "pages": _own_pages}


# ---- what a pass cannot do without ------------------------------------------------------------------------------

def _visible(p, c):
    """How many positions the token at position p sees."""
    first = max(c["sink"], p + 1 - c["recent"])
    return min(c["sink"], p + 1) + max(0, p + 1 - first)


def work(case):
    c, op, b = case, case["op"], case["batch"]
    if op in ("window", "mass"):
        new, ctx = _spread(c["new_min"], c["tokens"], b), _spread(c["ctx_min"], c["ctx_max"], b)
        pairs = sum(_visible(x + t, c) for n, x in zip(new, ctx) for t in range(n))
        # the rows that any of a request's tokens sees
        rows = sum(min(c["sink"], n + x) + max(0, n + x - max(c["sink"], x + 1 - c["recent"])) for n, x in zip(new, ctx))
        if op == "window":
            return {"bytes": sum(new) * c["hq"] * (4 * c["d"] + 4) + rows * c["hkv"] * 4 * c["d"],
                    "flops": 4 * c["d"] * c["hq"] * pairs}
        length = sum(new) + sum(ctx)
        return {"bytes": sum(new) * c["hq"] * (2 * c["d"] + 4) + c["hkv"] * (rows * 2 * c["d"] + 8 * length),
                "flops": 2 * c["d"] * c["hq"] * pairs}
    if op == "evict":
        total = 0
        for n, k in zip(_spread(c["len_min"], c["len_max"], b), _spread(c["k_min"], c["k_max"], b)):
            cand = max(0, n - c["recent"] - c["sink"])
            kept = min(k, cand)
            left = min(n, c["sink"]) + kept + min(c["recent"], max(0, n - c["sink"]))
            # candidates' weights; kept rows of K and V moved; their weights moved; indices written
            moved = left - c["sink"] if kept < cand else 0
            total += c["hkv"] * (4 * cand + moved * 8 * c["d"] + 8 * left + 4 * kept)
        return {"bytes": total, "flops": 0}
    if op == "verify":  # one row of each side where the drafts end, and two probabilities of each draft before it
        row = 4 * c["vocab"] * (1 if c["greedy"] else 2)
        return {"bytes": b * (row + c["drafts"] * 20 + 8), "flops": 3 * b * c["vocab"]}
    lens = _spread(c["len_min"], c["len_max"], b)
    grown = sum(-(-(n + c["grow"]) // PAGE) - -(-n // PAGE) for n in lens)
    return {"bytes": 4 * (6 * b + 5 * grown), "flops": 0}


# ---- the definitions in 64 bits ---------------------------------------------------------------------------------

def _line(s, pool, r, length):
    """The rows of request r by position, in 64 bits: [Hkv][length][D]."""
    return torch.cat(list(pool[s["page_table"][r, :-(-length // PAGE)].long()]), 1)[:, :length].double()


def exact(case, seed):
    s = prepare(case, seed)
    c, op, b = case, case["op"], case["batch"]
    if op in ("window", "mass"):
        hkv, g = c["hkv"], c["hq"] // c["hkv"]
        out = {n: s[n].double() for n in (("out", "lse") if op == "window" else ("mass",))}
        for r in range(b):
            length, n = int(s["seq_lens"][r]), int(s["new_lens"][r])
            k, v = _line(s, s["k_pool"], r, length), _line(s, s["v_pool"], r, length)
            if op == "mass":
                out["mass"][r, :, :length - n] *= c["decay"]
                out["mass"][r, :, length - n:length] = 0
            j = torch.arange(length, device=DEV)
            for t0 in range(0, n, 1024):
                t1 = min(n, t0 + 1024)
                p = length - n + torch.arange(t0, t1, device=DEV)[:, None]
                low = 0 if c["sink"] else max(0, length - n + t0 + 1 - c["recent"])  # nobody here sees what lies below
                hidden = ((j > p) | ((j >= c["sink"]) & (j <= p - c["recent"])))[:, low:]
                for h in range(hkv):
                    for i in range(h * g, h * g + g):
                        x = s["q"][r, t0:t1, i].double() @ k[h, low:].T / math.sqrt(c["d"])
                        x = x.masked_fill_(hidden, -math.inf)
                        if op == "mass":
                            w = (x - s["lse"][r, t0:t1, i, None].double()).exp_()
                            out["mass"][r, h, low:length] += w.sum(0)
                        else:
                            out["lse"][r, t0:t1, i] = torch.logsumexp(x, -1)
                            out["out"][r, t0:t1, i] = torch.softmax(x, -1) @ v[h, low:]
        return out
    if op == "evict":
        out = {n: s[n].double() for n in ("k_pool", "v_pool")}
        out.update(idx=s["idx"].clone(), count=None, new_lens=None, mass=s["mass_out"].double())
        for r in range(b):
            n, k = int(s["seq_lens"][r]), int(s["k_per_req"][r])
            lo, hi = min(n, c["sink"]), max(c["sink"], n - c["recent"])
            table = s["page_table"][r].long()
            for h in range(c["hkv"]):
                w = s["mass"][r, h, lo:min(n, hi)].double().cpu().tolist()
                best = sorted(sorted(range(len(w)), key=lambda i: (-w[i], i))[:k])
                src = torch.tensor(list(range(lo)) + [lo + i for i in best] + list(range(min(n, hi), n)), device=DEV)
                to = torch.arange(len(src), device=DEV)
                out["idx"][r, h, :len(best)] = src[lo:lo + len(best)].to(torch.int32)
                out["mass"][r, h, :len(src)] = s["mass"][r, h, src].double()
                for name in ("k_pool", "v_pool"):
                    out[name][table[to // PAGE], h, to % PAGE] = s[name][table[src // PAGE], h, src % PAGE].double()
        return out
    return None  # whole numbers
