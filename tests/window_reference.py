"""Attention through a sliding window with sinks, its weights, eviction by them and draft verification in plain
numpy, fp64 (exact integers where a result is one)."""
import math
from fractions import Fraction

import numpy as np
import torch


class Cache:
    """Paged bf16 K and V of requests with n new tokens each, pages scattered over the pool."""

    def __init__(self, seed, lens, hq, hkv, d, spare=3, fill=None):
        g = np.random.default_rng(seed)
        self.lens, self.hq, self.hkv, self.d = list(lens), hq, hkv, d
        need = [-(-n // 16) for n in lens]
        self.pages = sum(need) + spare
        ids = g.permutation(self.pages)
        self.table = np.zeros((len(lens), max(1, max(need)) + 1), np.int32)
        at = 0
        for r, n in enumerate(need):
            self.table[r, :n] = ids[at:at + n]
            at += n
        self.k = torch.from_numpy(g.standard_normal((self.pages, hkv, 16, d)).astype(np.float32)).to(torch.bfloat16)
        self.v = torch.from_numpy(g.standard_normal((self.pages, hkv, 16, d)).astype(np.float32)).to(torch.bfloat16)
        if fill is not None:  # what nobody has written
            used = np.zeros((self.pages, 16), bool)
            for r, n in enumerate(lens):
                for j in range(n):
                    used[self.table[r, j // 16], j % 16] = True
            stale = torch.from_numpy(~used)[:, None, :, None].expand(-1, hkv, -1, d)
            self.k[stale] = fill
            self.v[stale] = fill

    def rows(self, pool, r, h):
        n = self.lens[r]
        pages = torch.from_numpy(self.table[r].astype(np.int64))
        return pool[pages, h].reshape(-1, self.d)[:n].double().numpy()

    def device(self):
        import sparse_kv_long_sfi_gb300 as sfi
        self.shape = sfi.AttnShape(self.hq, self.hkv, self.d)
        self.kv = sfi.PagedKV(self.k.cuda(), self.v.cuda(), torch.from_numpy(self.table).cuda(),
                              torch.tensor(self.lens, dtype=torch.int32, device="cuda"))
        return self.shape, self.kv


def queries(seed, b, t, hq, d):
    g = np.random.default_rng(seed)
    return torch.from_numpy(g.standard_normal((b, t, hq, d)).astype(np.float32)).to(torch.bfloat16)


def sees(p, n, sink, recent):
    j = np.arange(n)
    return (j <= p) & ((j < sink) | (j > p - recent))


def token(cache, r, h, q, p, sink, recent):
    """One query row: out, lse, weights over the cache, sum w |v|, largest sum |q k| scale among what it sees."""
    k, v = cache.rows(cache.k, r, h // (cache.hq // cache.hkv)), cache.rows(cache.v, r, h // (cache.hq // cache.hkv))
    see = sees(p, len(k), sink, recent)
    if not see.any():
        return np.zeros(cache.d), -math.inf, np.zeros(len(k)), np.zeros(cache.d), 0.0
    scale = 1 / math.sqrt(cache.d)
    qd = q.double().numpy()
    x = k[see] @ qd * scale
    m = x.max()
    e = np.exp(x - m)
    w = np.zeros(len(k))
    w[see] = e / e.sum()
    return (w[see] @ v[see], m + math.log(e.sum()), w, w[see] @ np.abs(v[see]),
            float((np.abs(k[see]) @ np.abs(qd)).max() * scale))


def out_bound(ref, mag, d):
    """The output is rounded to bf16 (2^-8 of it), each weight before the product with V too (2^-8 of sum w |v|);
    scores and sums are fp32: d products each, and the exponential's 2^-22."""
    return 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -12) * mag + 1e-30


def lse_bound(lse, score_mag, d):
    """fp32 dot products (d terms, each sum off by its magnitude's 2^-23), the exponential (2^-22), sums, log2."""
    return 2 * d * 2.0 ** -24 * score_mag + 2.0 ** -19 * (1 + abs(lse))


def keep(weights, length, sink, recent, k):
    """Positions kept of one (request, KV head), ascending, and the chosen candidates among them."""
    lo, hi = min(sink, length), max(min(sink, length), length - recent)
    best = sorted(sorted(range(lo, hi), key=lambda j: (-weights[j], j))[:k])
    return list(range(lo)) + best + list(range(hi, length)), best


def fixed(p):
    """A probability in units of 2^-56."""
    return 0 if not p > 0 else math.floor(Fraction(min(float(p), 1.0)) * 2 ** 56)


def verify(target, draft, tokens, u, n):
    """Accepted drafts of one request and the token behind them."""
    a = 0
    while a < n:
        q = Fraction(float(draft[a][tokens[a]])) if draft is not None else Fraction(1)
        p = float(target[a][tokens[a]])
        if math.isnan(p) or math.isnan(float(u[a])) or not Fraction(float(u[a])) * q < Fraction(p):
            break
        a += 1
    w = [fixed(x) for x in target[a]]
    if a < n:
        rest = ([max(x - fixed(y), 0) for x, y in zip(w, draft[a])] if draft is not None
                else [0 if i == tokens[a] else x for i, x in enumerate(w)])
        w = rest if sum(rest) else w
    total, cum = sum(w), 0
    if not total:
        return a, -1
    goal = Fraction(float(u[len(tokens)])) * total
    for i, x in enumerate(w):
        cum += x
        if cum > goal:
            return a, i
    raise AssertionError("no step above the goal")
