"""The 4-bit cache in plain numpy, from its definition: where each code and scale lies in a
block, group quantisation to nearest even, and attention in fp64 over what the codes say."""
import numpy as np

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)
# e4m3: 127 finite magnitudes (code 127 is NaN)
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1])


def offsets(d):
    """(byte, shift, scale byte) of K[token][dim] and of V[token][dim] in a block."""
    tok, dim = np.arange(16)[:, None], np.arange(d)[None]
    k = (tok * (d // 2) + dim // 2, np.broadcast_to(dim % 2 * 4, (16, d)), 8 * d + tok * (d // 16) + dim // 16)
    a, b, c, e, f = dim // 64, dim // 16 % 4, dim // 8 % 2, dim // 2 % 4, dim % 2
    t, h, low = tok // 4, tok // 2 % 2, tok % 2
    v = (9 * d + 512 * a + 128 * e + 32 * t + 16 * f + 4 * b + 2 * h + c, np.broadcast_to(low * 4, (16, d)),
         17 * d + t * (d // 4) + 4 * (dim // 16) + tok % 4)
    return k, v


def nearest_even(x, table):
    mid = (table[1:] + table[:-1]) / 2
    lo, hi = np.searchsorted(mid, x, "left"), np.searchsorted(mid, x, "right")
    return np.where(lo == hi, lo, np.where(lo % 2 == 0, lo, hi))


def quantise(x, g):
    """x fp64 [..., D] -> codes [..., D], scale codes [..., D/16] (uint8)."""
    xg = x.reshape(*x.shape[:-1], -1, 16)
    fine = np.isfinite(xg).all(-1)
    xf = np.where(fine[..., None], xg, 0.0)
    s = nearest_even(np.minimum(np.abs(xf).max(-1) / 6 / g, 448.0), E4M3)
    step = (E4M3[s] * g)[..., None]
    y = np.where(step > 0, np.abs(xf) / np.where(step > 0, step, 1), 0)
    code = nearest_even(np.minimum(y, 6.0), GRID)
    code = np.where((step > 0) & fine[..., None], code + 8 * np.signbit(xf), 0)
    return code.reshape(x.shape).astype(np.uint8), np.where(fine, s, 127).astype(np.uint8)


def values(code, scale, g):
    s = np.append(E4M3, np.nan)[scale & 127] * g
    v = np.where(code >= 8, -1.0, 1.0) * GRID[code & 7]
    return v * np.repeat(s, 16, -1)


def write_rows(block, which, rows, code, scale):
    """Put codes [n][D] and scales [n][D/16] of the rows (K: which 0, V: 1) into a block, in place."""
    d = code.shape[-1]
    byte, shift, at = offsets(d)[which]
    for i, row in enumerate(rows):
        for x in range(d):
            b, s = byte[row, x], shift[row, x]
            block[b] = (block[b] & (0xF0 if s == 0 else 0x0F)) | (code[i, x] << s)
        block[at[row, ::16]] = scale[i]


def read_rows(blocks, d, g_k, g_v):
    """Blocks [..., 18 D] -> K, V fp64 [..., 16, D]."""
    out = []
    for (byte, shift, at), g in zip(offsets(d), (g_k, g_v)):
        code = blocks[..., byte] >> shift & 15
        out.append(values(code, blocks[..., at[:, ::16]], g))
    return out


def positions(pool, table, L, d, g_k, g_v):
    """K, V fp64 [Hkv][L][D] of one request."""
    blocks = pool[table[:-(-L // 16)]]
    return [x.swapaxes(0, 1).reshape(pool.shape[1], -1, d)[:, :L] for x in read_rows(blocks, d, g_k, g_v)]


def attend(q, k, v, seen, scale):
    """q [G][D], k/v [N][D], seen [N] -> out [G][D], lse [G], logits [G][N], and the bounds on the
    fp32 kernel's out and logits (see test_gpu_kv4)."""
    with np.errstate(invalid="ignore", over="ignore"):
        x = (q @ k.T) * scale
        dx = 2.0 ** -23 * q.shape[-1] * (np.abs(q) @ np.abs(k).T) * scale
        if not seen.any():
            z = np.zeros((q.shape[0], v.shape[1]))
            return z, np.full(q.shape[0], -np.inf), x, z + 1e-30, dx, np.zeros(q.shape[0])
        xs, vs = x[:, seen], v[seen]
        m = xs.max(-1, keepdims=True)
        p = np.exp(xs - m)
        n = p.sum(-1, keepdims=True)
        p = p / n
        out = p @ vs
        eps = 2 * dx[:, seen].max(-1) + 2.0 ** -19 + (seen.sum() / 8 + 64) * 2.0 ** -23
        bound = eps[:, None] * (p @ np.abs(vs)) + 2.0 ** -32 * np.abs(vs).sum(0) + 1e-30
        return out, (m + np.log(n))[:, 0], x, bound, dx, eps
