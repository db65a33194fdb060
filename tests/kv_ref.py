"""Float64 reference of the paged NVFP4 KV cache: the append (norm, rotation,
NVFP4 codes) and the attention, from their definitions, in numpy.

The cache's byte layout, for checking against: page p, head h, token t of the
page lie in 2304 bytes (K codes 16 x 64, V codes 16 x 64, K scales 16 x 8, V
scales 16 x 8) at ((p * heads + h) * (page_size / 16) + t / 16) * 2304."""
import numpy as np

from tests import pins

D = 128
GROUP = 2304


def _nearest_even(v, levels):
    """Index of the nearest of the increasing levels (ties: the even index), saturating."""
    levels = np.asarray(levels)
    up = np.clip(np.searchsorted(levels, v, side="left"), 0, len(levels) - 1)
    dn = np.maximum(up - 1, 0)
    a, b = np.abs(v - levels[dn]), np.abs(levels[up] - v)
    return np.where((a < b) | ((a == b) & (dn % 2 == 0)), dn, up)


def nvfp4(y, gs):
    """(codes [..., 128] of 4 bits, scale bytes [..., 8]) of float64 y [..., 128]."""
    e4m3 = pins.e4m3_table()[:127]  # +0 .. 448
    e2m1 = pins.e2m1_table()[:8]
    b = y.reshape(y.shape[:-1] + (8, 16))
    sf = _nearest_even(np.abs(b).max(-1) * gs / 6.0, e4m3)
    s = e4m3[sf][..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        v = np.where(s > 0, np.abs(b) * gs / s, 0.0)
    code = _nearest_even(v, e2m1) | (np.signbit(b).astype(np.int64) << 3)
    return code.reshape(y.shape).astype(np.uint8), sf.astype(np.uint8)


def rotate(x, w, eps, pos, table):
    """(o, M) of float64 x [T, H, 128]: the normed and rotated rows, and the
    sums of magnitudes |t_i c| + |t_j s| times rstd behind each element."""
    r = 1.0
    if w is not None:
        r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        x = x * w
    cs = table.astype(np.float64)[np.clip(pos, 0, len(table) - 1)][:, None]
    c, s = cs[..., :64], cs[..., 64:]
    a, b = x[..., :64], x[..., 64:]
    o = np.concatenate([a * c - b * s, b * c + a * s], -1) * r
    a, b, c, s = np.abs(a), np.abs(b), np.abs(c), np.abs(s)
    return o, np.concatenate([a * c + b * s, b * c + a * s], -1) * r


def group_at(pages, heads, page_size, slot, head):
    """Byte offset of the slot's group of one head, and its row in the group."""
    page, t = slot // page_size, slot % page_size
    return ((page * heads + head) * (page_size // 16) + t // 16) * GROUP, t % 16


def store(pool, page_size, slot, head, kc, ksf, vc, vsf):
    """Writes one token's codes and scales of one head into the flat cache bytes."""
    pages, heads = pool.shape[:2]
    at, r = group_at(pages, heads, page_size, slot, head)
    flat = pool.reshape(-1)
    for base, codes, sbase, sf in ((0, kc, 2048, ksf), (1024, vc, 2176, vsf)):
        flat[at + base + r * 64:at + base + r * 64 + 64] = codes[0::2] | (codes[1::2] << 4)
        flat[at + sbase + r * 8:at + sbase + r * 8 + 8] = sf


def load(pool, page_size, pages, n, head, gs_k, gs_v):
    """Float64 keys and values [n, 128] of the first n tokens of a page list."""
    heads = pool.shape[1]
    e2m1, e4m3 = pins.e2m1_table(), pins.e4m3_table()
    g = pool.reshape(pool.shape[0], heads, -1, GROUP)[np.asarray(pages, np.int64), head].reshape(-1, GROUP)

    def part(codes, scales, gs):
        c = g[:, codes:codes + 1024].reshape(-1, 64)[:n]
        v = np.empty((n, D))
        v[:, 0::2], v[:, 1::2] = e2m1[c & 15], e2m1[c >> 4]
        return v * np.repeat(e4m3[g[:, scales:scales + 128].reshape(-1, 8)[:n]], 16, axis=1) / gs

    return part(0, 2048, gs_k), part(1024, 2176, gs_v)


def attend(q, keys, values, first, scale, window, seen_pages=None):
    """One head: queries [n, 128] at positions first .. against keys [m, 128].
    Returns (out, lse, A, S): A = sum p |v| per element and S = the largest
    sum |q k| scale of a visible key, for the error bounds."""
    n, m = len(q), len(keys)
    pos = first + np.arange(n)[:, None]
    j = np.arange(m)
    seen = j <= pos
    if window:
        seen &= j > pos - window
    if seen_pages is not None:
        seen &= seen_pages
    keys = np.where(seen.any(0)[:, None], keys, 0.0)
    values = np.where(seen.any(0)[:, None], values, 0.0)
    s = np.where(seen, scale * (q @ keys.T), -np.inf)
    top = np.where(seen.any(1), s.max(1, initial=-np.inf), 0.0)
    e = np.exp(s - top[:, None])
    total = e.sum(1)
    with np.errstate(divide="ignore"):
        lse = np.where(total > 0, top + np.log(total), -np.inf)
    p = e / np.where(total > 0, total, 1.0)[:, None]
    mag = np.where(seen, scale * (np.abs(q) @ np.abs(keys).T), 0.0).max(1, initial=0.0)
    return p @ values, lse, p @ np.abs(values), mag
