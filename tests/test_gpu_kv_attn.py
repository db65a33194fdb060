"""Attention over the paged NVFP4 cache against the float64 reference.

Bounds, with u = 2^-24, S the largest sum |q k| scale of a visible key and A =
sum p |v| (both from the reference): a score is a sum of 128 exact products in
fp32, wrong by at most 130 * 2u S (2u an addition: the order and the rounding
inside a matrix instruction are not given), 2u of it from the scale, and for
bf16 queries 2^-24 S from their fp16 copy; call it ds.  A probability is wrong
by the factor e^ds, 2^-11 (fp16) and 2^-21 (ex2, sums), an output by those
times 2 A (numerator and denominator) and by its own sum over the keys, n / 16
+ 64 additions of at most 2u A; then one rounding to the dtype.  lse: ds, the
sum's additions and 4u of itself."""
import math

import numpy as np
import pytest
import torch

import nvfp4_quant_gb300 as rq
import synth
from nvfp4_quant_gb300 import build as rq_build
from tests import kv_ref, pins
from tests.gpu_util import Guarded, dev16, f32dev, host16

pytestmark = pytest.mark.gpu

D, U = 128, 2.0 ** -24
GS_K, GS_V = 2688.0 / 9.0, 2688.0 / 5.5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    rq_build.build()
    rq.lib()


class Cache:
    """A cache with the given sequence lengths in scattered pages, the bytes of
    tokens past a sequence's end all ones (NaN scales)."""

    def __init__(self, seed, lens, hk, page, spare=2, stride_extra=0, spread=1.0):
        r = np.random.default_rng(seed)
        self.lens, self.hk, self.page = list(lens), hk, page
        need = [-(-n // page) for n in lens]
        self.pages = sum(need) + spare
        order = r.permutation(self.pages).astype(np.int32)
        self.table = np.full((len(lens), max(1, max(need)) + stride_extra), -1, np.int32)
        self.pool = np.full((self.pages, hk, page * 144), 0xFF, np.uint8)
        at = 0
        flat = self.pool.reshape(self.pages, hk, page // 16, 2304)
        for b, n in enumerate(lens):
            self.table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
            kc, ks = kv_ref.nvfp4(r.standard_normal((n, hk, D)) * spread, GS_K)
            vc, vs = kv_ref.nvfp4(r.standard_normal((n, hk, D)), GS_V)
            t = np.arange(n)
            p, g, i = self.table[b, t // page], t % page // 16, t % 16
            for base, codes, sbase, sf in ((0, kc, 2048, ks), (1024, vc, 2176, vs)):
                packed = codes[..., 0::2] | (codes[..., 1::2] << 4)
                for h in range(hk):
                    rows = flat[:, h, :, base:base + 1024].reshape(self.pages, page // 16, 16, 64)
                    rows[p, g, i] = packed[:, h]
                    flat[:, h, :, base:base + 1024] = rows.reshape(self.pages, page // 16, 1024)
                    rows = flat[:, h, :, sbase:sbase + 128].reshape(self.pages, page // 16, 16, 8)
                    rows[p, g, i] = sf[:, h]
                    flat[:, h, :, sbase:sbase + 128] = rows.reshape(self.pages, page // 16, 128)
        self.dpool = torch.from_numpy(self.pool).cuda()
        self.dtable = torch.from_numpy(self.table).cuda()
        self.dlens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")


def compare(cache, q, starts, got, lse, scale, window, dt, table=None):
    """Every row of got (bits) and lse against the reference; rows outside the
    sequences are not looked at."""
    qf = pins.bits_to_f64(q, dt)
    gf = pins.bits_to_f64(got, dt)
    per = q.shape[1] // cache.hk
    table = cache.table if table is None else table
    gk, gv = float(np.float32(GS_K)), float(np.float32(GS_V))
    scale = float(np.float32(scale))
    half = 2.0 ** -8 if dt == "bf16" else 2.0 ** -11
    for b, n in enumerate(cache.lens):
        a, z = starts[b], starts[b + 1]
        if a == z:
            continue
        ids = table[b, :-(-n // cache.page)]
        ok = (ids >= 0) & (ids < cache.pages)
        seen = np.repeat(ok, cache.page)[:n]
        for h in range(cache.hk):
            k, v = kv_ref.load(cache.pool, cache.page, np.where(ok, ids, 0), n, h, gk, gv)
            for i in range(h * per, (h + 1) * per):
                o, l, mag, s = kv_ref.attend(qf[a:z, i], k, v, n - (z - a), scale, window, seen)
                ds = (130 * 2 * U + 2 * U + 2.0 ** -24) * s
                sums = (n / 16 + 64) * 2 * U
                tol = mag * (2 * (ds + 2.0 ** -11 + 2.0 ** -21) + sums)[:, None] if np.ndim(ds) else \
                    mag * (2 * (ds + 2.0 ** -11 + 2.0 ** -21) + sums)
                tol = tol + np.abs(o) * half * (1 + 2.0 ** -8) + 2.0 ** -25
                bad = ~(np.abs(gf[a:z, i] - o) <= tol)
                assert not bad.any(), "seq %d head %d: %d of %d outputs off, worst %.3g of the bound" % (
                    b, i, bad.sum(), bad.size, (np.abs(gf[a:z, i] - o) / tol).max())
                if lse is not None:
                    fine = np.isfinite(l)
                    assert np.array_equal(np.isneginf(lse[a:z, i]), ~fine)
                    off = np.abs(lse[a:z, i][fine] - l[fine])
                    assert np.all(off <= (ds + sums + 2.0 ** -20)[fine] + 4 * U * np.abs(l[fine]))


def run_decode(cache, hq, dt, window=0, scale=None, seed=0, q=None, table=None, with_lse=True, qpad=0):
    n = len(cache.lens)
    scale = scale or 1 / math.sqrt(D)
    q = synth.normal_tensor(seed, 4, (n, hq, D), dt) if q is None else q
    buf = torch.zeros((n, hq * D + qpad), dtype=torch.int16, device="cuda")
    buf[:, :hq * D] = dev16(q, dt).view(torch.int16).view(n, hq * D)
    qd = buf.view(torch.bfloat16 if dt == "bf16" else torch.float16)[:, :hq * D].unflatten(1, (hq, D))
    out = Guarded((n, hq, D), qd.dtype)
    lse = Guarded((n, hq), torch.float32) if with_lse else None
    ws = torch.full((rq.rq_paged_attn_nvfp4_workspace_bytes(hq, cache.hk),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    rq.rq_paged_decode_attn_nvfp4(qd, cache.dpool, cache.page,
                                  cache.dtable if table is None else torch.from_numpy(table).cuda(),
                                  cache.dlens, f32dev(GS_K), f32dev(GS_V), scale, out.t, ws, window,
                                  None if lse is None else lse.t)
    torch.cuda.synchronize()
    assert out.guards_intact() and (lse is None or lse.guards_intact())
    compare(cache, q, list(range(n + 1)), host16(out.t), None if lse is None else lse.t.cpu().numpy(),
            scale, window, dt, table)
    return host16(out.t)


def run_extend(cache, hq, new, dt, window=0, seed=0, max_q=None, behind=0, q=None, table=None, scale=None):
    scale = scale or 1 / math.sqrt(D)
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    t = int(starts[-1]) + behind
    q = synth.normal_tensor(seed, 4, (t, hq, D), dt) if q is None else q
    qd = dev16(q, dt)
    out = Guarded((t, hq, D), qd.dtype)
    out.t.view(torch.int16).fill_(0x1234)
    lse = Guarded((t, hq), torch.float32)
    lse.t.fill_(7.0)
    ws = torch.full((rq.rq_paged_attn_nvfp4_workspace_bytes(hq, cache.hk),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    rq.rq_paged_extend_attn_nvfp4(qd, cache.dpool, cache.page,
                                  cache.dtable if table is None else torch.from_numpy(table).cuda(),
                                  torch.from_numpy(starts).cuda(), cache.dlens,
                                  max(new) if max_q is None else max_q, f32dev(GS_K), f32dev(GS_V), scale,
                                  out.t, ws, window, lse.t)
    torch.cuda.synchronize()
    assert out.guards_intact() and lse.guards_intact()
    compare(cache, q, list(starts), host16(out.t), lse.t.cpu().numpy(), scale, window, dt, table)
    if behind:
        assert np.all(host16(out.t)[-behind:] == 0x1234) and torch.all(lse.t[-behind:] == 7.0)
    return host16(out.t)


LENS = [1, 0, 15, 16, 17, 31, 33, 64, 250, 257, 1000, 2049]


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("hq, hk, page", [(1, 1, 16), (2, 2, 48), (16, 8, 64), (9, 3, 16), (5, 1, 32),
                                          (16, 2, 128), (12, 1, 16), (16, 1, 64), (40, 2, 16), (48, 1, 32)])
def test_decode(hq, hk, page, dt):
    run_decode(Cache(1, LENS, hk, page), hq, dt, seed=hq)


@pytest.mark.parametrize("hq, hk, page, dt", [(2, 2, 48, "fp16"), (16, 2, 16, "bf16"), (32, 2, 32, "bf16"),
                                              (20, 1, 64, "fp16")])
def test_decode_wide_table(hq, hk, page, dt):
    """Tables wider than the sequences need (long-context capacity)."""
    c = Cache(30, LENS, hk, page, stride_extra=20000 // page)
    run_decode(c, hq, dt)
    run_extend(c, hq, [1, 0, 2, 1, 3, 1, 1, 2, 1, 1, 2, 4], dt, window=40)


@pytest.mark.parametrize("seqs, hq, hk", [(9, 16, 8), (72, 8, 1), (9, 32, 2), (300, 4, 4)])
def test_decode_batches(seqs, hq, hk):
    lens = np.random.default_rng(seqs).integers(0, 600, seqs)
    lens[seqs // 2] = 2100
    run_decode(Cache(31, lens.tolist(), hk, 32), hq, "bf16")


@pytest.mark.parametrize("window", [1, 5, 16, 100, 511, 5000])
def test_decode_window(window):
    run_decode(Cache(2, LENS, 2, 32), 8, "bf16", window=window)
    run_decode(Cache(2, LENS, 2, 16), 32, "fp16", window=window)


def test_window_up_to_the_largest_int():
    """A window past every length hides nothing, whatever the positions."""
    c = Cache(33, [1, 2, 0, 90, 300], 2, 16)
    run_decode(c, 4, "bf16", window=2 ** 31 - 1)
    run_extend(c, 4, [9, 2, 40, 5, 20], "bf16", window=2 ** 31 - 1)
    run_extend(c, 4, [900, 2, 40, 500, 300], "fp16", window=2 ** 31 - 4)


@pytest.mark.parametrize("window", [1, 37, 100])
@pytest.mark.parametrize("new", [1, 3, 150])
def test_bytes_before_the_window_are_not_looked_at(window, new):
    """Tokens that no query sees hold NaN scales (a page given to others)."""
    c = Cache(34, [40, 200, 901, 1500], 2, 32)
    new = [min(new, n) for n in c.lens]
    flat = c.pool.reshape(c.pages, 2, 2, 2304)
    for b, n in enumerate(c.lens):
        for t in range(max(0, n - new[b] - window + 1)):
            g, i = flat[c.table[b, t // 32], :, t % 32 // 16], t % 16
            for base, size in ((0, 64), (1024, 64), (2048, 8), (2176, 8)):
                g[:, base + i * size:base + (i + 1) * size] = 0xFF
    c.dpool = torch.from_numpy(c.pool).cuda()
    if max(new) == 1:
        run_decode(c, 4, "bf16", window=window)
        run_decode(c, 32, "fp16", window=window)
    run_extend(c, 4, new, "fp16", window=window)


def test_decode_one_long_sequence():
    """One sequence over every SM, 40,007 keys; one and two KV heads."""
    run_decode(Cache(3, [40007], 1, 64), 4, "fp16")
    run_decode(Cache(3, [40007], 2, 64), 24, "bf16", window=33333)


@pytest.mark.parametrize("n", [130, 700, 1500])
def test_decode_many_sequences(n):
    """More sequences than threads of a CTA, most of them short."""
    r = np.random.default_rng(n)
    run_decode(Cache(4, r.integers(0, 60, n).tolist(), 1, 16), 2, "bf16")


def test_decode_strides():
    c = Cache(5, [100, 37, 260], 2, 16, stride_extra=3)
    run_decode(c, 4, "bf16", qpad=40)
    run_decode(c, 4, "fp16", qpad=8, with_lse=False)


@pytest.mark.parametrize("bad", [-1, -2 ** 31, 2 ** 31 - 1, "pages"])
def test_bad_page_ids_hide_their_tokens(bad):
    c = Cache(6, [200, 48, 64, 300], 2, 16)
    table = c.table.copy()
    value = c.pages if bad == "pages" else bad
    table[0, 3] = table[0, 12] = value
    table[1, :] = value  # nothing left: out 0, lse -inf
    table[3, 0] = value
    out = run_decode(c, 8, "bf16", table=table)
    assert not out[1].any()
    run_extend(c, 4, [5, 48, 30, 1], "fp16", table=table)


def test_lengths_out_of_range_are_clamped():
    c = Cache(7, [64, 96], 1, 32)
    c.dlens = torch.tensor([-5, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    c.lens = [0, 96]  # the table holds 3 pages of 32
    run_decode(c, 4, "bf16")


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_score_ranges(dt):
    """Rows whose scores are huge, equal, tiny or of rising size (the running
    maximum moves late), and queries of very different sizes within a row."""
    c = Cache(8, [700, 700, 700, 700], 2, 16)
    q = synth.normal_tensor(1, 4, (4, 4, D), dt)
    q[0] = 0
    f = pins.bits_to_f64(q, dt)
    f[1] *= 60.0
    f[2] *= 2.0 ** -20
    f[3, :, :100] *= 2.0 ** -16
    f[3, :, 100] *= 500.0
    run_decode(c, 4, dt, q=synth.to_bits(f, dt))
    # keys that grow along the sequence: one channel rises with the token
    k = np.zeros((700, 2, D))
    k[:, :, 7] = np.linspace(-9, 9, 700)[:, None]
    kc, ks = kv_ref.nvfp4(k, GS_K)
    vc, vs = kv_ref.nvfp4(np.random.default_rng(5).standard_normal((700, 2, D)), GS_V)
    for t in range(700):
        for h in range(2):
            kv_ref.store(c.pool, 16, int(c.table[1, t // 16]) * 16 + t % 16, h, kc[t, h], ks[t, h], vc[t, h], vs[t, h])
    c.dpool.copy_(torch.from_numpy(c.pool))
    g = np.ones((4, 4, D))
    g[:, :, 7] = [60.0, -60.0, 9.0, 500.0]
    run_decode(c, 4, dt, q=synth.to_bits(g, dt))


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("hq, hk, page", [(4, 4, 16), (16, 8, 64), (6, 2, 48), (8, 1, 32), (24, 1, 16)])
def test_extend_few_queries(hq, hk, page, dt):
    """Runs of 0 to 9 queries, among them runs longer than the sequence (their
    first queries see nothing)."""
    lens = [1, 5, 3, 64, 100, 257, 0, 1000, 33]
    new = [1, 0, 6, 4, 7, 2, 3, 5, 9]
    run_extend(Cache(9, lens, hk, page), hq, new, dt, behind=5)


@pytest.mark.parametrize("window", [0, 1, 17, 130, 1000])
@pytest.mark.parametrize("hq, hk, page, dt", [(4, 2, 16, "bf16"), (8, 1, 64, "fp16"), (3, 3, 32, "bf16")])
def test_extend_prompts(hq, hk, page, dt, window):
    """Prompts and chunks of one to some hundreds of tokens."""
    lens = [1, 127, 128, 129, 300, 513, 700, 40, 0, 20]
    new = [1, 127, 128, 100, 300, 257, 33, 0, 0, 45]
    run_extend(Cache(10, lens, hk, page), hq, new, dt, window=window, behind=3)


@pytest.mark.parametrize("window", [0, 60])
@pytest.mark.parametrize("hq, hk, page, dt", [(16, 2, 16, "bf16"), (20, 4, 48, "fp16"), (8, 8, 32, "bf16"),
                                              (48, 2, 64, "fp16")])
def test_extend_mixed_batch(hq, hk, page, dt, window):
    """A batch of single tokens, drafted runs, chunks and prompts: both of the
    library's attention kernels take their part of it."""
    r = np.random.default_rng(hq)
    new = [1, 4, 90, 1, 0, 130, 257, 33, 1, 7, 300, 64, 2, 150]
    old = r.integers(0, 400, len(new))
    lens = [int(a + b) for a, b in zip(old, new)]
    lens[5] = 100  # fewer keys than queries
    run_extend(Cache(21, lens, hk, page), hq, new, dt, window=window, behind=2)


def test_extend_prompts_of_many_heads():
    run_extend(Cache(22, [128, 129, 500, 640], 4, 16), 32, [128, 129, 255, 300], "bf16")
    run_extend(Cache(22, [700] * 9, 4, 64), 4, [200] * 9, "fp16", window=333)


def test_extend_bad_pages_in_a_prompt():
    """Unreadable pages in the middle of chunks whose rows fill several blocks."""
    c = Cache(23, [900, 640], 2, 16)
    table = c.table.copy()
    table[0, [0, 7, 8, 9, 10, 11, 12, 13, 14, 15, 40]] = -1
    table[1, :] = c.pages
    out = run_extend(c, 32, [420, 333], "bf16", table=table)
    assert not out[420:].any()


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_extend_score_ranges(dt):
    """As test_score_ranges, for chunks: rows without size, large and small
    rows, keys that grow so that the maximum moves in every tile."""
    c = Cache(24, [1000, 700], 2, 32)
    k = np.zeros((1000, 2, D))
    k[:, :, 7] = np.linspace(-9, 9, 1000)[:, None]
    kc, ks = kv_ref.nvfp4(k, GS_K)
    vc, vs = kv_ref.nvfp4(np.random.default_rng(5).standard_normal((1000, 2, D)), GS_V)
    for t in range(1000):
        for h in range(2):
            kv_ref.store(c.pool, 32, int(c.table[0, t // 32]) * 32 + t % 32, h, kc[t, h], ks[t, h], vc[t, h], vs[t, h])
    c.dpool.copy_(torch.from_numpy(c.pool))
    f = pins.bits_to_f64(synth.normal_tensor(1, 4, (600, 16, D), dt), dt)
    f[:200, :, 7] *= np.linspace(-60, 60, 200)[:, None]
    f[200:260] *= 40.0
    f[260:300] *= 2.0 ** -18
    f[300:310] = 0
    f[310:400, :, :100] *= 2.0 ** -16
    run_extend(c, 16, [300, 300], dt, q=synth.to_bits(f, dt))


def test_extend_long_chunk():
    run_extend(Cache(11, [3000], 1, 64), 4, [1100], "bf16")
    run_extend(Cache(11, [2500, 600], 2, 16), 4, [700, 600], "fp16", window=600)


@pytest.mark.parametrize("window", [0, 200])
def test_extend_wide_table(window):
    """Room for 20,000 keys, few of them there: parts of blocks that have nothing to do."""
    c = Cache(40, [500, 90, 1300, 3000, 4], 2, 32, stride_extra=600)
    run_extend(c, 16, [400, 90, 700, 50, 4], "bf16", window=window, behind=2)
    run_extend(c, 32, [400, 90, 700, 900, 4], "fp16", window=window)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_extend_more_blocks_than_sms(dt):
    """Blocks after one another on an SM, many of them without a key."""
    run_extend(Cache(37, [40, 700, 0, 300], 1, 16), 16, [3000, 600, 70, 1000], dt)
    run_extend(Cache(38, [1000, 5, 1500], 4, 32), 32, [1000, 900, 700], dt, window=333)


@pytest.mark.parametrize("lens, new, hq, hk, dt, window", [
    ([9600], [600], 8, 1, "bf16", 0), ([5000, 3], [300, 3], 16, 1, "fp16", 3000),
    ([8300, 4100, 700], [333, 129, 600], 16, 1, "bf16", 0), ([2500], [2400], 8, 2, "fp16", 0)])
def test_extend_few_blocks_of_many_keys(lens, new, hq, hk, dt, window):
    """Blocks of rows whose keys several SMs share: joined, the same each time,
    and with pages that cannot be read."""
    c = Cache(36, lens, hk, 64)
    a = run_extend(c, hq, new, dt, window=window)
    assert np.array_equal(a, run_extend(c, hq, new, dt, window=window))
    table = c.table.copy()
    table[0, 1::3] = -1
    table[0, 20:36] = -1
    run_extend(c, hq, new, dt, window=window, table=table)


@pytest.mark.parametrize("max_q", [0, 1, 7, 100000])
def test_max_q_len_is_a_hint(max_q):
    """The bound chooses kernels; whatever it says, the results are right."""
    run_extend(Cache(12, [40, 300, 700], 2, 32), 6, [3, 200, 1], "bf16", max_q=max_q)


def test_starts_out_of_order_are_clamped():
    """Decreasing or out-of-range starts: no row outside q is touched."""
    c = Cache(13, [50, 60], 1, 16)
    q = dev16(synth.normal_tensor(1, 4, (6, 2, D), "bf16"), "bf16")
    for starts in ([0, 4, 2], [-9, 3, 1 << 30], [5, 5, 99]):
        out = Guarded((6, 2, D), q.dtype)
        ws = torch.empty(rq.rq_paged_attn_nvfp4_workspace_bytes(2, 1), dtype=torch.uint8, device="cuda")
        rq.rq_paged_extend_attn_nvfp4(q, c.dpool, 16, c.dtable,
                                      torch.tensor(starts, dtype=torch.int32, device="cuda"), c.dlens, 6,
                                      f32dev(GS_K), f32dev(GS_V), 0.1, out.t, ws)
        torch.cuda.synchronize()
        assert out.guards_intact()


def test_workspaces_that_are_refused():
    """One whose memory is not what its size says, too small, or none."""
    c = Cache(35, [20], 1, 16)
    q = torch.zeros((1, 2, D), dtype=torch.bfloat16, device="cuda")
    n = rq.rq_paged_attn_nvfp4_workspace_bytes(2, 1)
    for ws in (torch.empty(1, dtype=torch.uint8, device="cuda").expand(n),
               torch.empty((n, 2), dtype=torch.uint8, device="cuda")[:, 0], None):
        with pytest.raises(ValueError):
            rq.rq_paged_decode_attn_nvfp4(q, c.dpool, 16, c.dtable, c.dlens, f32dev(1), f32dev(1), 0.1, q.clone(), ws)
    with pytest.raises(rq.RQError):
        rq.paged_decode_attn_nvfp4(q, c.dpool, 16, c.dtable, c.dlens, f32dev(1), f32dev(1), 0.1,
                                   workspace=torch.empty(n - 1, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        rq.paged_decode_attn_nvfp4(q[0], c.dpool, 16, c.dtable, c.dlens, f32dev(1), f32dev(1), 0.1)


def test_decode_equals_extend_by_one():
    c = Cache(14, [1, 100, 517, 0, 64], 2, 32)
    q = synth.normal_tensor(3, 4, (5, 6, D), "bf16")
    assert np.array_equal(run_decode(c, 6, "bf16", q=q), run_extend(c, 6, [1] * 5, "bf16", q=q))


def test_repeatable_and_graph_replay():
    """Two eager calls and a graph's replays, on new inputs too, give the same bits."""
    c = Cache(15, [900, 3, 77, 5000], 4, 64)
    q = dev16(synth.normal_tensor(1, 4, (4, 16, D), "bf16"), "bf16")
    q2 = dev16(synth.normal_tensor(2, 4, (4, 16, D), "bf16"), "bf16")
    one, two = f32dev(GS_K), f32dev(GS_V)
    call = lambda x, **kw: rq.paged_decode_attn_nvfp4(x, c.dpool, 64, c.dtable, c.dlens, one, two, 0.09, **kw)[0]  # noqa: E731
    a, a2 = call(q), call(q2)
    assert torch.equal(call(q).view(torch.int16), a.view(torch.int16))
    ws = [torch.empty(rq.rq_paged_attn_nvfp4_workspace_bytes(16, 4), dtype=torch.uint8, device="cuda") for _ in range(2)]
    x = q.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call(x, workspace=ws[0])
    for src, want in ((q, a), (q2, a2), (q, a)):
        x.copy_(src)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    # two streams at once, a workspace each
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(10):
        for i in range(2):
            outs[i].append(call((q, q2)[i], workspace=ws[i], stream=s[i]))
    torch.cuda.synchronize()
    for i, want in ((0, a), (1, a2)):
        assert all(torch.equal(o.view(torch.int16), want.view(torch.int16)) for o in outs[i])


@pytest.mark.parametrize("lens, new, hq, hk", [([9600, 40], [600, 40], 8, 1), ([1000, 0, 1500, 700], [1000, 50, 700, 700], 32, 4),
                                               ([2500, 1], [900, 1], 16, 2)])
def test_extend_repeats_streams_and_replays(lens, new, hq, hk):
    """The same bits from calls one after another on one workspace, from two streams
    at once, and from a captured call replayed between others on its stream."""
    c = Cache(39, lens, hk, 32)
    starts = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    q = [dev16(synth.normal_tensor(i, 4, (sum(new), hq, D), "bf16"), "bf16") for i in range(2)]
    one, two = f32dev(GS_K), f32dev(GS_V)
    call = lambda x, **kw: rq.paged_extend_attn_nvfp4(x, c.dpool, 32, c.dtable, starts, c.dlens, max(new), one, two,  # noqa: E731
                                                      0.09, **kw)[0].view(torch.int16)
    want = [call(x) for x in q]
    ws = [torch.full((rq.rq_paged_attn_nvfp4_workspace_bytes(hq, hk),), 0xFF, dtype=torch.uint8, device="cuda")
          for _ in range(2)]
    for i in range(20):
        assert torch.equal(call(q[i % 2], workspace=ws[0]), want[i % 2])
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = [(i, call(q[i], workspace=ws[i], stream=s[i])) for _ in range(10) for i in range(2)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i, o in outs)
    x = q[0].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call(x, workspace=ws[0])
    for i in (0, 1, 1, 0):
        x.copy_(q[i])
        g.replay()
        other = call(q[1 - i], workspace=ws[0])
        torch.cuda.synchronize()
        assert torch.equal(out, want[i]) and torch.equal(other, want[1 - i])


def test_far_pages():
    """Pages more than 4 GB into the cache."""
    c = Cache(16, [150, 90], 2, 64)
    far = 240000
    pool = torch.full((far, 2, 64 * 144), 0xFF, dtype=torch.uint8, device="cuda")  # 4.4 GB
    pool[far - c.pages:] = c.dpool
    q = dev16(synth.normal_tensor(1, 4, (2, 8, D), "fp16"), "fp16")
    one, two = f32dev(GS_K), f32dev(GS_V)
    want = rq.paged_decode_attn_nvfp4(q, c.dpool, 64, c.dtable, c.dlens, one, two, 0.09)[0]
    got = rq.paged_decode_attn_nvfp4(q, pool, 64, torch.where(c.dtable < 0, c.dtable, c.dtable + (far - c.pages)),
                                     c.dlens, one, two, 0.09)[0]
    starts = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    ext = rq.paged_extend_attn_nvfp4(q, pool, 64, torch.where(c.dtable < 0, c.dtable, c.dtable + (far - c.pages)),
                                     starts, c.dlens, 2000, one, two, 0.09)[0]
    torch.cuda.synchronize()
    assert torch.equal(want.view(torch.int16), got.view(torch.int16))
    off = (ext.float() - want.float()).abs().max().item()
    assert off <= 2.0 ** -9  # two sums of the same terms, outputs below 1


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_prompt_then_tokens(dt):
    """As a program uses them: a prompt is appended and attended, then tokens
    one by one and a drafted run, on one stream without a wait in between; each
    result against the float64 attention over the cache's own values."""
    hq, hk, page, lens = 6, 2, 16, [53, 16, 70]
    pages_per = 7
    r = np.random.default_rng(20)
    c = Cache(17, [0] * 3, hk, page, spare=3 * pages_per)
    c.table = r.permutation(3 * pages_per).astype(np.int32).reshape(3, pages_per)
    c.pages = 3 * pages_per
    table = synth.rope_cos_sin(256, D)
    dtable, dcs = torch.from_numpy(c.table).cuda(), torch.from_numpy(table).cuda()
    pool = rq.nvfp4_kv_pool(c.pages, hk, page)
    gk, gv = f32dev(GS_K), f32dev(GS_V)
    qw, kw = (dev16(synth.to_bits(1 + 0.1 * r.standard_normal(D), dt), dt) for _ in range(2))
    have = [0, 0, 0]
    for step, new in enumerate((lens, [1, 1, 1], [1, 1, 1], [3, 0, 4])):
        t = sum(new)
        qkv = dev16(synth.to_bits(r.standard_normal((t, hq + 2 * hk, D)), dt), dt)
        pos = np.concatenate([np.arange(a, a + n) for a, n in zip(have, new)]).astype(np.int32)
        seq = np.repeat(np.arange(3), new)
        slots = c.table[seq, pos // page].astype(np.int64) * page + pos % page
        q = rq.qkv_rope_nvfp4_kv_append(qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:], qw, kw, 1e-6,
                                        torch.from_numpy(pos).cuda(), dcs, gk, gv, pool,
                                        torch.from_numpy(slots).cuda(), page)
        have = [a + n for a, n in zip(have, new)]
        klens = torch.tensor(have, dtype=torch.int32, device="cuda")
        starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        if new == [1, 1, 1]:
            out, lse = rq.paged_decode_attn_nvfp4(q, pool, page, dtable, klens, gk, gv, 1 / math.sqrt(D), with_lse=True)
        else:
            out, lse = rq.paged_extend_attn_nvfp4(q, pool, page, dtable, torch.from_numpy(starts).cuda(), klens,
                                                  max(new), gk, gv, 1 / math.sqrt(D), with_lse=True)
        torch.cuda.synchronize()
        c.pool, c.lens = pool.cpu().numpy(), list(have)
        compare(c, host16(q), list(starts), host16(out), lse.cpu().numpy(), 1 / math.sqrt(D), 0, dt)
