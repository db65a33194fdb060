"""Cases of the NVFP4 KV-cache operators: the append of keys and values to a
paged 4-bit cache (per-head RMSNorm and RoPE on the way), and the attention
that reads the cache, for single tokens (decode) and for runs of new tokens
(extend).

A case is a dict of plain values; every sequence length follows from it.  The
plain forms below are elementary torch operations.  They work in 32 bits, and
in 64 where an NVFP4 code is decided (a value next to a rounding border has to
fall on the right side of it); results are rounded once.  The cache is compared
byte by byte: its codes are the correctly rounded ones, so they have one value.

Cache: uint8 [pages, kv heads, page_size * 144]; each 16 tokens of a page are
2304 bytes: K codes [16][64], V codes [16][64], K scales [16][8], V scales
[16][8].
"""
import math

import torch

own = False

D = 128            # elements of a head
GROUP = 16         # tokens of one group of the cache
GROUP_BYTES = 2304
EPS = 1e-6
THETA = 1.0e6
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of a batch of 64: 64 new tokens, the launch's latency counts
        dict(name="append_step64", op="append", tokens=64, hq=16, hk=8, dt="bf16", norm=True, page=16,
             padding=0),
        # the library's Q/K workload (4096 tokens, 16 + 8 heads) with V and pages of 64 tokens
        dict(name="append_4096", op="append", tokens=4096, hq=16, hk=8, dt="bf16", norm=True, page=64,
             padding=0),
        # a long prompt of a model without Q/K norms, fp16, with padding tokens at the end
        dict(name="append_32749", op="append", tokens=32749, hq=32, hk=8, dt="fp16", norm=False, page=32,
             padding=13),
        # one chat turn, one sequence: latency of a single-token call
        dict(name="decode_1x1000", op="decode", seqs=1, kv=1000, spread=0, hq=16, hk=8, dt="bf16",
             page=16, window=0, lse=False),
        # a serving batch with contexts between a few tokens and 4096
        dict(name="decode_64_ragged", op="decode", seqs=64, kv=4096, spread=4000, hq=32, hk=8, dt="fp16",
             page=64, window=0, lse=True),
        # few very long documents: one sequence's keys go over many SMs
        dict(name="decode_3x131001", op="decode", seqs=3, kv=131001, spread=20000, hq=16, hk=8, dt="bf16",
             page=128, window=0, lse=False),
        # a large batch at long contexts, 8 query heads to a KV head: the cache is far larger than L2
        dict(name="decode_128x8192", op="decode", seqs=128, kv=8192, spread=0, hq=64, hk=8, dt="bf16",
             page=64, window=0, lse=False),
        # four drafted tokens a sequence are checked at once
        dict(name="extend_draft_32x4", op="extend", seqs=32, q=4, qspread=0, kv=2048, spread=1500, hq=32,
             hk=8, dt="fp16", page=32, window=0, lse=False),
        # new prompts of about a thousand tokens (the cache holds nothing else yet)
        dict(name="extend_prompts_8x1024", op="extend", seqs=8, q=1024, qspread=300, kv=0, spread=0, hq=16,
             hk=8, dt="bf16", page=16, window=0, lse=True),
        # chunks of two long prompts after 14 thousand cached tokens, odd lengths
        dict(name="extend_chunk_2x2047", op="extend", seqs=2, q=2047, qspread=0, kv=14333, spread=999,
             hq=32, hk=8, dt="fp16", page=64, window=0, lse=False),
        # a sliding-window layer's chunk
        dict(name="extend_window_4x1500", op="extend", seqs=4, q=1500, qspread=0, kv=9000, spread=2500,
             hq=32, hk=4, dt="bf16", page=64, window=2048, lse=False),
        # one long prompt in one call
        dict(name="extend_prompt_8192", op="extend", seqs=1, q=8192, qspread=0, kv=0, spread=0, hq=32,
             hk=8, dt="bf16", page=64, window=0, lse=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "decode", "extend"))
    hk = rng.choice((1, 2, 3, 4, 8))
    hq = hk * rng.choice((1, 2, 3, 4, 5, 8))
    c = dict(op=op, hq=hq, hk=hk, dt=rng.choice(("bf16", "fp16")), page=16 * rng.choice((1, 2, 3, 4, 8)))
    if op == "append":
        return dict(c, tokens=_log(rng, 1, 32000 * 48 // max(48, hq + 2 * hk)), norm=rng.random() < 0.6,
                    padding=rng.choice((0, 0, 1, 5)))
    c = dict(c, window=rng.choice((0, 0, 0, _log(rng, 16, 4096))), lse=rng.random() < 0.3)
    if op == "decode":
        seqs = _log(rng, 1, 128)
        kv = _log(rng, 1, min(131072, (1 << 20) // seqs))
        return dict(c, seqs=seqs, kv=kv, spread=rng.choice((0, kv // 3, kv)))
    seqs, q = _log(rng, 1, 16), _log(rng, 2, 4096)
    seqs = max(1, min(seqs, 8192 // q))
    kv = min(rng.choice((0, _log(rng, 1, 8000))), max(0, 1900000000 // (hq * seqs * q) - q))
    return dict(c, seqs=seqs, q=q, qspread=rng.choice((0, q // 2, q - 1)), kv=kv,
                spread=rng.choice((0, kv // 2)))


def _lengths(case):
    """(query lengths, key lengths) of the sequences."""
    n = case["seqs"]
    back = lambda top, spread, i: max(0, top - (spread * ((i * 37 + 11) % n)) // max(1, n - 1))  # noqa: E731
    old = [back(case["kv"], case["spread"], i) if n > 1 else case["kv"] for i in range(n)]
    if case["op"] == "decode":
        return [1] * n, [max(1, k) for k in old]
    new = [max(1, back(case["q"], case["qspread"], i) if n > 1 else case["q"]) for i in range(n)]
    return new, [a + b for a, b in zip(old, new)]


def _visible(case):
    """(query-key pairs, keys read) summed over the sequences."""
    pairs = keys = 0
    w = case["window"]
    for nq, nk in zip(*_lengths(case)):
        first = nk - nq  # position of the first query
        if not w:
            pairs += nq * first + nq * (nq + 1) // 2
            keys += nk
        else:
            short = max(0, min(nq, w - first))  # queries whose window reaches back to key 0
            pairs += short * first + short * (short + 1) // 2 + (nq - short) * w
            keys += min(nk, nq + w - 1)
    return pairs, keys


def work(case):
    hq, hk = case["hq"], case["hk"]
    if case["op"] == "append":
        t, live = case["tokens"], case["tokens"] - min(case["padding"], case["tokens"] - 1)
        return {"bytes": t * (hq * 512 + 16) + live * hk * (512 + 144) + t * 512,
                "flops": t * (hq + 2 * hk) * D * 8}
    pairs, keys = _visible(case)
    t = sum(_lengths(case)[0])
    return {"bytes": keys * hk * 144 + t * hq * (512 + (4 if case["lse"] else 0)),
            "flops": 4 * D * hq * pairs}


# ---------------------------------------------------------------- inputs
def _quantise(y, gs):
    """NVFP4 of [..., 128] float64 values: (packed codes uint8 [..., 64], scales uint8 [..., 8])."""
    b = y.unflatten(-1, (8, 16))
    t = (b.abs().amax(-1) * gs / 6.0).clamp(max=448.0)
    step = torch.ldexp(torch.ones_like(t), torch.frexp(t)[1].clamp(min=-5) - 4)  # of E4M3 at t
    sf = (torch.round(t / step) * step).clamp(max=448.0)
    v = torch.where(sf[..., None] > 0, b * gs / sf[..., None], torch.zeros_like(b)).abs()
    code = ((v > 0.25).to(torch.uint8) + (v >= 0.75) + (v > 1.25) + (v >= 1.75) + (v > 2.5)
            + (v >= 3.5) + (v > 5.0)) | (torch.signbit(b).to(torch.uint8) << 3)
    code = code.flatten(-2)
    return (code[..., 0::2] | (code[..., 1::2] << 4),
            sf.float().to(torch.float8_e4m3fn).view(torch.uint8))


def _parts(pool):
    """K codes, V codes [pages, heads, groups, 16, 64], K scales, V scales [..., 16, 8]: views of the cache."""
    g = pool.unflatten(-1, (-1, GROUP_BYTES))
    return (g[..., :1024].unflatten(-1, (GROUP, 64)), g[..., 1024:2048].unflatten(-1, (GROUP, 64)),
            g[..., 2048:2176].unflatten(-1, (GROUP, 8)), g[..., 2176:].unflatten(-1, (GROUP, 8)))


def _table(n):
    inv = THETA ** (-torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)
    ang = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 7 + 1)
    normal = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    perm = lambda n: torch.randperm(n, generator=gen, device="cuda")  # noqa: E731
    dt, hq, hk, page = DT[case["dt"]], case["hq"], case["hk"], case["page"]
    one = lambda v: torch.tensor([v], dtype=torch.float32, device="cuda")  # noqa: E731
    s = dict(case=case, dt=dt, hq=hq, hk=hk, page=page)
    if case["op"] == "append":
        n = case["tokens"]
        qkv = normal(n, hq + 2 * hk, D)
        qkv[:, hq:hq + hk] *= 1.0 + 3.0 * (torch.rand(hk, D, generator=gen, device="cuda") < 0.03)
        qkv = qkv.to(dt)  # the fused projection's output: q, k and v are views into it
        s.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hk], v=qkv[:, hq + hk:])
        weight = lambda: (1 + 0.1 * normal(D)).to(dt) if case["norm"] else None  # noqa: E731
        s.update(qw=weight(), kw=weight())
        # contexts of up to 4096 tokens, wherever the new tokens stand in them
        s.update(positions=torch.randint(0, 4096, (n,), generator=gen, device="cuda").int(),
                 table=_table(4096))
        pages = -(-n // page) + 3
        slots = perm(pages)[torch.arange(n, device="cuda") // page] * page + torch.arange(n, device="cuda") % page
        s["live"] = n - min(case["padding"], n - 1)
        slots[s["live"]:] = -1
        s.update(slots=slots, gs_k=one(2688.0 / 14.0), gs_v=one(2688.0 / 5.5),
                 pool=torch.zeros(pages, hk, page * 144, dtype=torch.uint8, device="cuda"))
        return s
    new, keys = _lengths(case)
    per = -(-max(keys) // page)
    count = [-(-k // page) for k in keys]
    total = sum(count) + 2
    gs_k, gs_v = 2688.0 / 9.0, 2688.0 / 5.5
    pool = torch.empty(total, hk, page * 144, dtype=torch.uint8, device="cuda")
    kc, vc, ks, vs = _parts(pool)
    step = max(1, (1 << 25) // (hk * page * D))
    for a in range(0, total, step):
        z = pool[a:a + step].shape[0]
        kc[a:a + z], ks[a:a + z] = _quantise(normal(z, hk, page // GROUP, GROUP, D).double() * 1.3, gs_k)
        vc[a:a + z], vs[a:a + z] = _quantise(normal(z, hk, page // GROUP, GROUP, D).double(), gs_v)
    order = perm(total).int()
    block_table = torch.zeros(len(keys), per, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(count):
        block_table[i, :n] = order[at:at + n]
        at += n
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    s.update(pool=pool, block_table=block_table, kv_lens=ints(keys), q_starts=ints(starts), max_q=max(new),
             max_kv=max(keys), q=normal(starts[-1], hq, D).to(dt), gs_k=one(gs_k), gs_v=one(gs_v),
             scale=1.0 / math.sqrt(D), window=case["window"], lse=case["lse"])
    return s


# ---------------------------------------------------------------- plain forms
def _rotate(x, w, positions, table):
    """RMSNorm (with a weight) and NeoX rotation of [tokens, heads, 128], in x's precision."""
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.to(x.dtype)
    c, s = table[positions.long()].to(x.dtype)[:, None].split(64, -1)
    a, b = x[..., :64], x[..., 64:]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def _plain_append(s):
    q_out = _rotate(s["q"].float(), s["qw"], s["positions"], s["table"]).to(s["dt"])
    n = s["live"]
    k = _rotate(s["k"][:n].double(), s["kw"], s["positions"][:n], s["table"])  # 64 bits: code borders
    slot = s["slots"][:n]
    page, at = slot // s["page"], slot % s["page"]
    kc, vc, ks, vs = _parts(s["pool"])
    kc[page, :, at // GROUP, at % GROUP], ks[page, :, at // GROUP, at % GROUP] = _quantise(k, s["gs_k"].double())
    vc[page, :, at // GROUP, at % GROUP], vs[page, :, at // GROUP, at % GROUP] = _quantise(
        s["v"][:n].double(), s["gs_v"].double())
    return {"q": q_out, "pool": s["pool"]}


def _values(codes, scales, gs):
    """The float32 values of [b, pages, heads, groups, 16, 64] codes, as [b, heads, tokens, 128]."""
    lut = torch.tensor(E2M1, dtype=torch.float32, device="cuda")
    v = torch.stack([lut[(codes & 15).int()], lut[(codes >> 4).int()]], -1).flatten(-2).unflatten(-1, (8, 16))
    v = v * (scales.contiguous().view(torch.float8_e4m3fn).float() / gs)[..., None]
    return v.flatten(-2).transpose(1, 2).flatten(2, 4)


def _plain_attention(s):
    table = s["block_table"].long()
    kc, vc, ks, vs = (p[table] for p in _parts(s["pool"]))
    keys, values = _values(kc, ks, s["gs_k"]), _values(vc, vs, s["gs_v"])
    n, tq, hk = len(table), s["max_q"], s["hk"]
    ar = torch.arange(s["q"].shape[0], device="cuda")
    seq = torch.searchsorted(s["q_starts"][1:], ar.int(), right=True)  # of each query token
    row = ar - s["q_starts"].long()[seq]
    q = torch.zeros(n, tq, s["hq"], D, device="cuda")
    q[seq, row] = s["q"].float()
    q = q.unflatten(2, (hk, -1)).permute(0, 2, 3, 1, 4)  # [n, hk, G, tq, D]
    scores = (q.flatten(2, 3) @ keys.transpose(-1, -2)).unflatten(2, (-1, tq)) * s["scale"]
    lens, nq = s["kv_lens"].long(), s["q_starts"].diff().long()
    p = (lens - nq)[:, None] + torch.arange(tq, device="cuda")  # positions of the queries
    j = torch.arange(keys.shape[2], device="cuda")
    seen = (j <= p[..., None]) & (j < lens[:, None, None])
    if s["window"]:
        seen &= j > p[..., None] - s["window"]
    scores = scores.masked_fill(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True).clamp(min=-1e30)
    e = torch.exp(scores - top)
    del scores
    total = e.sum(-1, keepdim=True)
    o = (e.flatten(2, 3) @ values).unflatten(2, (-1, tq)) / total.clamp(min=1e-30)
    out = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[seq, row].to(s["dt"])
    if not s["lse"]:
        return {"out": out}
    lse = (torch.log(total) + top)[..., 0].permute(0, 3, 1, 2).flatten(2, 3)[seq, row]
    return {"out": out, "lse": lse}


# ---------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if not own:
        return _plain_append(s) if op == "append" else _plain_attention(s)
    import nvfp4_quant_gb300 as rq
    if op == "append":
        q = rq.qkv_rope_nvfp4_kv_append(s["q"], s["k"], s["v"], s["qw"], s["kw"], EPS, s["positions"],
                                        s["table"], s["gs_k"], s["gs_v"], s["pool"], s["slots"], s["page"])
        return {"q": q, "pool": s["pool"]}
    if op == "decode":
        out, lse = rq.paged_decode_attn_nvfp4(s["q"], s["pool"], s["page"], s["block_table"], s["kv_lens"],
                                              s["gs_k"], s["gs_v"], s["scale"], window=s["window"],
                                              with_lse=s["lse"])
    else:
        out, lse = rq.paged_extend_attn_nvfp4(s["q"], s["pool"], s["page"], s["block_table"], s["q_starts"],
                                              s["kv_lens"], s["max_q"], s["gs_k"], s["gs_v"], s["scale"],
                                              window=s["window"], with_lse=s["lse"])
    return {"out": out, "lse": lse} if s["lse"] else {"out": out}


# ---------------------------------------------------------------- from the definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        x = s["q"].double()
        if s["qw"] is not None:
            x = x / torch.sqrt(torch.sum(x * x, -1, keepdim=True) / D + EPS) * s["qw"].double()
        row = s["table"].double()[s["positions"].long()]
        turn = torch.complex(row[:, :64], row[:, 64:])[:, None]
        z = torch.complex(x[..., :64], x[..., 64:]) * turn
        return {"q": torch.cat([z.real, z.imag], -1), "pool": None}
    new, keys = _lengths(case)
    hk, per = case["hk"], case["hq"] // case["hk"]
    level = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    out = torch.zeros(sum(new), case["hq"], D, dtype=torch.float64, device="cuda")
    lse = torch.full((sum(new), case["hq"]), -math.inf, dtype=torch.float64, device="cuda")
    at = 0
    for b, (nq, nk) in enumerate(zip(new, keys)):
        pages = s["pool"][s["block_table"][b, :-(-nk // case["page"])].long()]
        q = s["q"][at:at + nq].double()
        pos = torch.arange(nk - nq, nk, device="cuda")[:, None]
        for h in range(hk):
            g = pages[:, h].reshape(-1, GROUP_BYTES)  # groups of 16 tokens

            def cached(codes, scales, gs):
                c = g[:, codes:codes + 1024].reshape(-1, 64)[:nk].long()
                x = torch.empty(nk, D, dtype=torch.float64, device="cuda")
                x[:, 0::2], x[:, 1::2] = level[c & 15], level[c // 16]
                f = g[:, scales:scales + 128].reshape(-1, 8)[:nk].contiguous().view(torch.float8_e4m3fn).double()
                return x * f.repeat_interleave(16, 1) / gs.double()

            k, v = cached(0, 2048, s["gs_k"]), cached(1024, 2176, s["gs_v"])
            for a in range(0, nq, 1024):  # queries at once, to bound the memory
                z = min(nq, a + 1024)
                hide = torch.arange(nk, device="cuda") > pos[a:z]
                if case["window"]:
                    hide |= torch.arange(nk, device="cuda") <= pos[a:z] - case["window"]
                for i in range(h * per, (h + 1) * per):
                    w = (q[a:z, i] @ k.T / math.sqrt(D)).masked_fill_(hide, -math.inf)
                    l = torch.logsumexp(w, -1)
                    lse[at + a:at + z, i] = l
                    out[at + a:at + z, i] = torch.exp(w - l[:, None]) @ v
        at += nq
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}
