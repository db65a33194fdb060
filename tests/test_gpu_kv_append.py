"""The append to the paged NVFP4 cache against the float64 reference.

The cache's bytes have to be equal: the codes are defined by the real-valued
formula, which float64 decides (nothing here lies within 2^-40 of a border
without lying on it).  q_out is fp32 arithmetic rounded once: half a step of
the dtype (2^-8 / 2^-11 of the value, 2^-25 for fp16 subnormals) plus 20 * 2^-24
of the magnitudes that the rotation adds (tests.kv_ref.rotate's M: two products
and an addition 2 u, the sum of 128 squares in at most 11 additions and the
root 9 u, the product with it 1 u; 20 u holds them all)."""
import numpy as np
import pytest
import torch

import nvfp4_quant_gb300 as rq
import synth
from nvfp4_quant_gb300 import build as rq_build
from tests import kv_ref, pins
from tests.gpu_util import GUARD, POISON, Guarded, dev16, f32dev, host16

pytestmark = pytest.mark.gpu

D = 128


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    rq_build.build()
    rq.lib()


def check_append(q, k, v, qw, kw, pos, table, slots, page, pages, gs_k, gs_v, dt, eps=1e-6, stride=None):
    """Runs the call on the bits q [T, Hq, 128], k, v [T, Hk, 128] and compares
    everything it writes."""
    t, hq, hk = q.shape[0], q.shape[1], k.shape[1]
    width = (hq + 2 * hk) * D
    fused = torch.zeros((t, stride or width), dtype=torch.int16, device="cuda").view(
        torch.bfloat16 if dt == "bf16" else torch.float16)
    views = []
    at = 0
    for a in (q, k, v):
        w = a.shape[1] * D
        fused[:, at:at + w] = dev16(a, dt).view(t, w)
        views.append(fused[:, at:at + w].unflatten(1, (a.shape[1], D)))
        at += w
    pool = Guarded((pages, hk, page * 144), torch.uint8)
    start = np.random.default_rng(1).integers(0, 256, (pages, hk, page * 144)).astype(np.uint8)
    pool.t.copy_(torch.from_numpy(start))
    out = Guarded((t, hq, D), fused.dtype)
    w16 = lambda w: None if w is None else dev16(w, dt)  # noqa: E731
    rq.rq_qkv_rope_nvfp4_kv_append(*views, w16(qw), w16(kw), eps, torch.from_numpy(pos).cuda(),
                                   torch.from_numpy(table).cuda(), f32dev(gs_k), f32dev(gs_v), out.t,
                                   pool.t, torch.from_numpy(slots).cuda(), page)
    torch.cuda.synchronize()
    f64 = lambda a: pins.bits_to_f64(a, dt)  # noqa: E731
    e = float(np.float32(eps))
    o, mag = kv_ref.rotate(f64(q), None if qw is None else f64(qw), e, pos, table)
    got = f64(host16(out.t))
    half = np.abs(o) * (2.0 ** -8 if dt == "bf16" else 2.0 ** -11) + (2.0 ** -25 if dt == "fp16" else 0)
    assert np.all(np.abs(got - o) <= half * (1 + 2.0 ** -10) + 20 * 2.0 ** -24 * mag)
    assert out.guards_intact() and pool.guards_intact()
    ko, _ = kv_ref.rotate(f64(k), None if kw is None else f64(kw), e, pos, table)
    gk, gv = float(np.float32(gs_k)), float(np.float32(gs_v))
    kc, ks = kv_ref.nvfp4(ko, gk)
    vc, vs = kv_ref.nvfp4(f64(v), gv)
    for i in range(t):
        if 0 <= slots[i] < pages * page:
            for h in range(hk):
                kv_ref.store(start, page, int(slots[i]), h, kc[i, h], ks[i, h], vc[i, h], vs[i, h])
    same = pool.t.cpu().numpy() == start
    assert same.all(), "%d of %d cache bytes differ, first at (page, head, byte) %s" % (
        (~same).sum(), same.size, np.argwhere(~same)[:4].tolist())


def inputs(seed, t, hq, hk, dt, norm="both", max_pos=None):
    q, k, qw, kw, pos, table = synth.qk_input(seed, t, hq, hk, D, dt)
    v = synth.normal_tensor(seed, 20, (t, hk, D), dt)
    r = np.random.default_rng(seed)
    if max_pos:
        table = synth.rope_cos_sin(max_pos, D)
        pos = r.integers(0, max_pos, t).astype(np.int32)
    return (q, k, v, qw if norm in ("both", "q") else None, kw if norm in ("both", "k") else None, pos,
            table)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("t, hq, hk, page, norm", [
    (1, 16, 8, 16, "both"), (1, 1, 1, 16, "none"), (3, 5, 1, 48, "both"), (5, 3, 3, 32, "q"),
    (37, 7, 2, 64, "k"), (64, 16, 8, 16, "both"), (64, 32, 4, 128, "none"), (700, 16, 8, 64, "both"),
    (701, 9, 3, 16, "both"), (1500, 32, 8, 32, "both"),
])
def test_append(t, hq, hk, page, norm, dt):
    x = inputs(11 + t, t, hq, hk, dt, norm, max_pos=5000 if t > 1 else None)
    pages = -(-t // page) + 2
    slots = np.random.default_rng(t).permutation(pages * page)[:t].astype(np.int64)
    check_append(*x, slots, page, pages, 2688.0 / 14, 2688.0 / 5.5, dt)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_padding_slots_and_strides(dt):
    """Slots outside the cache store nothing; the other rows' bytes stay; a
    token stride beyond the heads; positions outside the table are clamped."""
    t, page, pages = 50, 16, 6
    x = list(inputs(5, t, 4, 2, dt, max_pos=64))
    x[5] = np.concatenate([[-7, 64, 2 ** 31 - 1, -2 ** 31], x[5][4:]]).astype(np.int32)
    slots = np.random.default_rng(2).permutation(pages * page)[:t].astype(np.int64)
    slots[[0, 7, 20, 49]] = [-1, pages * page, 1 << 40, -(1 << 40)]
    check_append(*x, slots, page, pages, 200.0, 400.0, dt, stride=8 * D + 24)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_values_on_rounding_borders(dt):
    """Small integers without norms at position 0 with global scales that are
    powers of two: a large share of the codes and scales are exact ties."""
    t, hk, page = 96, 3, 32
    r = np.random.default_rng(8)
    bits = lambda a: synth.to_bits(a.astype(np.float64), dt)  # noqa: E731
    q = bits(r.integers(-12, 13, (t, 2, D)))
    k, v = bits(r.integers(-24, 25, (t, hk, D))), bits(r.integers(-96, 97, (t, hk, D)) / 4)
    pos, table = np.zeros(t, np.int32), synth.rope_cos_sin(2, D)
    for gs_k, gs_v in ((1.0, 1.0), (4.0, 0.5), (1.5, 6.0)):
        check_append(q, k, v, None, None, pos, table, np.arange(t, dtype=np.int64), page, 3, gs_k, gs_v, dt)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_extreme_rows(dt):
    """Zero rows, one non-zero element, outliers that make other blocks' scales
    0 or subnormal, saturated scales, tiny values, with and without norms."""
    t, page = 24, 16
    for norm in ("both", "none"):
        q, k, v, qw, kw, pos, table = inputs(9, t, 2, 2, dt, norm, max_pos=300)
        zero = np.zeros(D, np.uint16)
        big = synth.to_bits(np.full(1, 3000.0), dt)[0]
        small = synth.to_bits(np.full(1, 3e-5), dt)[0]
        for a in (q, k, v):
            a[0], a[1, 0] = 0, zero
            a[1, 0, 77] = big
            a[2, 1, 5], a[2, 1, 70] = big, big ^ 0x8000
            a[3] = small
            a[4, 0, :64] = 0x8000  # negative zeros
        check_append(q, k, v, qw, kw, pos, table, np.arange(t, dtype=np.int64), page, 2, 190.0, 400.0, dt)
        check_append(q, k, v, qw, kw, pos, table, np.arange(t, dtype=np.int64), page, 2, 1e-3, 3e5, dt)


def test_long_call_and_far_pages():
    """8191 tokens, and a cache of more than 4 GB whose last pages are written
    (offsets past 32 bits)."""
    t, hk, page = 8191, 2, 64
    x = inputs(3, t, 2, hk, "bf16", max_pos=9000)
    pages = -(-t // page)
    slots = np.arange(t, dtype=np.int64)[::-1].copy()
    check_append(*x, slots, page, pages, 190.0, 400.0, "bf16")
    q, k, v, qw, kw, pos, table = inputs(4, 40, 2, 8, "fp16", max_pos=100)
    far = 70000
    pool = torch.zeros((far, 8, 64 * 144), dtype=torch.uint8, device="cuda")  # 5.2 GB
    slots = torch.arange(40, device="cuda") + (far - 1) * 64
    args = [dev16(a, "fp16") for a in (q, k, v, qw, kw)]
    rq.qkv_rope_nvfp4_kv_append(*args, 1e-6, torch.from_numpy(pos).cuda(), torch.from_numpy(table).cuda(),
                                f32dev(190.0), f32dev(400.0), pool, slots, 64)
    near = torch.zeros((1, 8, 64 * 144), dtype=torch.uint8, device="cuda")
    rq.qkv_rope_nvfp4_kv_append(*args, 1e-6, torch.from_numpy(pos).cuda(), torch.from_numpy(table).cuda(),
                                f32dev(190.0), f32dev(400.0), near, torch.arange(40, device="cuda"), 64)
    torch.cuda.synchronize()
    assert torch.equal(pool[-1:], near) and near.any()
    assert not pool[:-1].any()


def test_binding_checks():
    x = torch.zeros((2, 4, D), dtype=torch.bfloat16, device="cuda")
    good = dict(pool=rq.nvfp4_kv_pool(2, 4, 16), slots=torch.zeros(2, dtype=torch.int64, device="cuda"),
                pos=torch.zeros(2, dtype=torch.int32, device="cuda"), cs=torch.zeros((8, D), device="cuda"))
    call = lambda q=x, k=x, v=x, w=None, **kw: rq.qkv_rope_nvfp4_kv_append(  # noqa: E731
        q, k, v, w, None, 1e-6, kw.get("pos", good["pos"]), kw.get("cs", good["cs"]), f32dev(1), f32dev(1),
        kw.get("pool", good["pool"]), kw.get("slots", good["slots"]), kw.get("page", 16))
    call()
    for bad in (dict(k=x.half()), dict(v=x[:1]), dict(w=torch.ones(64, dtype=x.dtype, device="cuda")),
                dict(pos=good["pos"].long()), dict(cs=good["cs"][:, :64]), dict(page=32),
                dict(slots=good["slots"].int()), dict(pool=good["pool"][:, :2]), dict(k=x[:, :2], v=x),
                dict(q=x.transpose(0, 1)), dict(slots=good["slots"].cpu())):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(ValueError):
        rq.nvfp4_kv_pool(1, 1, 20)
    torch.cuda.synchronize()
