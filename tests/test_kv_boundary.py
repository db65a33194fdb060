"""The paged NVFP4 cache's entry points without a GPU: bad arguments get the
documented status before any CUDA call (no pointer below is dereferenced), and
the float64 reference of the GPU tests holds on worked values."""
import numpy as np
import pytest
import torch

import nvfp4_quant_gb300 as rq
from nvfp4_quant_gb300 import build as rq_build
from tests import kv_ref, pins

OK, NULL, SHAPE, DTYPE, MISAL, ALIAS, UNSUP = 0, 1, 2, 3, 4, 5, 6

A = {n: 0x100000000 * (i + 1) for i, n in enumerate(
    ["q", "k", "v", "qw", "kw", "pos", "cs", "kg", "vg", "qo", "pool", "slots", "table", "starts",
     "lens", "out", "lse", "ws"])}


@pytest.fixture(scope="module")
def L():
    rq_build.build()
    return rq.lib()


def append(L, **kw):
    a = dict(A, qs=16 * 128, ks=8 * 128, vs=8 * 128, t=32, hq=16, hk=8, d=128, maxp=4096, pages=10,
             page=64, dt=0)
    a.update(kw)
    return L.rq_qkv_rope_nvfp4_kv_append(
        a["q"], a["k"], a["v"], a["qs"], a["ks"], a["vs"], a["t"], a["hq"], a["hk"], a["d"], a["qw"],
        a["kw"], 1e-6, a["pos"], a["cs"], a["maxp"], a["kg"], a["vg"], a["qo"], a["pool"], a["pages"],
        a["page"], a["slots"], a["dt"], None)


def decode(L, **kw):
    a = dict(A, qs=16 * 128, n=4, hq=16, hk=8, d=128, pages=10, page=64, stride=5, per=5, scale=0.1,
             window=0, bytes=rq.rq_paged_attn_nvfp4_workspace_bytes(16, 8), dt=1)
    a.update(kw)
    return L.rq_paged_decode_attn_nvfp4(
        a["q"], a["qs"], a["n"], a["hq"], a["hk"], a["d"], a["pool"], a["pages"], a["page"],
        a["table"], a["stride"], a["per"], a["lens"], a["scale"], a["window"], a["kg"], a["vg"],
        a["out"], a["lse"], a["ws"], a["bytes"], a["dt"], None)


def extend(L, **kw):
    a = dict(A, qs=16 * 128, t=40, n=4, maxq=16, hq=16, hk=8, d=128, pages=10, page=64, stride=5,
             per=5, scale=0.1, window=0, bytes=rq.rq_paged_attn_nvfp4_workspace_bytes(16, 8), dt=1)
    a.update(kw)
    return L.rq_paged_extend_attn_nvfp4(
        a["q"], a["qs"], a["t"], a["starts"], a["n"], a["maxq"], a["hq"], a["hk"], a["d"], a["pool"],
        a["pages"], a["page"], a["table"], a["stride"], a["per"], a["lens"], a["scale"], a["window"],
        a["kg"], a["vg"], a["out"], a["lse"], a["ws"], a["bytes"], a["dt"], None)


def test_sizes(L):
    assert rq.rq_nvfp4_kv_page_bytes(16) == 2304 and rq.rq_nvfp4_kv_page_bytes(64) == 64 * 144
    for bad in (0, -16, 8, 24, rq.RQ_KV_MAX_PAGE + 16):
        assert rq.rq_nvfp4_kv_page_bytes(bad) == 0
    assert rq.rq_paged_attn_nvfp4_workspace_bytes(16, 8) > 0
    for bad in ((0, 8), (16, 0), (10, 4), (-2, 1)):
        assert rq.rq_paged_attn_nvfp4_workspace_bytes(*bad) == 0


def test_constants_match_the_header():
    import re
    from tests.test_boundary import HEADER
    text = open(HEADER).read()
    for name in ("RQ_KV_MAX_PAGE", "RQ_ATTN_MAX_KEYS", "RQ_ATTN_MAX_TOKENS", "RQ_ATTN_MAX_SEQS"):
        assert int(re.search(r"#define\s+%s\s+(\d+)" % name, text).group(1)) == getattr(rq, name)


@pytest.mark.parametrize("want, kw", [
    (OK, dict(t=0)), (OK, dict(t=0, q=None, k=None, v=None, pool=None)), (OK, dict(hq=0, hk=0)),
    (DTYPE, dict(dt=2)), (DTYPE, dict(dt=-1, t=0)), (SHAPE, dict(t=-1)), (SHAPE, dict(hq=-1)),
    (SHAPE, dict(hk=65537)), (SHAPE, dict(maxp=0)), (UNSUP, dict(d=64)), (SHAPE, dict(page=24)),
    (SHAPE, dict(page=0)), (SHAPE, dict(page=65536 + 16)), (SHAPE, dict(pages=-1)),
    (SHAPE, dict(pages=1 << 30)), (SHAPE, dict(qs=15 * 128)), (MISAL, dict(ks=8 * 128 + 4)),
    (SHAPE, dict(vs=1 << 41)), (NULL, dict(q=None)), (NULL, dict(v=None)), (NULL, dict(qo=None)),
    (NULL, dict(kg=None)), (NULL, dict(vg=None)), (NULL, dict(slots=None)), (NULL, dict(pool=None)),
    (NULL, dict(pos=None)), (NULL, dict(cs=None)), (MISAL, dict(q=A["q"] + 8)),
    (MISAL, dict(kw=A["kw"] + 2)), (MISAL, dict(slots=A["slots"] + 4)), (MISAL, dict(pool=A["pool"] + 4)),
    (MISAL, dict(kg=A["kg"] + 1)), (ALIAS, dict(qo=A["q"])), (ALIAS, dict(qo=A["pool"] + 64)),
    (ALIAS, dict(pool=A["slots"] - 10 * 8 * 64 * 144 + 16)), (ALIAS, dict(pool=A["v"])),
])
def test_append_refusals(L, want, kw):
    assert append(L, **kw) == want


COMMON = [
    (DTYPE, dict(dt=5)), (SHAPE, dict(n=-1)), (SHAPE, dict(hq=15)), (SHAPE, dict(hq=0)),
    (SHAPE, dict(hk=0)), (UNSUP, dict(d=96)), (SHAPE, dict(page=8)), (SHAPE, dict(pages=-2)),
    (SHAPE, dict(per=6)), (SHAPE, dict(per=-1)), (SHAPE, dict(scale=0.0)), (SHAPE, dict(scale=-1.0)),
    (SHAPE, dict(scale=float("nan"))), (SHAPE, dict(scale=float("inf"))), (SHAPE, dict(scale=3e38)),
    (SHAPE, dict(window=-1)), (SHAPE, dict(bytes=1000)),
    (SHAPE, dict(per=1 << 25, stride=1 << 25)), (SHAPE, dict(qs=128)), (MISAL, dict(qs=16 * 128 + 1)),
    (NULL, dict(q=None)), (NULL, dict(pool=None)), (NULL, dict(table=None)), (NULL, dict(lens=None)),
    (NULL, dict(kg=None)), (NULL, dict(vg=None)), (NULL, dict(out=None)), (NULL, dict(ws=None)),
    (MISAL, dict(q=A["q"] + 2)), (MISAL, dict(out=A["out"] + 8)), (MISAL, dict(ws=A["ws"] + 4)),
    (MISAL, dict(lens=A["lens"] + 2)), (MISAL, dict(lse=A["lse"] + 2)), (ALIAS, dict(out=A["q"])),
    (ALIAS, dict(out=A["pool"])), (ALIAS, dict(ws=A["out"] - 16)), (ALIAS, dict(lse=A["out"])),
]


@pytest.mark.parametrize("want, kw", COMMON + [(OK, dict(n=0)), (OK, dict(n=0, q=None, out=None)),
                                               (SHAPE, dict(n=(1 << 20) + 1))])
def test_decode_refusals(L, want, kw):
    assert decode(L, **kw) == want


@pytest.mark.parametrize("want, kw", COMMON + [
    (OK, dict(n=0)), (OK, dict(t=0)), (SHAPE, dict(t=(1 << 24) + 1)), (SHAPE, dict(maxq=-1)),
    (NULL, dict(starts=None)), (MISAL, dict(starts=A["starts"] + 2)), (ALIAS, dict(out=A["starts"] - 16)),
    (SHAPE, dict(t=1 << 20, hq=2048, hk=1, qs=2048 * 128))])
def test_extend_refusals(L, want, kw):
    assert extend(L, **kw) == want


def test_binding_refuses_host_and_misshapen_tensors():
    x = torch.zeros((2, 4, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        rq.qkv_rope_nvfp4_kv_append(x, x, x, None, None, 1e-6, torch.zeros(2, dtype=torch.int32),
                                    torch.zeros(8, 128), torch.ones(1), torch.ones(1),
                                    torch.zeros((1, 4, 2304), dtype=torch.uint8),
                                    torch.zeros(2, dtype=torch.int64), 16)
    with pytest.raises(ValueError, match="CUDA"):
        rq.paged_decode_attn_nvfp4(x, torch.zeros((1, 4, 2304), dtype=torch.uint8), 16,
                                   torch.zeros((2, 1), dtype=torch.int32),
                                   torch.zeros(2, dtype=torch.int32), torch.ones(1), torch.ones(1), 1.0,
                                   workspace=torch.zeros(16, dtype=torch.uint8))


def test_reference_quantiser_on_worked_values():
    """gs = 1: a = 6 gives sf = 1 and the codes of the values themselves (ties to
    the even code, signs kept); a block of zeros gives sf = 0; saturation."""
    y = np.zeros((2, 128))
    y[0, :16] = [6, -6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.0, 0.2500001, 4.99999, -2.6, 0.5, 1, 3]
    y[1, :16] = 1e6
    c, sf = kv_ref.nvfp4(y, 1.0)
    assert list(c[0, :16]) == [7, 15, 0, 2, 2, 4, 4, 6, 6, 8, 1, 6, 13, 1, 2, 5]
    assert sf[0, 0] == 0x38 and not sf[0, 1:].any() and not c[0, 16:].any()
    assert sf[1, 0] == 0x7E and (c[1, :16] == 7).all()


def test_reference_quantiser_against_the_oracle():
    """Where the oracle's fp32 steps are exact (a global scale of 2^k, block
    maxima of 6 * 2^n), both give the same bytes."""
    import oracle as O
    r = np.random.default_rng(3)
    y = r.standard_normal((40, 128)).astype(np.float32)
    y.reshape(40, 8, 16)[..., 3] = 6.0 * 2.0 ** r.integers(0, 3, (40, 8))
    bits = (y.view(np.uint32) >> 16).astype(np.uint16)
    p, sf = O.quant_nvfp4("bf16", bits, 2.0)
    c, s = kv_ref.nvfp4(pins.bits_to_f64(bits, "bf16"), 2.0)
    assert np.array_equal(s, sf.reshape(s.shape))
    assert np.array_equal(c[:, 0::2] | (c[:, 1::2] << 4), p)


def test_reference_store_and_load_round_trip():
    r = np.random.default_rng(4)
    pool = np.zeros((3, 2, 32 * 144), np.uint8)
    y = r.standard_normal((64, 2, 2, 128))
    want = np.empty((64, 2, 2, 128))
    for t in range(64):
        for h in range(2):
            kc, ks = kv_ref.nvfp4(y[t, h, 0], 3.0)
            vc, vs = kv_ref.nvfp4(y[t, h, 1], 5.0)
            page = (2, 0)[t // 32]
            kv_ref.store(pool, 32, page * 32 + t % 32, h, kc, ks, vc, vs)
            for k, (codes, sf, gs) in enumerate(((kc, ks, 3.0), (vc, vs, 5.0))):
                want[t, h, k] = pins.e2m1_table()[codes] * np.repeat(pins.e4m3_table()[sf], 16) / gs
    for h in range(2):
        k, v = kv_ref.load(pool, 32, [2, 0], 64, h, 3.0, 5.0)
        assert np.array_equal(k, want[:, h, 0]) and np.array_equal(v, want[:, h, 1])
    assert not pool[1].any()
