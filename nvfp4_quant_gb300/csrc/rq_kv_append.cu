// rq_kv_append.cu -- appends keys and values to a paged KV cache held in
// NVFP4: per-head Q/K RMSNorm, NeoX RoPE, Q in the dtype, K and V as E2M1
// codes with one E4M3 scale per 16 elements.
//
//   n = x rstd w (no weight: n = x);  o_i = n_i c_i - n_{i+64} s_i,
//   o_{i+64} = n_{i+64} c_i + n_i s_i;  Q: dt(o);  K: NVFP4(o);  V: NVFP4(v);
//   NVFP4 of a block of 16 with a = max |y|: sf = E4M3(gs a / 6), codes
//   E2M1(y gs / sf).
//
// Codes are decided by the real-valued formula, not by a sequence of fp32
// roundings: y is known to within a bound d (below), so each code is formed
// from both ends of [y - d, y + d], and where the two differ (a value next to
// a rounding border) the code is decided exactly: for V by one comparison of
// exact products, for K (about one step of four heads in a hundred) by forming
// the step again in double-float arithmetic.  The bytes of the cache therefore
// do not depend on the order of the fp32 sums.
//
// Mapping.  8 lanes own a head row: lane l holds elements 8 l .. 8 l + 7 and
// 64 + 8 l .. + 7 (two 16-byte loads), so a rotation pair (i, i + 64) lies in
// one lane and needs no exchange; the sum of squares is three shuffles, the
// maximum of a 16-element block one.  A warp takes 4 rows of one kind (Q, K or
// V heads of one token) a step and STEPS steps a unit, all of whose loads are
// issued first; the token's table row stays in registers for the unit.
//
// What bounds it: 256 (Hq + 2 Hk) bytes in and 256 Hq + 144 Hk out a token.
// 32,749 tokens of 32 + 8 heads (726 MB) take 143 us, 5.1 TB/s: the loads' latency
// at the 20 warps an SM that 96 registers allow (issue 54 %, ALU 45 %).  4096 of
// 16 + 8 take 20 us, of which 5 are a short launch's.
#include "rq_device.cuh"
#include "rq_launch.h"

#include <atomic>

namespace rq {

namespace {

constexpr int kAppendBlock = 128;
constexpr int kD = 128;

// Error of o in units of M rstd, M = max over the block of |t_i c| + |t_j s|
// (t = x w, exact in fp32), u = 2^-24: the rounded product and the FMA 2 u,
// the sum of squares (11 additions in a row, at most) and the root 9 u, the
// products with rstd, gs and 1 / sf (approximate reciprocals) 8 u: below
// 20 u.  V is only multiplied: below 5 u.
constexpr float kEpsK = 20 * 0x1p-24f;
constexpr float kEpsV = 6 * 0x1p-24f;

__device__ __forceinline__ float rsqrt_approx(float x)
{
    float r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float rcp_approx(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// ---- codes that the bound leaves open: the same step in double-float
// arithmetic (fp32 pairs, about 2^-44 of M; products of inputs exact), and
// each open code decided by comparing y gs with border * sf, both sides exact
// where the inputs make a tie possible.  (fp64 would do the same, but this
// GPU's few fp64 lanes took 10 us a step: 4096 tokens of 16 + 8 heads 213 us.)
__device__ __forceinline__ F2 f2_mul(const F2 &a, const F2 &b)
{
    F2 p = two_prod(a.h, b.h);
    p.l = __fmaf_rn(a.h, b.l, __fmaf_rn(a.l, b.h, p.l));
    return fast_two_sum(p.h, p.l);
}

__device__ __forceinline__ F2 f2_add(const F2 &a, const F2 &b)
{
    const F2 s = two_sum(a.h, b.h);
    return fast_two_sum(s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l)));
}

// |a| > t, or |a| == t and `tie`
__device__ __forceinline__ bool above(const F2 &a, float t, bool tie)
{
    const float l = a.h < 0.0f ? -a.l : a.l, h = fabsf(a.h);
    return h > t || (h == t && (l > 0.0f || (l == 0.0f && tie)));
}

// The border between E2M1 codes k and k + 1 (k < 7).
__device__ __forceinline__ float code_border(uint32_t k)
{
    return k < 4 ? 0.25f + 0.5f * k : (k == 4 ? 2.5f : (k == 5 ? 3.5f : 5.0f));
}

// 1 / sqrt(a): a Newton step, with its second-order term, from the approximate
// root; the residual 1 - a r^2 is formed in double-float.
__device__ __forceinline__ F2 f2_rsqrt(const F2 &a)
{
    const float r = rsqrt_approx(a.h);
    const F2 q = two_prod(r, r);
    F2 p = two_prod(a.h, q.h);
    p.l = __fmaf_rn(a.h, q.l, __fmaf_rn(a.l, q.h, p.l));
    const float e = __fsub_rn(__fsub_rn(1.0f, p.h), p.l);
    return fast_two_sum(r, __fmul_rn(r, __fmaf_rn(__fmul_rn(0.375f, e), e, __fmul_rn(0.5f, e))));
}

// Codes and scale byte of a block from its lane's 8 products y gs (the
// neighbouring lane has the others).
__device__ __forceinline__ uint32_t block_codes_exact(const F2 (&y)[8], uint32_t &sf)
{
    F2 a{0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const F2 v{fabsf(y[e].h), y[e].h < 0.0f ? -y[e].l : y[e].l};
        if (v.h > a.h || (v.h == a.h && v.l > a.l)) a = v;
    }
    const F2 o{__shfl_xor_sync(0xFFFFFFFFu, a.h, 1), __shfl_xor_sync(0xFFFFFFFFu, a.l, 1)};
    if (o.h > a.h || (o.h == a.h && o.l > a.l)) a = o;
    const float t = a.h * (1.0f / 6.0f);
    const uint32_t two = e4m3x2(t * (1.0f - 0x1p-20f), t * (1.0f + 0x1p-20f));
    sf = two & 0xFFu;
    if (sf != (two >> 8)) {  // next to the border between two scales
        const float border = 0.5f * (e4m3_value(sf) + e4m3_value(two >> 8));
        if (above(a, 6.0f * border, sf & 1)) sf = two >> 8;
    }
    const float f = e4m3_value(sf);
    const float enc = f > 0.0f ? rcp_approx(f) : 0.0f;
    float up[8], dn[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float v = fabsf(y[e].h) * enc;
        up[e] = v * (1.0f + 0x1p-20f);
        dn[e] = v * (1.0f - 0x1p-20f);
    }
    uint32_t c = e2m1x8(dn);
    const uint32_t open = c ^ e2m1x8(up);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if ((open >> (4 * e)) & 7u) {
            const uint32_t k = (c >> (4 * e)) & 7u;
            if (above(y[e], code_border(k) * f, k & 1)) c += 1u << (4 * e);
        }
        if (__float_as_uint(y[e].h) >> 31) c |= 8u << (4 * e);
    }
    return c;
}

// The codes of K row `head` of token tok, decided as above: {codes of elements
// 8 l .., codes of 64 + 8 l .., scale byte of the lower block, of the upper
// block}.  Every lane of the warp calls it (head past the last: any codes).  It
// reads the row again rather than take it, which keeps the common path's
// registers few.
template <typename DT>
__device__ __noinline__ uint4 key_codes_exact(const KVAppendParams &p, int64_t tok, int head, float gs)
{
    const int l = threadIdx.x & 7;
    uint4 xl = make_uint4(0, 0, 0, 0), xh = xl, wl = xl, wh = xl;
    if (head < p.hk) {
        const uint8_t *src = static_cast<const uint8_t *>(p.k) + (tok * p.k_stride + (int64_t)head * kD) * 2;
        xl = ld_stream16(src + l * 16);
        xh = ld_stream16(src + 128 + l * 16);
    }
    const bool normed = p.kw != nullptr;
    if (normed) {
        wl = ld_keep16(static_cast<const uint8_t *>(p.kw) + l * 16);
        wh = ld_keep16(static_cast<const uint8_t *>(p.kw) + 128 + l * 16);
    }
    int pos = ld_s32(p.pos + tok);
    pos = pos < 0 ? 0 : (pos >= p.max_pos ? (int)(p.max_pos - 1) : pos);
    const float *cs = p.cos_sin + (int64_t)pos * kD;
    const float eps = p.eps;
    float x0[8], x1[8];
    unpack8<DT>(xl, x0);
    unpack8<DT>(xh, x1);
    F2 ss{0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < 8; ++e) {  // squares are exact
        ss = f2_add(ss, F2{__fmul_rn(x0[e], x0[e]), 0.0f});
        ss = f2_add(ss, F2{__fmul_rn(x1[e], x1[e]), 0.0f});
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1)
        ss = f2_add(ss, F2{__shfl_xor_sync(0xFFFFFFFFu, ss.h, o), __shfl_xor_sync(0xFFFFFFFFu, ss.l, o)});
    F2 r{gs, 0.0f};
    if (normed) {
        const F2 mean = f2_add(F2{ss.h * (1.0f / kD), ss.l * (1.0f / kD)}, F2{eps, 0.0f});
        r = f2_mul(f2_rsqrt(mean), r);
        float w[8];
        unpack8<DT>(wl, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) x0[e] = __fmul_rn(x0[e], w[e]);  // exact
        unpack8<DT>(wh, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) x1[e] = __fmul_rn(x1[e], w[e]);
    }
    uint4 out;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        F2 y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float a = half ? x1[e] : x0[e], b = half ? x0[e] : -x1[e];
            const F2 p = two_prod(a, cs[8 * l + e]), q = two_prod(b, cs[64 + 8 * l + e]);
            y[e] = f2_mul(f2_add(p, q), r);
            if (y[e].h == 0.0f) y[e].h = copysignf(0.0f, __fadd_rn(p.h, q.h));
        }
        uint32_t sf;
        const uint32_t c = block_codes_exact(y, sf);
        if (half == 0) {
            out.x = c;
            out.z = sf;
        } else {
            out.y = c;
            out.w = sf;
        }
    }
    return out;
}

// Scale byte of a block from its largest magnitude a, known to +- d; `open` is
// set where a border lies within.
__device__ __forceinline__ uint32_t block_scale(float a, float d, float gs, uint32_t &next, bool &open)
{
    const float g6 = gs * (1.0f / 6.0f);
    const uint32_t two = e4m3x2((a - d) * g6, (a + d) * g6);
    next = two >> 8;
    open = (two & 0xFFu) != next;
    return two & 0xFFu;
}

__device__ __forceinline__ float max8(const float2 (&y)[4])
{
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) a = fmaxf(a, fmaxf(fabsf(y[i].x), fabsf(y[i].y)));
    return a;
}

__device__ __forceinline__ uint32_t e2m1x4p(const float2 (&v)[4])
{
    const float f[8] = {v[0].x, v[0].y, v[1].x, v[1].y, v[2].x, v[2].y, v[3].x, v[3].y};
    return e2m1x8(f);
}

// K: codes and scale byte of 8 of a block's 16 elements (the neighbouring lane
// holds the other 8), m the max over this lane's elements of the error bound's
// M.  `unsure`: a border lies within the bound.
__device__ __forceinline__ uint32_t key_codes(const float2 (&y)[4], float m, float gs, uint32_t &sf,
                                              bool &unsure)
{
    float a = max8(y);
    a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, 1));
    m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    uint32_t next;
    bool open;
    sf = block_scale(a, m * kEpsK, gs, next, open);
    const float f = e4m3_value(sf);
    const float enc = f > 0.0f ? gs * rcp_approx(f) : 0.0f;
    const float d = m * kEpsK * enc;
    const float2 enc2 = make_float2(enc, enc);
    float2 up[4], dn[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 s = make_float2(copysignf(d, y[i].x), copysignf(d, y[i].y));
        up[i] = __ffma2_rn(y[i], enc2, s);
        dn[i] = __ffma2_rn(y[i], enc2, make_float2(-s.x, -s.y));
    }
    // The code further from zero carries the sign of y (signed zeros
    // included).  Where the interval crosses zero its other end is below d:
    // that code is 0 unless d itself reaches the first border (a scale
    // saturated far below the block's maximum), which leaves the block open.
    const uint32_t c = e2m1x4p(up);
    unsure |= open || ((c ^ e2m1x4p(dn)) & 0x77777777u) != 0 || d >= 0.25f;
    return c;
}

// V: the same for elements that are inputs, whose products with gs are exact
// as pairs of floats: whatever the bound leaves open is decided here.  (V's
// few bits put one block in thirty next to a border, since gs usually is 2688
// over a dtype value.)
__device__ __forceinline__ uint32_t value_codes(const float2 (&y)[4], float gs, uint32_t &sf)
{
    float a = max8(y);
    a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, 1));
    uint32_t next;
    bool border;
    sf = block_scale(a, a * kEpsV, gs, next, border);
    if (border && above(two_prod(a, gs), 3.0f * (e4m3_value(sf) + e4m3_value(next)), sf & 1)) sf = next;
    const float f = e4m3_value(sf);
    const float enc = f > 0.0f ? gs * rcp_approx(f) : 0.0f;
    const float e1 = enc * (1.0f + kEpsV), e0 = enc * (1.0f - kEpsV);
    float2 up[4], dn[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        up[i] = __fmul2_rn(y[i], make_float2(e1, e1));
        dn[i] = __fmul2_rn(y[i], make_float2(e0, e0));
    }
    uint32_t c = e2m1x4p(dn), open = c ^ e2m1x4p(up);
    while (open != 0) {
        const int sh = (__ffs((int)open) - 1) & ~3;
        float v = y[0].x;
#pragma unroll
        for (int e = 1; e < 8; ++e) v = sh == 4 * e ? (e & 1 ? y[e / 2].y : y[e / 2].x) : v;
        const uint32_t k = (c >> sh) & 7u;
        if (above(two_prod(v, gs), code_border(k) * f, k & 1)) c += 1u << sh;
        open &= ~(7u << sh);
    }
    return c;
}

template <typename DT>
__device__ __forceinline__ void unpack4(const uint4 &v, float2 (&f)[4])
{
    f[0] = make_float2(DT::lo(v.x), DT::hi(v.x));
    f[1] = make_float2(DT::lo(v.y), DT::hi(v.y));
    f[2] = make_float2(DT::lo(v.z), DT::hi(v.z));
    f[3] = make_float2(DT::lo(v.w), DT::hi(v.w));
}

__device__ __forceinline__ void load_pairs(const float *src, float2 (&f)[4])
{
    const uint4 a = ld_keep16(src), b = ld_keep16(src + 4);
    f[0] = make_float2(__uint_as_float(a.x), __uint_as_float(a.y));
    f[1] = make_float2(__uint_as_float(a.z), __uint_as_float(a.w));
    f[2] = make_float2(__uint_as_float(b.x), __uint_as_float(b.y));
    f[3] = make_float2(__uint_as_float(b.z), __uint_as_float(b.w));
}

template <typename DT, int STEPS>
__global__ void __launch_bounds__(kAppendBlock, 5)
kv_append_kernel(const __grid_constant__ KVAppendParams p)
{
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, l = lane & 7, sub = lane >> 3;
    // steps of a token: 4 Q heads each, then 4 K heads, then 4 V heads
    const int q_steps = (p.hq + 3) >> 2, k_steps = (p.hk + 3) >> 2;
    const int v_first = q_steps + k_steps, steps = v_first + k_steps;
    const int units = (steps + STEPS - 1) / STEPS;
    const int64_t warp0 = ((int64_t)blockIdx.x * kAppendBlock + threadIdx.x) >> 5;
    const int64_t nwarps = ((int64_t)gridDim.x * kAppendBlock) >> 5;
    const float k_gs = p.hk > 0 ? ld_f32(p.k_gs) : 1.0f, v_gs = p.hk > 0 ? ld_f32(p.v_gs) : 1.0f;
    const int64_t step_tok = nwarps / units;
    const int step_g = (int)(nwarps - step_tok * units);
    int64_t tok = warp0 / units;
    int g = (int)(warp0 - tok * units);
    // Where the warps are a multiple of the units, a warp would meet the same
    // unit of every token, and those of K take longer than those of Q: its unit
    // then moves on by one a turn (all units of a token are in one turn).
    int turn = 0;
    while (tok < p.n_tokens) {
        const int unit = g + turn < units ? g + turn : g + turn - units;
        const int s0 = unit * STEPS;
        uint4 xl[STEPS], xh[STEPS];
#pragma unroll
        for (int u = 0; u < STEPS; ++u) {
            const int st = s0 + u;
            const bool is_q = st < q_steps, is_k = !is_q && st < v_first;
            const int h = (st - (is_q ? 0 : (is_k ? q_steps : v_first))) * 4 + sub;
            const void *base = is_q ? p.q : (is_k ? p.k : p.v);
            const int64_t stride = is_q ? p.q_stride : (is_k ? p.k_stride : p.v_stride);
            const uint8_t *src = static_cast<const uint8_t *>(base) + (tok * stride + (int64_t)h * kD) * 2;
            xl[u] = xh[u] = make_uint4(0, 0, 0, 0);
            if (st < steps && h < (is_q ? p.hq : p.hk)) {
                xl[u] = ld_stream16(src + l * 16);
                xh[u] = ld_stream16(src + 128 + l * 16);
            }
        }
        float2 c[4], s[4];
        const float *cs = nullptr;
        if (s0 < v_first) {
            int pos = ld_s32(p.pos + tok);
            pos = pos < 0 ? 0 : (pos >= p.max_pos ? (int)(p.max_pos - 1) : pos);
            cs = p.cos_sin + (int64_t)pos * kD;
            load_pairs(cs + 8 * l, c);
            load_pairs(cs + 64 + 8 * l, s);
        }
        // the token's group and row in the cache, head 0 (slots outside store
        // nothing)
        uint8_t *group = nullptr;
        int row = 0;
        if (s0 + STEPS > q_steps && p.hk > 0) {
            int64_t slot;
            asm volatile("ld.global.nc.s64 %0, [%1];" : "=l"(slot) : "l"(p.slots + tok));
            if (slot >= 0 && slot < p.num_slots) {
                const uint32_t at = (uint32_t)(slot >> 4), page = at / (uint32_t)p.groups;
                group = p.pool + ((int64_t)page * p.hk * p.groups + (at - page * p.groups)) * kKVGroupBytes;
                row = (int)(slot & 15);
            }
        }

#pragma unroll
        for (int u = 0; u < STEPS; ++u) {
            const int st = s0 + u;  // the same for the whole warp, as are the branches on it
            if (st >= steps) break;
            uint32_t c0, c1, f0, f1;
            int h, codes_at;
            float2 a[4], b[4];
            unpack4<DT>(xl[u], a);
            unpack4<DT>(xh[u], b);
            if (st < v_first) {
                const bool is_q = st < q_steps;
                h = (is_q ? st : st - q_steps) * 4 + sub;
                codes_at = kKVCodesK;
                const void *wp = is_q ? p.qw : p.kw;
                uint4 wl = make_uint4(0, 0, 0, 0), wh = wl;
                float rstd = 1.0f;
                if (wp != nullptr) {
                    wl = ld_keep16(static_cast<const uint8_t *>(wp) + l * 16);
                    wh = ld_keep16(static_cast<const uint8_t *>(wp) + 128 + l * 16);
                    float2 sq = make_float2(0.0f, 0.0f);
#pragma unroll
                    for (int i = 0; i < 4; ++i) sq = __ffma2_rn(b[i], b[i], __ffma2_rn(a[i], a[i], sq));
                    rstd = rsqrt_approx(fmaf(group_sum<8>(sq.x + sq.y), 1.0f / kD, p.eps));
                    float2 w[4];
                    unpack4<DT>(wl, w);
#pragma unroll
                    for (int i = 0; i < 4; ++i) a[i] = __fmul2_rn(a[i], w[i]);
                    unpack4<DT>(wh, w);
#pragma unroll
                    for (int i = 0; i < 4; ++i) b[i] = __fmul2_rn(b[i], w[i]);
                }
                const float2 r2 = make_float2(rstd, rstd);
                float m0 = 0.0f, m1 = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 bs = __fmul2_rn(b[i], s[i]), as = __fmul2_rn(a[i], s[i]);
                    const float2 nbs = make_float2(-bs.x, -bs.y);
                    if (!is_q) {
                        m0 = fmaxf(m0, fmaxf(fmaf(fabsf(a[i].x), fabsf(c[i].x), fabsf(bs.x)),
                                             fmaf(fabsf(a[i].y), fabsf(c[i].y), fabsf(bs.y))));
                        m1 = fmaxf(m1, fmaxf(fmaf(fabsf(b[i].x), fabsf(c[i].x), fabsf(as.x)),
                                             fmaf(fabsf(b[i].y), fabsf(c[i].y), fabsf(as.y))));
                    }
                    a[i] = __fmul2_rn(__ffma2_rn(a[i], c[i], nbs), r2);
                    b[i] = __fmul2_rn(__ffma2_rn(b[i], c[i], as), r2);
                }
                if (is_q) {
                    if (h < p.hq) {
                        uint8_t *q = static_cast<uint8_t *>(p.q_out) + (tok * p.hq + h) * (int64_t)(kD * 2);
                        st16(q + l * 16, make_uint4(DT::pack(a[0].x, a[0].y), DT::pack(a[1].x, a[1].y),
                                                    DT::pack(a[2].x, a[2].y), DT::pack(a[3].x, a[3].y)));
                        st16(q + 128 + l * 16, make_uint4(DT::pack(b[0].x, b[0].y), DT::pack(b[1].x, b[1].y),
                                                          DT::pack(b[2].x, b[2].y), DT::pack(b[3].x, b[3].y)));
                    }
                    continue;
                }
                bool unsure = false;
                c0 = key_codes(a, m0 * rstd, k_gs, f0, unsure);
                c1 = key_codes(b, m1 * rstd, k_gs, f1, unsure);
                if (__any_sync(0xFFFFFFFFu, unsure)) {
                    const uint4 r = key_codes_exact<DT>(p, tok, h, k_gs);
                    c0 = r.x;
                    c1 = r.y;
                    f0 = r.z;
                    f1 = r.w;
                }
            } else {
                h = (st - v_first) * 4 + sub;
                codes_at = kKVCodesV;
                c0 = value_codes(a, v_gs, f0);
                c1 = value_codes(b, v_gs, f1);
            }
            if (h < p.hk && group != nullptr) {
                uint8_t *d = group + (int64_t)h * p.groups * kKVGroupBytes;
                uint8_t *codes = d + codes_at + row * 64 + l * 4;
                st4(codes, c0);
                st4(codes + 32, c1);
                if ((l & 1) == 0) {
                    uint8_t *sc = d + (codes_at == kKVCodesK ? kKVScalesK : kKVScalesV) + row * 8 + (l >> 1);
                    st1(sc, f0);
                    st1(sc + 4, f1);
                }
            }
        }
        if (step_g == 0 && ++turn == units) turn = 0;
        tok += step_tok;
        g += step_g;
        if (g >= units) {
            g -= units;
            ++tok;
        }
    }
}

// Steps of 4 head rows that a token takes.
int64_t steps_of(const KVAppendParams &p) { return (p.hq + 3) / 4 + 2 * (((int64_t)p.hk + 3) / 4); }

template <typename DT, int STEPS>
cudaError_t launch_steps(const KVAppendParams &p, int dev, cudaStream_t stream)
{
    static std::atomic<int> occ_cache[64];
    auto kern = kv_append_kernel<DT, STEPS>;
    int per_sm = dev < 64 ? occ_cache[dev].load(std::memory_order_relaxed) : 0;
    if (per_sm <= 0) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kAppendBlock, 0) != cudaSuccess ||
            per_sm < 1)
            per_sm = 1;
        if (dev < 64) occ_cache[dev].store(per_sm, std::memory_order_relaxed);
    }
    const int64_t units = (steps_of(p) + STEPS - 1) / STEPS;
    const int64_t need = (p.n_tokens * units * 32 + kAppendBlock - 1) / kAppendBlock;
    const int64_t full = (int64_t)device_sms(dev) * per_sm;
    return launch_pdl(kern, (unsigned)(need < full ? need : full), kAppendBlock, 0, stream, p);
}

}  // namespace

template <typename DT>
cudaError_t launch_kv_append(const KVAppendParams &p, cudaStream_t stream)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    // Few steps: one a warp, so that they spread over the SMs (1, 64, 256 and 600
    // tokens of 16 + 8 heads 2.2, 4.7, 5.5 and 6.5 us, with two a unit 2.7, 5.6, 6.2
    // and 6.8; 1200 tokens 9.7 and 8.9).  Otherwise two
    // a unit at 20 warps an SM (measured, 4096 tokens of 16 + 8 heads and
    // 32,749 of 32 + 8: 19.8 and 142 us; at 16 warps 20.1 and 147, at 24, with
    // more spills, 20.5 and 142; one step a unit 20.4 and 170, four 22.5 and
    // 149).
    return p.n_tokens * steps_of(p) < (int64_t)device_sms(dev) * 32
               ? launch_steps<DT, 1>(p, dev, stream)
               : launch_steps<DT, 2>(p, dev, stream);
}

template cudaError_t launch_kv_append<BF16>(const KVAppendParams &, cudaStream_t);
template cudaError_t launch_kv_append<FP16>(const KVAppendParams &, cudaStream_t);

}  // namespace rq
