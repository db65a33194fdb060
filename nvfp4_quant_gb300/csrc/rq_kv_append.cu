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
// a rounding border, about one step of four heads in a hundred) the warp
// forms the step again in double precision.  The bytes of the cache therefore
// do not depend on the order of the fp32 sums.
//
// Mapping.  8 lanes own a head row: lane l holds elements 8 l .. 8 l + 7 and
// 64 + 8 l .. + 7 (two 16-byte loads), so a rotation pair (i, i + 64) lies in
// one lane and needs no exchange; the sum of squares is three shuffles, the
// maximum of a 16-element block one.  A warp takes 4 rows a step and up to
// 4 * STEPS rows (Q heads, then K heads, then V heads of one token) a unit,
// all of whose loads are issued first; the token's table row stays in
// registers for the unit.
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
constexpr float kEpsK = 0x1p-19f;  // 32 u
constexpr float kEpsV = 0x1p-21f;  // 8 u

// A double as an fp32 value that rounds on to any shorter format as the double
// itself would: truncated, with the last bit set where bits were lost (round
// to odd; Boldo and Melquiond, "Emulation of a FMA and correctly rounded sums:
// proved algorithms using rounding to odd", IEEE Trans. Comput. 57(4), 2008).
__device__ __forceinline__ float to_odd(double d)
{
    const float f = __double2float_rz(d);
    return (double)f != d ? __uint_as_float(__float_as_uint(f) | 1u) : f;
}

// The step's codes in double precision: {codes of elements 8 l .., codes of 64
// + 8 l .., scale byte of the lower block, of the upper block}.  Every lane of
// the warp calls it.
template <typename DT>
__device__ __noinline__ uint4 append_codes_f64(uint4 xl, uint4 xh, uint4 wl, uint4 wh, bool normed,
                                               bool rotated, const float *cs, float eps, float gs)
{
    const int l = threadIdx.x & 7;
    float x[16], w[16];
    unpack8<DT>(xl, *reinterpret_cast<float(*)[8]>(x));
    unpack8<DT>(xh, *reinterpret_cast<float(*)[8]>(x + 8));
    unpack8<DT>(wl, *reinterpret_cast<float(*)[8]>(w));
    unpack8<DT>(wh, *reinterpret_cast<float(*)[8]>(w + 8));
    double ss = 0.0;
#pragma unroll
    for (int e = 0; e < 16; ++e) ss += (double)x[e] * x[e];
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
    const double rstd = normed ? 1.0 / sqrt(ss / kD + (double)eps) : 1.0;
    double y[16], lo = 0.0, hi = 0.0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const double a = normed ? (double)x[e] * w[e] : (double)x[e];
        const double b = normed ? (double)x[e + 8] * w[e + 8] : (double)x[e + 8];
        double c = 1.0, s = 0.0;
        if (rotated) {
            c = cs[8 * l + e];
            s = cs[64 + 8 * l + e];
        }
        y[e] = rotated ? (a * c - b * s) * rstd : a;
        y[e + 8] = rotated ? (b * c + a * s) * rstd : b;
        lo = fmax(lo, fabs(y[e]));
        hi = fmax(hi, fabs(y[e + 8]));
    }
    lo = fmax(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, 1));
    hi = fmax(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, 1));
    const uint32_t sl = e4m3x2(to_odd(lo * gs / 6.0), 0.0f) & 0xFF;
    const uint32_t sh = e4m3x2(to_odd(hi * gs / 6.0), 0.0f) & 0xFF;
    const float fl = e4m3_value(sl), fh = e4m3_value(sh);
    float vl[8], vh[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        vl[e] = fl > 0.0f ? to_odd(y[e] * gs / fl) : copysignf(0.0f, (float)y[e]);
        vh[e] = fh > 0.0f ? to_odd(y[e + 8] * gs / fh) : copysignf(0.0f, (float)y[e + 8]);
    }
    return make_uint4(e2m1x8(vl), e2m1x8(vh), sl, sh);
}

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

// Codes and scale byte of 8 of a block's 16 elements (the neighbouring lane
// holds the other 8).  m: max over this lane's elements of the error bound's
// M; eps: its factor.  `unsure` is set where a border lies within the bound.
__device__ __forceinline__ uint32_t block_codes(const float (&y)[8], float m, float eps, float gs,
                                                uint32_t &sf, bool &unsure)
{
    float a = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) a = fmaxf(a, fabsf(y[e]));
    a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, 1));
    m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    const float d = m * eps, g6 = gs * (1.0f / 6.0f);
    const uint32_t two = e4m3x2((a - d) * g6, (a + d) * g6);
    sf = two & 0xFFu;
    unsure |= sf != (two >> 8);
    const float f = e4m3_value(sf);
    const float enc = f > 0.0f ? gs * rcp_approx(f) : 0.0f;
    const float dv = d * enc;
    float up[8], dn[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float v = y[e] * enc, s = copysignf(dv, y[e]);
        up[e] = v + s;
        dn[e] = v - s;
    }
    // the code further from zero carries the sign of y (signed zeros
    // included).  Where the interval crosses zero the other end is below dv:
    // its code is 0 unless dv itself reaches the first border (a scale
    // saturated far below the block's maximum), which leaves the block open.
    const uint32_t c = e2m1x8(up);
    unsure |= ((c ^ e2m1x8(dn)) & 0x77777777u) != 0 || dv >= 0.25f;
    return c;
}

template <typename DT, int STEPS>
__global__ void __launch_bounds__(kAppendBlock)
kv_append_kernel(const KVAppendParams p)
{
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, l = lane & 7, sub = lane >> 3;
    const int rows = p.hq + 2 * p.hk;
    const int turned = p.hq + p.hk;  // rows that are rotated
    const int units = (rows + 4 * STEPS - 1) / (4 * STEPS);
    const int64_t warp0 = ((int64_t)blockIdx.x * kAppendBlock + threadIdx.x) >> 5;
    const int64_t nwarps = ((int64_t)gridDim.x * kAppendBlock) >> 5;
    const float k_gs = p.hk > 0 ? ld_f32(p.k_gs) : 1.0f, v_gs = p.hk > 0 ? ld_f32(p.v_gs) : 1.0f;
    const int64_t step_tok = nwarps / units;
    const int step_g = (int)(nwarps - step_tok * units);
    int64_t tok = warp0 / units;
    int g = (int)(warp0 - tok * units);
    while (tok < p.n_tokens) {
        const int h0 = g * 4 * STEPS;
        uint4 xl[STEPS], xh[STEPS];
#pragma unroll
        for (int u = 0; u < STEPS; ++u) {
            const int h = h0 + 4 * u + sub;
            const uint8_t *src =
                h < p.hq    ? static_cast<const uint8_t *>(p.q) + (tok * p.q_stride + (int64_t)h * kD) * 2
                : h < turned ? static_cast<const uint8_t *>(p.k) +
                                  (tok * p.k_stride + (int64_t)(h - p.hq) * kD) * 2
                            : static_cast<const uint8_t *>(p.v) +
                                  (tok * p.v_stride + (int64_t)(h - turned) * kD) * 2;
            xl[u] = xh[u] = make_uint4(0, 0, 0, 0);
            if (h < rows) {
                xl[u] = ld_stream16(src + l * 16);
                xh[u] = ld_stream16(src + 128 + l * 16);
            }
        }
        float2 c[4], s[4];
        const float *cs = nullptr;
        if (h0 < turned) {
            int pos = ld_s32(p.pos + tok);
            pos = pos < 0 ? 0 : (pos >= p.max_pos ? (int)(p.max_pos - 1) : pos);
            cs = p.cos_sin + (int64_t)pos * kD;
            const uint4 c0 = ld_keep16(cs + 8 * l), c1 = ld_keep16(cs + 8 * l + 4);
            const uint4 s0 = ld_keep16(cs + 64 + 8 * l), s1 = ld_keep16(cs + 64 + 8 * l + 4);
            c[0] = make_float2(__uint_as_float(c0.x), __uint_as_float(c0.y));
            c[1] = make_float2(__uint_as_float(c0.z), __uint_as_float(c0.w));
            c[2] = make_float2(__uint_as_float(c1.x), __uint_as_float(c1.y));
            c[3] = make_float2(__uint_as_float(c1.z), __uint_as_float(c1.w));
            s[0] = make_float2(__uint_as_float(s0.x), __uint_as_float(s0.y));
            s[1] = make_float2(__uint_as_float(s0.z), __uint_as_float(s0.w));
            s[2] = make_float2(__uint_as_float(s1.x), __uint_as_float(s1.y));
            s[3] = make_float2(__uint_as_float(s1.z), __uint_as_float(s1.w));
        }
        // where the token's K and V rows of head 0 start (slots outside the
        // cache store nothing)
        uint8_t *dst = nullptr;
        int row16 = 0;
        if (h0 + 4 * STEPS > p.hq && p.hk > 0) {
            int64_t slot;
            asm volatile("ld.global.nc.s64 %0, [%1];" : "=l"(slot) : "l"(p.slots + tok));
            if (slot >= 0 && slot < p.num_slots) {
                const uint32_t group = (uint32_t)(slot >> 4), page = group / (uint32_t)p.groups;
                dst = p.pool + ((int64_t)page * p.hk * p.groups + (group - page * p.groups)) * kKVGroupBytes +
                      (slot & 15) * 64;
                row16 = (int)(slot & 15);
            }
        }

#pragma unroll
        for (int u = 0; u < STEPS; ++u) {
            const int hu = h0 + 4 * u, h = hu + sub;
            if (hu >= rows) break;
            const bool is_q = h < p.hq, is_v = h >= turned;
            float y0[8], y1[8];
            unpack8<DT>(xl[u], y0);
            unpack8<DT>(xh[u], y1);
            float m0 = 0.0f, m1 = 0.0f, eps = kEpsV;
            const void *wp = is_q ? p.qw : p.kw;
            const bool normed = !is_v && wp != nullptr;
            uint4 wl = make_uint4(0, 0, 0, 0), wh = wl;
            if (hu < turned) {
                float2 a[4], b[4];
                float2 sq = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    a[i] = make_float2(y0[2 * i], y0[2 * i + 1]);
                    b[i] = make_float2(y1[2 * i], y1[2 * i + 1]);
                    sq = __ffma2_rn(a[i], a[i], sq);
                    sq = __ffma2_rn(b[i], b[i], sq);
                }
                const float ss = group_sum<8>(sq.x + sq.y);
                const float rstd = normed ? rsqrt_approx(fmaf(ss, 1.0f / kD, p.eps)) : 1.0f;
                const float2 r2 = make_float2(rstd, rstd);
                if (normed) {
                    wl = ld_keep16(static_cast<const uint8_t *>(wp) + l * 16);
                    wh = ld_keep16(static_cast<const uint8_t *>(wp) + 128 + l * 16);
                    float w[8];
                    unpack8<DT>(wl, w);
#pragma unroll
                    for (int i = 0; i < 4; ++i) a[i] = __fmul2_rn(a[i], make_float2(w[2 * i], w[2 * i + 1]));
                    unpack8<DT>(wh, w);
#pragma unroll
                    for (int i = 0; i < 4; ++i) b[i] = __fmul2_rn(b[i], make_float2(w[2 * i], w[2 * i + 1]));
                }
                if (!is_v) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 bs = __fmul2_rn(b[i], s[i]), as = __fmul2_rn(a[i], s[i]);
                        const float2 lo = __fmul2_rn(__ffma2_rn(a[i], c[i], make_float2(-bs.x, -bs.y)), r2);
                        const float2 hi = __fmul2_rn(__ffma2_rn(b[i], c[i], as), r2);
                        y0[2 * i] = lo.x;
                        y0[2 * i + 1] = lo.y;
                        y1[2 * i] = hi.x;
                        y1[2 * i + 1] = hi.y;
                        if (!is_q) {
                            m0 = fmaxf(m0, fmaxf(fmaf(fabsf(a[i].x), fabsf(c[i].x), fabsf(bs.x)),
                                                 fmaf(fabsf(a[i].y), fabsf(c[i].y), fabsf(bs.y))));
                            m1 = fmaxf(m1, fmaxf(fmaf(fabsf(b[i].x), fabsf(c[i].x), fabsf(as.x)),
                                                 fmaf(fabsf(b[i].y), fabsf(c[i].y), fabsf(as.y))));
                        }
                    }
                    m0 *= rstd;
                    m1 *= rstd;
                    eps = kEpsK;
                }
            }
            if (is_q) {
                uint8_t *q = static_cast<uint8_t *>(p.q_out) + (tok * p.hq + h) * (int64_t)(kD * 2);
                st16(q + l * 16, pack8<DT>(y0));
                st16(q + 128 + l * 16, pack8<DT>(y1));
            }
            if (hu + 3 < p.hq) continue;  // four Q rows
            if (is_v) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    m0 = fmaxf(m0, fabsf(y0[e]));
                    m1 = fmaxf(m1, fabsf(y1[e]));
                }
            }
            const float gs = is_v ? v_gs : k_gs;
            bool unsure = false;
            uint32_t f0, f1;
            uint32_t c0 = block_codes(y0, m0, eps, gs, f0, unsure);
            uint32_t c1 = block_codes(y1, m1, eps, gs, f1, unsure);
            if (__any_sync(0xFFFFFFFFu, unsure && !is_q && h < rows)) {
                const uint4 r = append_codes_f64<DT>(xl[u], xh[u], wl, wh, normed, !is_v, cs, p.eps, gs);
                c0 = r.x;
                c1 = r.y;
                f0 = r.z;
                f1 = r.w;
            }
            if (!is_q && h < rows && dst != nullptr) {
                uint8_t *d = dst + (int64_t)(is_v ? h - turned : h - p.hq) * p.groups * kKVGroupBytes;
                uint8_t *codes = d + (is_v ? kKVCodesV : kKVCodesK);
                st4(codes + l * 4, c0);
                st4(codes + 32 + l * 4, c1);
                if ((l & 1) == 0) {  // scales: 8 bytes a token (the codes' row is 64)
                    uint8_t *sc = d - row16 * 56 + (is_v ? kKVScalesV : kKVScalesK);
                    st1(sc + (l >> 1), f0);
                    st1(sc + 4 + (l >> 1), f1);
                }
            }
        }
        tok += step_tok;
        g += step_g;
        if (g >= units) {
            g -= units;
            ++tok;
        }
    }
}

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
    const int64_t units = (p.hq + 2 * (int64_t)p.hk + 4 * STEPS - 1) / (4 * STEPS);
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
    // few rows: one step a warp, so that they spread over the SMs
    const int64_t rows = p.n_tokens * (p.hq + 2 * (int64_t)p.hk);
    return rows < (int64_t)device_sms(dev) * 128 ? launch_steps<DT, 1>(p, dev, stream)
                                                : launch_steps<DT, 4>(p, dev, stream);
}

template cudaError_t launch_kv_append<BF16>(const KVAppendParams &, cudaStream_t);
template cudaError_t launch_kv_append<FP16>(const KVAppendParams &, cudaStream_t);

}  // namespace rq
