// rq_paged_attn.cuh -- what the two attention kernels over the paged NVFP4
// cache share: a sequence's queries and keys, conversions, the last step.
#pragma once

#include "rq_device.cuh"
#include "rq_launch.h"

namespace rq {

constexpr float kNoMax = -3.0e38f;  // running maximum before any key is seen
constexpr float kPMax = 32768.0f;   // a sum of exponentials beyond it moves the maximum
constexpr float kLeastScale = 1e-37f;  // of scores: -inf times it stays -inf

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

template <int B>
__device__ __forceinline__ uint32_t e2m1_pair(uint32_t w)  // byte B of w -> f16x2
{
    uint32_t d;
    if (B == 0) asm("{ .reg .b8 a, b, c, e; mov.b32 {a, b, c, e}, %1; cvt.rn.f16x2.e2m1x2 %0, a; }" : "=r"(d) : "r"(w));
    if (B == 1) asm("{ .reg .b8 a, b, c, e; mov.b32 {a, b, c, e}, %1; cvt.rn.f16x2.e2m1x2 %0, b; }" : "=r"(d) : "r"(w));
    if (B == 2) asm("{ .reg .b8 a, b, c, e; mov.b32 {a, b, c, e}, %1; cvt.rn.f16x2.e2m1x2 %0, c; }" : "=r"(d) : "r"(w));
    if (B == 3) asm("{ .reg .b8 a, b, c, e; mov.b32 {a, b, c, e}, %1; cvt.rn.f16x2.e2m1x2 %0, e; }" : "=r"(d) : "r"(w));
    return d;
}

// two E4M3 bytes (low half of w) -> f16x2
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t w)
{
    uint32_t d;
    asm("{ .reg .b16 h; cvt.u16.u32 h, %1; cvt.rn.f16x2.e4m3x2 %0, h; }" : "=r"(d) : "r"(w));
    return d;
}

// A sequence's queries (rows q0 .. q0 + nq - 1, the first at position
// first_pos) and the keys [lo, hi) that some of them see, lo a multiple of 16.
struct Seq {
    int q0, nq, first_pos, lo, hi;
};

__device__ __forceinline__ Seq load_seq(const PagedAttnParams &p, int b)
{
    Seq s;
    if (p.q_starts != nullptr) {
        const int a = ld_s32(p.q_starts + b), z = ld_s32(p.q_starts + b + 1);
        s.q0 = min(max(a, 0), (int)p.n_tokens);
        s.nq = min(max(z, s.q0), (int)p.n_tokens) - s.q0;
    } else {
        s.q0 = b;
        s.nq = 1;
    }
    s.hi = min(max(ld_s32(p.kv_lens + b), 0), p.max_keys);
    s.first_pos = s.hi - s.nq;
    s.lo = p.window > 0 ? max(0, s.first_pos - p.window + 1) & ~15 : 0;
    return s;
}

// A bf16 query row enters as fp16 times 2^-e, e the exponent of its largest
// element (kept where 2^e and 2^-e are normal).  {2^-e, 2^e} from that element.
__device__ __forceinline__ float2 row_power(float largest)
{
    const int e = min(max((int)(__float_as_uint(largest) >> 23) - 127, -126), 126);
    return make_float2(__uint_as_float((uint32_t)(127 - e) << 23), __uint_as_float((uint32_t)(127 + e) << 23));
}

// Factor of O for the output row: 1 / (l gs_v), 0 where no key was seen.
__device__ __forceinline__ float out_factor(float l, float v_gs)
{
    return l > 0.0f ? 1.0f / (l * v_gs) : (l == 0.0f ? 0.0f : l);
}

__device__ __forceinline__ float lse_of(float m, float l)
{
    return l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
}

// The workspace begins with counters of the tensor-memory kernel, set to 0 by the
// split kernel before it: the row blocks that its CTAs have taken, and the parts
// that are there of each block that several CTAs share, per warp.
constexpr int kSharedBlocks = 128;  // and parts of them; a part is 256 rows of O, m and l
constexpr size_t kTakenBytes = 16 + kSharedBlocks * 8 * sizeof(unsigned);
constexpr size_t kSharedPartBytes = 256 * 130 * sizeof(float);

template <typename DT>
cudaError_t launch_paged_attn_tc(const PagedAttnParams &p, size_t parts_at, cudaStream_t stream);

}  // namespace rq
