// rq_paged_attn_tc.cu -- attention over the paged NVFP4 cache for runs of
// queries (prompts, chunks), on the fifth-generation tensor cores.
//
// A CTA takes blocks of 256 rows (query, head of the KV head's group) of a
// sequence, one after another, as two tiles of 128 and walks the keys in tiles
// of 128.  Per tile of keys:
//   S_t = Q_t K^T        tcgen05.mma, both operands in shared memory,
//   P_t = 2^(S_t c - m)  a thread a row, from and to tensor memory (the fp16 P
//                        over S's own columns),
//   O_t += P_t V         tcgen05.mma, P from tensor memory, V from shared,
// with S and O of both tiles in all 512 tensor-memory columns.  Roles:
//   warps 0-3, 4-7   the rows of tile 0, tile 1: softmax, the last step, and the
//                    next block's queries
//   warps 8-11       a token each: codes from global memory (one tile ahead in
//                    registers), decoded to fp16 rows in shared memory
//   warp 12          issues the products: PV_0(j) QK_0(j+1) PV_1(j) QK_1(j+1),
//                    so that one tile's softmax runs under the other's products
//   warp 13          finds the next block (a counter that all CTAs share)
// m is the row's maximum when it was last looked at.  That is when a tile's sum
// of P passes kPMax (so no P exceeds it, and fp16 holds them all): the row's O
// is then rescaled in tensor memory, after the product before.  Between, no
// maximum is formed.
//
// What bounds it: 4 * 128 flops a visible pair on the tensor cores.  The
// operands of a 128 x 128 x 16 product are 8 KB of shared memory in its 64
// clocks (4 KB with P in tensor memory), the decoded tile another 32 bytes a
// clock, and the exponentials need half the time of the products.  A tile takes
// about 2900 clocks where its products take 2048: S waits 1350 for the product
// with V, its own and the signals, P 1550 for the softmax.  Without exponentials
// and decoding it still took 2500.  8192 tokens of 32 + 8 heads: 376 us, 1460
// TFLOP/s.
//
// From a block's last P to the next block's first scores it is 9000 clocks (last
// product 2200, output 4000, queries into the tiles 1800, product 1000), from a
// CTA's start 12,000 to 15,000: one CTA a block took that each time (8 prompts of
// 1024 tokens 58 us, 55 like this).  The code is long for the instruction caches:
// what few tiles need is kept out of the loop over the keys (with the masks inline
// 8192 tokens took 417 us).
//
// Every wait has a time limit (kWaitNs): past it the CTA gives up, writes NaN
// for its block and leaves, tensor memory freed.  No valid call meets it.
#include "rq_paged_attn.cuh"

#include <atomic>
#include <type_traits>

namespace rq {

namespace {

constexpr int kD = 128, kTile = 128, kRows = 2 * kTile;
constexpr int kThreads = 14 * 32;
constexpr uint32_t kTileBytes = kTile * kD * 2;  // 32 KB
// shared memory (from a 1024-byte boundary): Q0 Q1 K[2] V[2], then the small part
constexpr uint32_t kQ = 0, kK = 2 * kTileBytes, kV = kK + 2 * kTileBytes, kSmall = kV + 2 * kTileBytes;
constexpr int kPartTiles = 8;  // tiles of keys that a part has at least
constexpr unsigned long long kWaitNs = 1000000000ull;

struct TcParams : PagedAttnParams {
    unsigned limit;  // row blocks, at most
    int width;       // the window, or more than any sequence has
    size_t parts_at; // of the parts, behind the counters
};

// A block of rows: its sequence and KV head, the rows row0 .. row0 + rows - 1 of
// the sequence (none: there is no more work), and the keys [first, hi) that some
// of them see, in n tiles from lo; or one of the parts of a block whose keys
// several CTAs share (parts 0: the others have it all).
struct Work {
    int seq, head, q0, first_pos, row0, rows, lo, first, hi, n, parts, part, shared, slot;
};

struct Small {
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], pv_done[2], q_full[2], drained;
    uint64_t work_full[2], work_empty[2], claim;
    alignas(16) uint32_t seen[4][4];  // tile's readable tokens, ring of 4
    Work work[2];
    uint32_t tmem;
    int failed;
    float k_gs, v_gs;
    int64_t scan[14];
    int64_t upto[kThreads];  // row blocks of the sequences up to the thread's last
};
constexpr size_t kSmemBytes = 1024 + kSmall + sizeof(Small);

// tensor memory columns: S0 S1 O0 O1
constexpr uint32_t kColS = 0, kColO = 256;

// kind::f16 instruction descriptor: fp32 accumulator, fp16 operands, M = 128,
// N = 128; bit 16: B is N-major (V).
constexpr uint32_t kIdescQK = (1u << 4) | ((128u / 8) << 17) | ((128u / 16) << 24);
constexpr uint32_t kIdescPV = kIdescQK | (1u << 16);

// Shared-memory operand descriptor, 128-byte swizzle (rows of 64 fp16, 8 rows
// a kilobyte): K-major operands step 1 KB every 8 rows; N-major ones (V, rows
// are keys) 1 KB every 8 keys and 16 KB from channels 0-63 to 64-127.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t leading)
{
    return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)(leading >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile("{ .reg .pred p; setp.ne.u32 p, %4, 0;\n"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }"
                 :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile("{ .reg .pred p; setp.ne.u32 p, %4, 0;\n"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }"
                 :: "r"(d), "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add) : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                 :: "r"(bar) : "memory");
}
__device__ __forceinline__ void tm_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tm_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void async_proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 32 columns of the warp's 32 rows; the values are there after tm_wait_ld,
// which takes them as operands so that no use moves above it.
__device__ __forceinline__ void tm_load32(uint32_t addr, uint32_t (&v)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]),
          "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]),
          "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]),
          "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(addr));
}
__device__ __forceinline__ void tm_wait_ld(uint32_t (&v)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]),
                   "+r"(v[15]), "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]),
                   "+r"(v[22]), "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]),
                   "+r"(v[29]), "+r"(v[30]), "+r"(v[31])
                 :: "memory");
}
__device__ __forceinline__ void tm_store32(uint32_t addr, const uint32_t *v)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
        :: "r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
           "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
           "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]),
           "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}
__device__ __forceinline__ void bar_init(uint64_t *bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" :: "r"(smem_addr(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(bar) : "memory");
}
__device__ __forceinline__ unsigned long long now_ns()
{
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
// Waits until the barrier's phase of the given parity is over; gives up after
// a time, or when another role of the CTA has (false).
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int *failed,
                                         unsigned long long limit)
{
    unsigned long long start = 0;
    for (uint32_t n = 0;; ++n) {
        uint32_t done;
        asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                     : "=r"(done) : "r"(bar), "r"(parity) : "memory");
        if (done) return true;
        if ((n & 63) == 63) {
            if (*failed) return false;
            const unsigned long long t = now_ns();
            if (start == 0) start = t;
            if (t - start > limit) {
                *failed = 1;
                return false;
            }
        }
    }
}

__device__ __forceinline__ bool elect_one()
{
    uint32_t one;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xFFFFFFFF; selp.u32 %0, 1, 0, p; }" : "=r"(one));
    return one != 0;
}

// The same for a whole warp: every lane gets one answer.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *failed,
                                          unsigned long long limit = kWaitNs)
{
    return __all_sync(0xFFFFFFFFu, bar_wait(bar, parity, failed, limit));
}

// Whether it is over already.
__device__ __forceinline__ bool warp_test(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile("{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                 : "=r"(done) : "r"(bar), "r"(parity) : "memory");
    return __all_sync(0xFFFFFFFFu, done);
}

// Row tiles of the sequence for this kernel.
__device__ __forceinline__ int row_blocks(const PagedAttnParams &p, const Seq &s)
{
    const int rows = s.nq * p.per;
    return rows > p.few ? (rows + kRows - 1) / kRows : 0;
}

// A key or value row of a tile: 64 bytes of codes and 8 scales in registers,
// and whether it is one (else its values are 0).
struct Row {
    uint4 c[4];
    uint2 f;
    bool there;
};

__device__ __forceinline__ void load_row(Row &r, const uint8_t *codes, const uint8_t *scales)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) r.c[i] = ld_keep16(codes + 16 * i);
    asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];" : "=r"(r.f.x), "=r"(r.f.y) : "l"(scales));
}

// Decodes into the row at shared address `to` (swizzled: `to` holds (row & 7)
// << 4 in the bits that the chunk's number is xored into), 32 channels at a time
// in the order that keeps uses away from what they wait for.
__device__ __forceinline__ void decode_row(const Row &r, uint32_t to)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w[4] = {r.c[i].x, r.c[i].y, r.c[i].z, r.c[i].w};
        const uint32_t two = e4m3_pair((r.there ? ((i & 2) ? r.f.y : r.f.x) : 0u) >> ((i & 1) * 16));
        const uint32_t f[2] = {__byte_perm(two, two, 0x1010), __byte_perm(two, two, 0x3232)};
        uint32_t x[16];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            x[4 * c] = e2m1_pair<0>(w[c]);
            x[4 * c + 1] = e2m1_pair<1>(w[c]);
            x[4 * c + 2] = e2m1_pair<2>(w[c]);
            x[4 * c + 3] = e2m1_pair<3>(w[c]);
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) x[k] = FP16::mul2(x[k], f[k >> 3]);
#pragma unroll
        for (int c = 0; c < 4; ++c)
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};"
                         :: "r"((to ^ ((4 * (i & 1) + c) << 4)) + (i >> 1) * (kTileBytes / 2)), "r"(x[4 * c]),
                            "r"(x[4 * c + 1]), "r"(x[4 * c + 2]), "r"(x[4 * c + 3]) : "memory");
    }
}

// A producer thread's token of each tile: where it lies, from tile to tile
// without a division, and the page id of one tile further ahead.
struct Feed {
    int tok, first, hi, at, page, in, pages, rest, id;
    const int32_t *table;
    const uint8_t *pool;
    int64_t page_bytes;

    // of the token, or of the sequence's first page where it has none
    __device__ __forceinline__ int page_id() const { return ld_s32(table + (at < hi ? page : 0)); }

    __device__ __forceinline__ void start(const PagedAttnParams &p, int seq, int head, int lo, int first_, int hi_,
                                          int tok_)
    {
        tok = tok_;
        first = first_;
        hi = hi_;
        at = lo + tok;
        page = (at >> 4) / p.groups;
        in = (at >> 4) - page * p.groups;
        pages = 8 / p.groups;  // a tile is 8 groups
        rest = 8 - pages * p.groups;
        table = p.table + (int64_t)seq * p.table_stride;
        pool = p.pool + (int64_t)head * p.groups * kKVGroupBytes;
        page_bytes = (int64_t)p.hk * p.groups * kKVGroupBytes;
        id = page_id();
    }

    // The group of the tile's token, or, where there is none that can be read,
    // of other memory (a load under a condition would be waited for at once);
    // on to the next tile.
    __device__ __forceinline__ const uint8_t *step(const PagedAttnParams &p, bool &there)
    {
        there = at >= first && at < hi && id >= 0 && id < p.num_pages;
        const uint8_t *g = there ? pool + id * page_bytes + in * kKVGroupBytes : p.workspace;
        at += kTile;
        page += pages;
        in += rest;
        if (in >= p.groups) {
            in -= p.groups;
            ++page;
        }
        id = page_id();
        return g;
    }

    __device__ __forceinline__ void load(Row &r, const uint8_t *g, bool there, int codes, int scales) const
    {
        load_row(r, g + codes + (tok & 15) * 64, g + scales + (tok & 15) * 8);
        r.there = there;
    }
};

// 32 channels of a row's sums into the tile as the output's.
template <typename DT>
__device__ __forceinline__ void put_out(uint32_t tile, int r, int c, const uint32_t (&y)[32], float inv)
{
#pragma unroll
    for (int k = 0; k < 32; k += 8) {
        float e[8];
#pragma unroll
        for (int n = 0; n < 8; ++n) e[n] = inv == 0.0f ? 0.0f : __uint_as_float(y[k + n]) * inv;
        const uint4 v = pack8<DT>(e);
        const int chunk = 4 * c + k / 8;
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};"
                     :: "r"(tile + (chunk >> 3) * (kTileBytes / 2) + r * 128 + (((chunk & 7) ^ (r & 7)) << 4)),
                        "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
    }
}

// A part of a block whose keys several CTAs share: a row's O, m and l go to
// the workspace (4 channels of all rows together).  The warp that finds all the
// others' there joins them in the order of the keys and puts the output into the
// tile.  (Not inline: the kernel's main loop has no register to spare.)
struct Joined {
    float m, l;
    bool last;
};
template <typename DT>
__device__ __noinline__ Joined share_part(uint8_t *part0, unsigned *there, int mine, int parts, int row, uint32_t o_at,
                                          uint32_t tile, int r, float m, float l, float v_gs)
{
    constexpr int kPart = kSharedPartBytes / sizeof(float4);
    float4 *const rows0 = reinterpret_cast<float4 *>(part0) + row;
    float2 *const ml0 = reinterpret_cast<float2 *>(reinterpret_cast<float4 *>(part0) + 32 * kRows) + row;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
        uint32_t y[32];
        tm_load32(o_at + 32 * c, y);
        tm_wait_ld(y);
#pragma unroll
        for (int k = 0; k < 32; k += 4)
            __stcg(rows0 + mine * kPart + (8 * c + k / 4) * kRows,
                   l == 0.0f ? make_float4(0.0f, 0.0f, 0.0f, 0.0f)
                             : make_float4(__uint_as_float(y[k]), __uint_as_float(y[k + 1]),
                                           __uint_as_float(y[k + 2]), __uint_as_float(y[k + 3])));
    }
    __stcg(ml0 + mine * (2 * kPart), make_float2(m, l));
    __threadfence();
    __syncwarp();
    unsigned before = 0;
    if ((threadIdx.x & 31) == 0) before = atomicAdd(there, 1u);
    Joined j = {m, l, __shfl_sync(0xFFFFFFFFu, before, 0) == (unsigned)parts - 1};
    if (!j.last) return j;
    __threadfence();
    j.m = kNoMax;
    j.l = 0.0f;
    for (int n = 0; n < parts; ++n) j.m = fmaxf(j.m, __ldcg(ml0 + n * (2 * kPart)).x);
    for (int n = 0; n < parts; ++n) {
        const float2 ml = __ldcg(ml0 + n * (2 * kPart));
        j.l = fmaf(ex2(ml.x - j.m), ml.y, j.l);
    }
    const float inv = out_factor(j.l, v_gs);
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
        uint32_t y[32] = {};
#pragma unroll 1
        for (int n = 0; n < parts; ++n) {
            const float f = ex2(__ldcg(ml0 + n * (2 * kPart)).x - j.m);
            float4 v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = __ldcg(rows0 + n * kPart + (8 * c + k) * kRows);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                y[4 * k] = __float_as_uint(fmaf(f, v[k].x, __uint_as_float(y[4 * k])));
                y[4 * k + 1] = __float_as_uint(fmaf(f, v[k].y, __uint_as_float(y[4 * k + 1])));
                y[4 * k + 2] = __float_as_uint(fmaf(f, v[k].z, __uint_as_float(y[4 * k + 2])));
                y[4 * k + 3] = __float_as_uint(fmaf(f, v[k].w, __uint_as_float(y[4 * k + 3])));
            }
        }
        put_out<DT>(tile, r, c, y, inv);
    }
    return j;
}

template <typename DT, bool SHARE>
__global__ void __launch_bounds__(kThreads, 1)
paged_attn_tc_kernel(const TcParams p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    Small &sm = *reinterpret_cast<Small *>(smem + kSmall);
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

    if (threadIdx.x == 0) {
        sm.failed = 0;
        for (int i = 0; i < 2; ++i) {
            bar_init(&sm.k_full[i], 4);
            bar_init(&sm.v_full[i], 4);
            bar_init(&sm.k_empty[i], 1);
            bar_init(&sm.v_empty[i], 1);
            bar_init(&sm.s_full[i], 1);
            bar_init(&sm.p_full[i], 4);
            bar_init(&sm.pv_done[i], 1);
            bar_init(&sm.q_full[i], 4);
            bar_init(&sm.work_full[i], 1);
            bar_init(&sm.work_empty[i], 13);
        }
        bar_init(&sm.claim, 1);
        bar_init(&sm.drained, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;"
                     :: "r"(smem_addr(&sm.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    pdl_wait();
    if (threadIdx.x == 0) {
        sm.k_gs = ld_f32(p.k_gs);
        sm.v_gs = ld_f32(p.v_gs);
        sm.work[0].rows = 0;
    }
    // Work in order: heads, a sequence's row blocks from its last (longest) one
    // on, sequences.  The blocks left over from whole waves of CTAs are cut by keys
    // into parts for all.
    unsigned whole = 0, parts = 1, total = 0;  // blocks not cut, parts of the others, works
    auto block_of = [&](unsigned id) { return !SHARE || id < whole ? id : whole + (id - whole) / parts; };
    // Work `id`: the at-th row block of sequence b, or a part of it.
    auto work_of = [&](unsigned id, int b, const Seq &s, int at, Work &w) {
        const int head = block_of(id) % (unsigned)p.hk;
        w.seq = b;
        w.head = head;
        w.q0 = s.q0;
        w.first_pos = s.first_pos;
        w.row0 = (row_blocks(p, s) - 1 - at) * kRows;
        w.rows = min(kRows, s.nq * p.per - w.row0);
        w.hi = s.first_pos + (w.row0 + w.rows - 1) / p.per + 1;
        w.first = p.window > 0 ? max(0, s.first_pos + w.row0 / p.per - p.window + 1) : 0;
        w.lo = w.first & ~15;
        w.n = w.hi > w.lo ? (w.hi - w.lo + kTile - 1) / kTile : 0;
        w.parts = 1;
        if (SHARE && id >= whole && parts > 1) {
            const int part = (id - whole) % parts, n = w.n, of = max(1, min((int)parts, n / kPartTiles));
            if (part >= of) {
                w.n = w.parts = 0;
            } else if (of > 1) {
                w.lo += n * part / of * kTile;
                w.n = n * (part + 1) / of - n * part / of;
                w.parts = of;
                w.part = part;
                w.shared = (id - whole) / parts;
                w.slot = w.shared * parts;  // of the first part
            }
        }
    };
    // ---- row blocks of the sequences before and in a thread's run of them; the
    // CTA's first one
    const int per_thread = (p.n_seqs + kThreads - 1) / kThreads;
    {
        const int b0 = min(p.n_seqs, (int)threadIdx.x * per_thread), b1 = min(p.n_seqs, b0 + per_thread);
        int64_t mine = 0;
        bool longer = false;  // some block may have keys for several parts
        for (int b = b0; b < b1; ++b) {
            const Seq s = load_seq(p, b);
            mine += row_blocks(p, s);
            if (SHARE) longer |= min(s.hi, p.width) >= 2 * kPartTiles * kTile - kRows;
        }
        int64_t upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
            if (lane >= o) upto += v;
        }
        if (lane == 31) sm.scan[warp] = upto;
        if (SHARE)
            longer = __syncthreads_or(longer);
        else
            __syncthreads();
        int64_t blocks = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w == warp) upto += blocks;
            blocks += sm.scan[w];
        }
        sm.upto[threadIdx.x] = upto;
        blocks = min(blocks * p.hk, (int64_t)p.limit);
        const unsigned over = SHARE ? (unsigned)blocks % gridDim.x : 0;
        whole = (unsigned)blocks - over;
        parts = longer && over > 0 ? max(1u, min(8u, min(gridDim.x, (unsigned)kSharedBlocks) / max(over, 1u))) : 1;
        total = whole + over * parts;
        int64_t at = blockIdx.x < total ? block_of(blockIdx.x) / p.hk : INT64_MAX;
        if (upto - mine <= at && at < upto) {
            at -= upto - mine;
            for (int b = b0; b < b1; ++b) {
                const Seq s = load_seq(p, b);
                const int n = row_blocks(p, s);
                if (at < n) {
                    work_of(blockIdx.x, b, s, (int)at, sm.work[0]);
                    break;
                }
                at -= n;
            }
        }
    }
    tm_fence_before();
    __syncthreads();
    tm_fence_after();
    const uint32_t tmem = sm.tmem;
    struct {
        uint32_t k_full, k_empty, v_full, v_empty, s_full, p_full, pv_done, q_full, drained, work_full, work_empty;
    } const bars = {smem_addr(sm.k_full), smem_addr(sm.k_empty), smem_addr(sm.v_full),    smem_addr(sm.v_empty),
                    smem_addr(sm.s_full), smem_addr(sm.p_full),  smem_addr(sm.pv_done),   smem_addr(sm.q_full),
                    smem_addr(&sm.drained), smem_addr(sm.work_full), smem_addr(sm.work_empty)};
    volatile int *failed = &sm.failed;
    // The CTA's i-th block of rows (rows = 0: there is none), for all roles but
    // the one that finds it.
    auto take = [&](int i, Work &w) {
        if (warp_wait(bars.work_full + 8 * (i & 1), (i >> 1) & 1, failed)) {
            w = sm.work[i & 1];
            __syncwarp();
            if (lane == 0) bar_arrive(bars.work_empty + 8 * (i & 1));
        } else {
            w.rows = 0;
        }
    };

    if (warp == 13) {
        // ---------------------------------------------------------- work
        // Blocks are taken from a counter that all CTAs share, each late in the
        // one before, the last (longest) block of a sequence first.
        bool more = sm.work[0].rows > 0;
        if (lane == 0) bar_arrive(bars.work_full);
        for (int i = 1; more; ++i) {
            // (the only wait for more than a tile's time)
            if (!warp_wait(smem_addr(&sm.claim), (i - 1) & 1, failed, (sm.work[(i - 1) & 1].n + 1) * kWaitNs)) break;
            if (i > 1 && !warp_wait(bars.work_empty + 8 * (i & 1), ((i >> 1) + 1) & 1, failed)) break;
            unsigned id = 0;
            if (lane == 0) id = gridDim.x + atomicAdd(reinterpret_cast<unsigned *>(p.workspace), 1u);
            id = __shfl_sync(0xFFFFFFFFu, id, 0);
            more = id < total;
            int64_t at = more ? block_of(id) / (unsigned)p.hk : 0;
            int run = 0;  // threads whose runs lie before the block
#pragma unroll
            for (int k = 0; k < kThreads / 32; ++k)
                run += __popc(__ballot_sync(0xFFFFFFFFu, sm.upto[k * 32 + lane] <= at));
            if (more) {
                if (run > 0) at -= sm.upto[run - 1];
                const int end = min(p.n_seqs, (run + 1) * per_thread);
                for (int b0 = run * per_thread; b0 < end; b0 += 32) {
                    const Seq s = load_seq(p, min(b0 + lane, end - 1));
                    const int mine = b0 + lane < end ? row_blocks(p, s) : 0;
                    int64_t upto = mine;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
                        if (lane >= o) upto += v;
                    }
                    if (upto - mine <= at && at < upto) {
                        work_of(id, b0 + lane, s, (int)(at - (upto - mine)), sm.work[i & 1]);
                    }
                    const int64_t all = __shfl_sync(0xFFFFFFFFu, upto, 31);
                    if (at < all) break;
                    at -= all;
                }
            } else if (lane == 0) {
                sm.work[i & 1].rows = 0;
            }
            __syncwarp();
            if (lane == 0) bar_arrive(bars.work_full + 8 * (i & 1));
        }
    } else if (warp == 12) {
        // ---------------------------------------------------------- products
        // The whole warp walks the loop, one elected lane issues: addresses
        // and descriptors then stay in uniform registers (a loop in one lane
        // alone spent 70 clocks a product moving them there, more than the
        // product takes: 587 us against 474 for 8192 tokens of 32 heads).
        const uint32_t base = smem_addr(smem);
        const uint64_t dq = operand(base + kQ, 16), dk = operand(base + kK, 16);
        const uint64_t dv = operand(base + kV, kTileBytes / 2);
        const bool lead = elect_one();
        auto qk = [&](int tt, int g) {
            const uint64_t a = dq + tt * (kTileBytes >> 4), bk = dk + (g & 1) * (kTileBytes >> 4);
            if (lead) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint32_t off = ((k >> 2) * (kTileBytes / 2) + (k & 3) * 32) >> 4;
                    mma_ss(tmem + kColS + tt * 128, a + off, bk + off, kIdescQK, k > 0);
                }
                mma_commit(bars.s_full + 8 * (tt));
                if (tt == 1) mma_commit(bars.k_empty + 8 * (g & 1));
            }
        };
        bool ok = true;
        int g = 0, q = 0;  // tiles of keys, blocks with keys so far
        for (int i = 0; ok; ++i) {
            Work w;
            take(i, w);
            if (w.rows == 0) break;
            if (w.n == 0) continue;
            const int end = g + w.n;
            ok = warp_wait(bars.k_full + 8 * (g & 1), (g >> 1) & 1, failed);
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
                if (!ok || !(ok = warp_wait(bars.q_full + 8 * tt, q & 1, failed))) break;
                tm_fence_after();
                qk(tt, g);
            }
            ++q;
            for (bool more = false; ok && g < end; ++g, more = true) {
                ok = warp_wait(bars.v_full + 8 * (g & 1), (g >> 1) & 1, failed) &&
                     (g + 1 == end || warp_wait(bars.k_full + 8 * ((g + 1) & 1), ((g + 1) >> 1) & 1, failed));
                const uint64_t bv = dv + (g & 1) * (kTileBytes >> 4);
#pragma unroll
                for (int tt = 0; tt < 2; ++tt) {
                    if (!ok || !(ok = warp_wait(bars.p_full + 8 * tt, g & 1, failed))) break;
                    tm_fence_after();
                    if (lead) {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            mma_ts(tmem + kColO + tt * 128, tmem + kColS + tt * 128 + k * 8, bv + k * (2048 >> 4),
                                   kIdescPV, more || k > 0);
                        mma_commit(bars.pv_done + 8 * tt);
                        if (tt == 1) mma_commit(bars.v_empty + 8 * (g & 1));
                    }
                    if (g + 1 < end) qk(tt, g + 1);
                }
            }
        }
        // no product may outlive the operands and the tensor memory, also
        // when the loop gave up
        int none = 0;
        if (lead) mma_commit(bars.drained);
        warp_wait(bars.drained, 0, &none);
    } else if (warp >= 8) {
        // ---------------------------------------------------------- keys and values
        // The next tile's bytes are asked for before this one is decoded; the next
        // block's first ones as well, if the block is known by then.
        const int tok = threadIdx.x - 8 * 32;
        const uint32_t to = smem_addr(smem) + tok * 128 + ((tok & 7) << 4);
        Feed feed;
        Row k, v;
        int i = 0, g = 0, left = 1;        // left: tiles of the block not yet asked for, and one
        bool ready = false, ended = false;  // a tile is in k and v; no block is left
        auto begin = [&](bool wait) {       // on to the next block with keys
            Work w;
            do {
                if (!wait && !warp_test(bars.work_full + 8 * (i & 1), (i >> 1) & 1)) return false;
                take(i++, w);
            } while (w.rows > 0 && w.n == 0);
            ended = w.rows == 0;
            if (ended) return false;
            feed.start(p, w.seq, w.head, w.lo, w.first, w.hi, tok);
            left = w.n;
            return true;
        };
        for (;;) {
            const int st = g & 1;
            if (ready) {
                if (g >= 2 && !warp_wait(bars.k_empty + 8 * st, ((g >> 1) + 1) & 1, failed)) break;
                const uint32_t seen = __ballot_sync(0xFFFFFFFFu, k.there);
                if (lane == 0) sm.seen[g & 3][warp - 8] = seen;
                decode_row(k, to + kK + st * kTileBytes);
                async_proxy_fence();
                __syncwarp();
                if (lane == 0) bar_arrive(bars.k_full + 8 * st);
            }
            // waits for the next block only with nothing left to decode: it may be
            // told after the last tile's use
            bool have = --left > 0;
            if (!have && !ended) have = begin(!ready);
            if (!have && !ready) break;
            bool there;
            const uint8_t *src = feed.step(p, there);  // (without one: of no use)
            feed.load(k, src, there, kKVCodesK, kKVScalesK);
            if (ready) {
                if (g >= 2 && !warp_wait(bars.v_empty + 8 * st, ((g >> 1) + 1) & 1, failed)) break;
                decode_row(v, to + kV + st * kTileBytes);
                async_proxy_fence();
                __syncwarp();
                if (lane == 0) bar_arrive(bars.v_full + 8 * st);
                ++g;
            }
            feed.load(v, src, there, kKVCodesV, kKVScalesV);
            ready = have;
            if (!have) left = 1;
        }
    } else {
        // ---------------------------------------------------------- rows
        const int t = warp >> 2, r = threadIdx.x & 127;          // tile and row of it
        const uint32_t tile = smem_addr(smem) + kQ + t * kTileBytes;
        const uint32_t at = tmem + ((uint32_t)(warp & 3) << 21);  // the warp's 32 rows
        const uint32_t s_at = at + kColS + t * 128, o_at = at + kColO + t * 128;
        // Queries: a warp its 32 rows, 16 lanes a row and all loads at once (a
        // thread a row took 5.8 us here); rows past the last repeat the block's
        // first one (a load under a condition would be waited for at once).
        uint4 x[16];
        auto load_q = [&](const Work &w) {
            const int row = w.row0 + (t * kTile + r < w.rows ? t * kTile + r : 0), query = row / p.per;
            const int64_t mine = (w.q0 + query) * p.q_stride + (int64_t)(w.head * p.per + row - query * p.per) * kD;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int64_t from = __shfl_sync(0xFFFFFFFFu, mine, 2 * i + (lane >> 4));
                x[i] = ld_keep16(static_cast<const uint8_t *>(p.q) + from * 2 + (lane & 15) * 16);
            }
        };
        // Into the tile, times a power of two for bf16; the scale of the row's
        // scores.
        auto put_q = [&]() {
            float back = 1.0f;  // of the thread's own row
            if (std::is_same<DT, BF16>::value) {
                // Largest magnitudes (bf16 bits without the sign order as the
                // values): the 16 lanes of a row hold 16 rows' partial ones, and
                // halving both leaves lane i of them with row i's.
                uint32_t a[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    uint32_t two[2];
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const uint4 w = x[2 * k + n];
                        two[n] = __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu),
                                          __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu));
                    }
                    a[k] = __vmaxu2(__byte_perm(two[0], two[1], 0x5410), __byte_perm(two[0], two[1], 0x7632));
                }
#pragma unroll
                for (int n = 4; n > 0; n >>= 1)
#pragma unroll
                    for (int k = 0; k < n; ++k) {
                        const bool up = lane & (2 * n);
                        const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, up ? a[k] : a[k + n], 2 * n);
                        a[k] = __vmaxu2(up ? a[k + n] : a[k], got);
                    }
                a[0] = __vmaxu2(a[0], __shfl_xor_sync(0xFFFFFFFFu, a[0], 1));
                const float2 pw = row_power(__uint_as_float(lane & 1 ? a[0] & 0xFFFF0000u : a[0] << 16));
                back = __shfl_sync(0xFFFFFFFFu, pw.y, (lane & 1) * 16 + (lane >> 1));
                float f[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) f[i] = __shfl_sync(0xFFFFFFFFu, pw.x, (lane & 16) + i);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float e[8];
                    unpack8<DT>(x[i], e);
#pragma unroll
                    for (int k = 0; k < 8; ++k) e[k] *= f[i];
                    x[i] = pack8<FP16>(e);
                }
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int to = (warp & 3) * 32 + 2 * i + (lane >> 4);
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};"
                             :: "r"(tile + ((lane >> 3) & 1) * (kTileBytes / 2) + to * 128 +
                                    (((lane & 7) ^ (to & 7)) << 4)),
                                "r"(x[i].x), "r"(x[i].y), "r"(x[i].z), "r"(x[i].w) : "memory");
            }
            async_proxy_fence();
            __syncwarp();
            if (lane == 0) bar_arrive(bars.q_full + 8 * t);
            return fmaxf(p.scale * back / sm.k_gs, kLeastScale);
        };

        // (a block's numbers stay in shared memory: the loop over its keys has no
        // register to spare)
        bool more = warp_wait(bars.work_full, 0, failed) && sm.work[0].rows > 0;
        float scale = 0.0f;
        if (more) {
            load_q(sm.work[0]);
            if (sm.work[0].n > 0) scale = put_q();
        }
        int g = 0;  // tiles of keys so far
        for (int i = 0; more; ++i) {
            const Work &w = sm.work[i & 1];
            // the row's keys [row_hi - width, row_hi), counted from lo less the
            // tiles before
            int row_hi = t * kTile + r < w.rows ? w.first_pos + (w.row0 + t * kTile + r) / p.per + 1 - w.lo : 0;
            const int end = g + w.n;
            // the next block is taken late, so that the last ones are shared out evenly
            if (threadIdx.x == 0 && w.n == 0) bar_arrive(smem_addr(&sm.claim));
            float m = kNoMax, l = 0.0f;
            for (bool begun = false; g < end; ++g, begun = true, row_hi -= kTile) {
                if (threadIdx.x == 0 && (begun ? end - g == 3 : end - g <= 3)) bar_arrive(smem_addr(&sm.claim));
                bool full = __all_sync(0xFFFFFFFFu, row_hi >= kTile && row_hi <= p.width);
                if (!warp_wait(bars.s_full + 8 * (t), g & 1, failed)) break;
                tm_fence_after();
                // nearly always every row sees the whole tile
                const uint4 readable = *reinterpret_cast<const uint4 *>(sm.seen[g & 3]);
                full = full && (readable.x & readable.y & readable.z & readable.w) == ~0u;
                uint32_t x0[32], x1[32];
                if (!full) {
                    // -inf for keys that a row does not see (in tensor memory, so that the
                    // code below, that most tiles take, is short)
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        const int below = row_hi - 32 * c, from = (int)((uint32_t)below - (uint32_t)p.width);
                        const uint32_t a = below >= 32 ? ~0u : (below <= 0 ? 0u : (1u << below) - 1u);
                        const uint32_t z = from <= 0 ? 0u : (from >= 32 ? ~0u : (1u << from) - 1u);
                        const uint32_t vis = a & ~z & sm.seen[g & 3][c];
                        tm_load32(s_at + 32 * c, x1);
                        tm_wait_ld(x1);
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (!(vis & (1u << k))) x1[k] = 0xFF800000u;
                        tm_store32(s_at + 32 * c, x1);
                    }
                    tm_wait_st();
                }
                auto top_of = [&](int c0, int c1) {  // the largest score of columns 32 c0 .. (in x1)
                    float top = kNoMax;
#pragma unroll 1
                    for (int c = c0; c < c1; ++c) {
                        tm_load32(s_at + 32 * c, x1);
                        tm_wait_ld(x1);
                        float a[4] = {top, kNoMax, kNoMax, kNoMax};
#pragma unroll
                        for (int k = 0; k < 32; ++k) a[k & 3] = fmaxf(a[k & 3], __uint_as_float(x1[k]) * scale);
                        top = fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3]));
                    }
                    return top;
                };
                // (of a tile that all see, a quarter: those far above it take the path below)
                if (!begun) m = top_of(0, full ? 1 : 4);
                uint32_t pk[64];
                float sum[4];
                // (one copy of the code: instructions that miss their cache cost more
                // than the branch)
#pragma unroll 1
                for (bool high = true;;) {
                    sum[0] = sum[1] = sum[2] = sum[3] = 0.0f;
                    const float2 s2 = make_float2(scale, scale), nm = make_float2(-m, -m);
                    auto exps = [&](uint32_t (&x)[32], int c) {  // one chunk of P and of the sum
                        // 16 at a time: the exponentials first, then what uses them
                        // (this file is compiled with little instruction scheduling,
                        // so that they stay apart: the scheduler's own order put each
                        // use behind its exponential and took 14 clocks an element of
                        // a lone warp where this takes 6.6)
#pragma unroll
                        for (int k0 = 0; k0 < 32; k0 += 16) {
                            float y[16];
#pragma unroll
                            for (int k = 0; k < 16; k += 2) {
                                const float2 z = __ffma2_rn(
                                    make_float2(__uint_as_float(x[k0 + k]), __uint_as_float(x[k0 + k + 1])), s2, nm);
                                y[k] = ex2(z.x);
                                y[k + 1] = ex2(z.y);
                            }
#pragma unroll
                            for (int k = 0; k < 16; ++k) sum[k & 3] += y[k];
#pragma unroll
                            for (int k = 0; k < 16; k += 2) pk[16 * c + (k0 + k) / 2] = FP16::pack(y[k], y[k + 1]);
                        }
                    };
                    tm_load32(s_at, x0);  // the next chunk's scores arrive meanwhile
                    tm_wait_ld(x0);
                    tm_load32(s_at + 32, x1);
                    exps(x0, 0);
                    tm_wait_ld(x1);
                    tm_load32(s_at + 64, x0);
                    exps(x1, 1);
                    tm_wait_ld(x0);
                    tm_load32(s_at + 96, x1);
                    exps(x0, 2);
                    tm_wait_ld(x1);
                    exps(x1, 3);
                    if (!__any_sync(0xFFFFFFFFu, high && sum[0] + sum[1] + sum[2] + sum[3] > kPMax)) break;
                    // a row's maximum has risen: take it, rescale, and form P again
                    // (S was formed after the product of the tile before; the first
                    // tile's product will replace O)
                    const float top = fmaxf(m, top_of(0, 4));
                    const float f = ex2(m - top);
                    m = top;
                    l *= f;
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        tm_load32(o_at + 32 * c, x1);
                        tm_wait_ld(x1);
#pragma unroll
                        for (int k = 0; k < 32; ++k) x1[k] = __float_as_uint(__uint_as_float(x1[k]) * f);
                        tm_store32(o_at + 32 * c, x1);
                    }
                    high = false;
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                tm_store32(s_at, pk);
                tm_store32(s_at + 32, pk + 32);
                tm_wait_st();
                tm_fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(bars.p_full + 8 * t);
            }
            // ------------------------------------------------------ last step
            bool store = !SHARE || w.parts == 1;
            if (SHARE && w.parts > 1) {
                if (!warp_wait(bars.pv_done + 8 * t, (end - 1) & 1, failed)) l = __uint_as_float(0x7FC00000u);
                tm_fence_after();
                const Joined j = share_part<DT>(
                    p.workspace + kTakenBytes + p.parts_at + w.slot * kSharedPartBytes,
                    reinterpret_cast<unsigned *>(p.workspace) + 4 + w.shared * 8 + warp, w.part, w.parts,
                    t * kTile + r, o_at, tile, r, m, l, sm.v_gs);
                m = j.m;
                l = j.l;
                store = j.last;
            }
            // the next block's queries on their way meanwhile
            const bool told = warp_wait(bars.work_full + 8 * ((i + 1) & 1), ((i + 1) >> 1) & 1, failed);
            more = told && sm.work[(i + 1) & 1].rows > 0;
            load_q(sm.work[more ? (i + 1) & 1 : i & 1]);
            if (w.n > 0) {
                warp_wait(bars.pv_done + 8 * t, (end - 1) & 1, failed);
                tm_fence_after();
            }
            // through the tile's place of Q, so that a row's 256 bytes leave together
            const bool bad = *failed;
            const float inv = bad ? __uint_as_float(0x7FC00000u) : out_factor(l, sm.v_gs);
            if (!SHARE || w.parts == 1) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t y[32];  // (of no meaning without keys: inv is 0 then)
                    tm_load32(o_at + 32 * c, y);
                    tm_wait_ld(y);
                    put_out<DT>(tile, r, c, y, inv);
                }
            }
            __syncwarp();
            const int row = w.row0 + t * kTile + r, query = row / p.per;
            const bool real = store && t * kTile + r < w.rows;
            const int out_row = (w.q0 + query) * p.hq + w.head * p.per + row - query * p.per;
#pragma unroll
            for (int n0 = 0; n0 < 16; n0 += 4) {
                int to[4];
                uint4 v[4];
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    to[n] = __shfl_sync(0xFFFFFFFFu, real ? out_row : -1, 2 * (n0 + n) + (lane >> 4));
                    const int from = (warp & 3) * 32 + 2 * (n0 + n) + (lane >> 4);
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(v[n].x), "=r"(v[n].y), "=r"(v[n].z), "=r"(v[n].w)
                                 : "r"(tile + ((lane >> 3) & 1) * (kTileBytes / 2) + from * 128 +
                                       (((lane & 7) ^ (from & 7)) << 4)) : "memory");
                }
#pragma unroll
                for (int n = 0; n < 4; ++n)
                    if (to[n] >= 0)
                        st16(static_cast<uint8_t *>(p.out) + (int64_t)to[n] * (kD * 2) + (lane & 15) * 16, v[n]);
            }
            if (real && p.lse != nullptr) p.lse[out_row] = bad ? __uint_as_float(0x7FC00000u) : lse_of(m, l);
            __syncwarp();
            if (lane == 0) bar_arrive(bars.work_empty + 8 * (i & 1));
            if (more && sm.work[(i + 1) & 1].n > 0) scale = put_q();
        }
    }
    // ---------------------------------------------------------------- leave
    tm_fence_before();
    __syncthreads();
    if (warp == 12) {
        tm_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" :: "r"(tmem) : "memory");
    }
}

template <typename DT, bool SHARE>
cudaError_t launch(const TcParams &p, int dev, unsigned ctas, cudaStream_t stream)
{
    static std::atomic<int> ready[64];
    auto kern = paged_attn_tc_kernel<DT, SHARE>;
    if (dev >= 64 || !ready[dev].load(std::memory_order_relaxed)) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready[dev].store(1, std::memory_order_relaxed);
    }
    return launch_pdl(kern, ctas, kThreads, kSmemBytes, stream, p);
}

}  // namespace

template <typename DT>
cudaError_t launch_paged_attn_tc(const PagedAttnParams &p, size_t parts_at, cudaStream_t stream)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    // every sequence has a part of a row block at most beside its full ones
    const int64_t rows = p.n_tokens * p.per;
    const int64_t blocks = (rows / kRows + (rows / (p.few + 1) < p.n_seqs ? rows / (p.few + 1) : p.n_seqs)) * p.hk;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    if (blocks == 0) return cudaSuccess;
    TcParams tp;
    static_cast<PagedAttnParams &>(tp) = p;
    tp.limit = (unsigned)blocks;
    tp.width = p.window > 0 ? p.window : 1 << 30;
    tp.parts_at = parts_at;
    // Few waves of blocks with many keys: those left over from whole waves are
    // shared out by keys.  2 chunks of 2047 tokens after 14 thousand, 3.4 waves: 662
    // us (710 without); 8 prompts of 1024, 3.4 waves of few keys, 57 us (55) and 5
    // waves in a window of 2048 keys 181 us (178): the longer kernel misses its
    // instruction cache more often.
    const int64_t sms = device_sms(dev);
    if (blocks <= 4 * sms && p.max_keys >= 2 * kPartTiles * kTile)
        return launch<DT, true>(tp, dev, (unsigned)(8 * blocks < sms ? 8 * blocks : sms), stream);
    return launch<DT, false>(tp, dev, (unsigned)(blocks < sms ? blocks : sms), stream);
}

template cudaError_t launch_paged_attn_tc<BF16>(const PagedAttnParams &, size_t, cudaStream_t);
template cudaError_t launch_paged_attn_tc<FP16>(const PagedAttnParams &, size_t, cudaStream_t);

}  // namespace rq
