// rq_paged_attn_tc.cu -- attention over the paged NVFP4 cache for runs of
// queries (prompts, chunks), on the fifth-generation tensor cores.
//
// A CTA takes 256 rows (query, head of the KV head's group) of a sequence as
// two tiles of 128 and walks the keys in tiles of 128.  Per tile of keys:
//   S_t = Q_t K^T        tcgen05.mma, both operands in shared memory,
//   P_t = 2^(S_t c - m)  a thread a row, from and to tensor memory (the fp16 P
//                        over S's own columns),
//   O_t += P_t V         tcgen05.mma, P from tensor memory, V from shared,
// with S and O of both tiles in all 512 tensor-memory columns.  Roles:
//   warps 0-3, 4-7   the rows of tile 0, tile 1: softmax, and the last step
//   warps 8-11       a token each: codes from global memory (one tile ahead in
//                    registers), decoded to fp16 rows in shared memory
//   warp 12          issues the products: PV_0(j) QK_0(j+1) PV_1(j) QK_1(j+1),
//                    so that one tile's softmax runs under the other's products
// m is the row's maximum when it was last looked at.  That is when a tile's sum
// of P passes kPMax (so no P exceeds it, and fp16 holds them all): the row's O
// is then rescaled in tensor memory, after the product before.  Between, no
// maximum is formed.
//
// What bounds it: 4 * 128 flops a visible pair on the tensor cores.  The
// operands of a 128 x 128 x 16 product are 8 KB of shared memory in its 64
// clocks (4 KB with P in tensor memory), the decoded tile another 32 bytes a
// clock, and the exponentials need half the time of the products.
//
// Every wait has a time limit (kWaitNs): past it the CTA gives up, writes NaN
// and leaves, tensor memory freed.  No valid call meets it.
#include "rq_paged_attn.cuh"

#include <atomic>
#include <type_traits>

namespace rq {

namespace {

constexpr int kD = 128, kTile = 128, kRows = 2 * kTile;
constexpr int kThreads = 13 * 32;
constexpr uint32_t kTileBytes = kTile * kD * 2;  // 32 KB
// shared memory (from a 1024-byte boundary): Q0 Q1 K[2] V[2], then the small part
constexpr uint32_t kQ = 0, kK = 2 * kTileBytes, kV = kK + 2 * kTileBytes, kSmall = kV + 2 * kTileBytes;
constexpr unsigned long long kWaitNs = 1000000000ull;

struct Small {
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], pv_done[2], drained;
    uint32_t seen[4][4];  // tile j's readable tokens, ring of 4
    uint32_t tmem;
    int failed;
    int seq, block;
    int64_t scan[13];
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
__device__ __forceinline__ void tm_store32(uint32_t addr, const uint32_t (&v)[32])
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
__device__ __forceinline__ void tm_store16(uint32_t addr, const uint32_t *v)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16};"
        :: "r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
           "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
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
// kWaitNs, or when another role of the CTA has (false).
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int *failed)
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
            if (t - start > kWaitNs) {
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
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *failed)
{
    return __all_sync(0xFFFFFFFFu, bar_wait(bar, parity, failed));
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

template <typename DT>
__global__ void __launch_bounds__(kThreads, 1)
paged_attn_tc_kernel(const PagedAttnParams p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    Small &sm = *reinterpret_cast<Small *>(smem + kSmall);
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

    // ---- which rows: CTA x / hk in the order of the sequences' row blocks,
    // the last (longest) block of a sequence first
    {
        const int per_thread = (p.n_seqs + kThreads - 1) / kThreads;
        const int b0 = min(p.n_seqs, (int)threadIdx.x * per_thread), b1 = min(p.n_seqs, b0 + per_thread);
        int64_t mine = 0;
        for (int b = b0; b < b1; ++b) mine += row_blocks(p, load_seq(p, b));
        int64_t upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
            if (lane >= o) upto += v;
        }
        if (lane == 31) sm.scan[warp] = upto;
        if (threadIdx.x == 0) {
            sm.seq = -1;
            sm.failed = 0;
            for (int i = 0; i < 2; ++i) {
                bar_init(&sm.k_full[i], 4);
                bar_init(&sm.v_full[i], 4);
                bar_init(&sm.k_empty[i], 1);
                bar_init(&sm.v_empty[i], 1);
                bar_init(&sm.s_full[i], 1);
                bar_init(&sm.p_full[i], 4);
                bar_init(&sm.pv_done[i], 1);
            }
            bar_init(&sm.drained, 1);
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        __syncthreads();
        for (int w = 0; w < warp; ++w) upto += sm.scan[w];
        int64_t at = blockIdx.x / p.hk;
        if (upto - mine <= at && at < upto) {
            at -= upto - mine;
            for (int b = b0; b < b1; ++b) {
                const int n = row_blocks(p, load_seq(p, b));
                if (at < n) {
                    sm.seq = b;
                    sm.block = n - 1 - (int)at;
                    break;
                }
                at -= n;
            }
        }
        __syncthreads();
        if (sm.seq < 0) return;
    }
    const int b = sm.seq, head = blockIdx.x % p.hk;
    const Seq s = load_seq(p, b);
    const int row0 = sm.block * kRows, rows = min(kRows, s.nq * p.per - row0);
    // keys that some row of the block sees: [first, hi), in n tiles from lo
    const int i_last = (row0 + rows - 1) / p.per, hi = s.first_pos + i_last + 1;
    const int first = p.window > 0 ? max(0, s.first_pos + row0 / p.per - p.window + 1) : 0, lo = first & ~15;
    const int n = hi > lo ? (hi - lo + kTile - 1) / kTile : 0;

    if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;"
                     :: "r"(smem_addr(&sm.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // ---- the first keys and values are asked for before the queries
    const bool producer = warp >= 8 && warp < 12;
    Feed feed;
    Row k, v;
    // ---- queries: a warp its 32 rows, 16 lanes a row and all loads at once (a
    // thread a row took 5.8 us here), times a power of two for bf16
    float scale = 0.0f;
    const int t = warp >> 2, r = threadIdx.x & 127;  // tile and row (warps 0-7)
    const int row = t * kTile + r;                   // of the block
    const int query = (row0 + row) / p.per, group_head = head * p.per + (row0 + row) - query * p.per;
    const int64_t out_row = (int64_t)(s.q0 + query) * p.hq + group_head;
    const bool real = row < rows;
    if (producer && n > 0) {  // (the branches are one, so that neither keeps registers for the other)
        bool there;
        feed.start(p, b, head, lo, first, hi, threadIdx.x - 8 * 32);
        const uint8_t *g = feed.step(p, there);
        feed.load(k, g, there, kKVCodesK, kKVScalesK);
        feed.load(v, g, there, kKVCodesV, kKVScalesV);
    } else if (warp < 8) {
        // rows past the last repeat the block's first one (a load under a
        // condition would be waited for at once)
        const int first_query = row0 / p.per, first_head = head * p.per + row0 - first_query * p.per;
        const int64_t mine = (s.q0 + (real ? query : first_query)) * p.q_stride +
                             (int64_t)(real ? group_head : first_head) * kD;
        uint4 x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int64_t at = __shfl_sync(0xFFFFFFFFu, mine, 2 * i + (lane >> 4));
            x[i] = ld_keep16(static_cast<const uint8_t *>(p.q) + at * 2 + (lane & 15) * 16);
        }
        float back = 1.0f;  // of the thread's own row
        if (std::is_same<DT, BF16>::value) {
            // largest magnitudes, four rows' reductions side by side: bf16 bits
            // without the sign order as the values
#pragma unroll
            for (int i0 = 0; i0 < 16; i0 += 4) {
                uint32_t a[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint4 w = x[i0 + i];
                    a[i] = __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu),
                                    __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu));
                }
#pragma unroll
                for (int o = 8; o > 0; o >>= 1)
#pragma unroll
                    for (int i = 0; i < 4; ++i) a[i] = __vmaxu2(a[i], __shfl_xor_sync(0xFFFFFFFFu, a[i], o));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 pw = row_power(__uint_as_float(max(a[i] << 16, a[i] & 0xFFFF0000u)));
                    float e[8];
                    unpack8<DT>(x[i0 + i], e);
#pragma unroll
                    for (int k = 0; k < 8; ++k) e[k] *= pw.x;
                    x[i0 + i] = pack8<FP16>(e);
                    const float other = __shfl_sync(0xFFFFFFFFu, pw.y, (lane & 1) * 16);
                    back = (lane >> 1) == i0 + i ? other : back;
                }
            }
        }
        const uint32_t tile = smem_addr(smem) + kQ + t * kTileBytes + ((lane >> 3) & 1) * (kTileBytes / 2);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int to = (warp & 3) * 32 + 2 * i + (lane >> 4);
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};"
                         :: "r"(tile + to * 128 + (((lane & 7) ^ (to & 7)) << 4)), "r"(x[i].x), "r"(x[i].y),
                            "r"(x[i].z), "r"(x[i].w) : "memory");
        }
        scale = fmaxf(p.scale * back / ld_f32(p.k_gs), kLeastScale);
        async_proxy_fence();
    }
    tm_fence_before();
    __syncthreads();
    tm_fence_after();
    const uint32_t tmem = sm.tmem;
    struct {
        uint32_t k_full, k_empty, v_full, v_empty, s_full, p_full, pv_done, drained;
    } const bars = {smem_addr(sm.k_full), smem_addr(sm.k_empty), smem_addr(sm.v_full),  smem_addr(sm.v_empty),
                    smem_addr(sm.s_full), smem_addr(sm.p_full),  smem_addr(sm.pv_done), smem_addr(&sm.drained)};
    volatile int *failed = &sm.failed;

    if (warp == 12) {
        // ---------------------------------------------------------- products
        // The whole warp walks the loop, one elected lane issues: addresses
        // and descriptors then stay in uniform registers (a loop in one lane
        // alone spent 70 clocks a product moving them there, more than the
        // product takes: 587 us against 474 for 8192 tokens of 32 heads).
        const uint32_t base = smem_addr(smem);
        const uint64_t dq = operand(base + kQ, 16), dk = operand(base + kK, 16);
        const uint64_t dv = operand(base + kV, kTileBytes / 2);
        const bool lead = elect_one();
        auto qk = [&](int tt, int j) {
            const uint64_t a = dq + tt * (kTileBytes >> 4), bk = dk + (j & 1) * (kTileBytes >> 4);
            if (lead) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint32_t off = ((k >> 2) * (kTileBytes / 2) + (k & 3) * 32) >> 4;
                    mma_ss(tmem + kColS + tt * 128, a + off, bk + off, kIdescQK, k > 0);
                }
                mma_commit(bars.s_full + 8 * (tt));
                if (tt == 1) mma_commit(bars.k_empty + 8 * (j & 1));
            }
        };
        bool ok = n > 0 && warp_wait(bars.k_full + 8 * (0), 0, failed);
        if (ok) {
            tm_fence_after();
            qk(0, 0);
            qk(1, 0);
        }
        for (int j = 0; ok && j < n; ++j) {
            ok = warp_wait(bars.v_full + 8 * (j & 1), (j >> 1) & 1, failed) &&
                 (j + 1 == n || warp_wait(bars.k_full + 8 * ((j + 1) & 1), ((j + 1) >> 1) & 1, failed));
            const uint64_t bv = dv + (j & 1) * (kTileBytes >> 4);
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
                if (!ok || !(ok = warp_wait(bars.p_full + 8 * (tt), j & 1, failed))) break;
                tm_fence_after();
                if (lead) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        mma_ts(tmem + kColO + tt * 128, tmem + kColS + tt * 128 + k * 8, bv + k * (2048 >> 4),
                               kIdescPV, j > 0 || k > 0);
                    mma_commit(bars.pv_done + 8 * (tt));
                    if (tt == 1) mma_commit(bars.v_empty + 8 * (j & 1));
                }
                if (j + 1 < n) qk(tt, j + 1);
            }
        }
        // no product may outlive the operands and the tensor memory, also
        // when the loop gave up
        int none = 0;
        if (lead) mma_commit(bars.drained);
        warp_wait(bars.drained, 0, &none);
    } else if (producer) {
        // ---------------------------------------------------------- keys and values
        const int tok = feed.tok;
        const uint32_t to = smem_addr(smem) + tok * 128 + ((tok & 7) << 4);
        for (int j = 0; j < n; ++j) {
            const int st = j & 1;
            if (j >= 2 && !warp_wait(bars.k_empty + 8 * st, ((j >> 1) + 1) & 1, failed)) break;
            const uint32_t seen = __ballot_sync(0xFFFFFFFFu, k.there);
            if (lane == 0) sm.seen[j & 3][warp - 8] = seen;
            decode_row(k, to + kK + st * kTileBytes);
            async_proxy_fence();
            __syncwarp();
            if (lane == 0) bar_arrive(bars.k_full + 8 * st);
            bool there;
            const uint8_t *g = feed.step(p, there);
            feed.load(k, g, there, kKVCodesK, kKVScalesK);
            if (j >= 2 && !warp_wait(bars.v_empty + 8 * st, ((j >> 1) + 1) & 1, failed)) break;
            decode_row(v, to + kV + st * kTileBytes);
            async_proxy_fence();
            __syncwarp();
            if (lane == 0) bar_arrive(bars.v_full + 8 * st);
            feed.load(v, g, there, kKVCodesV, kKVScalesV);
        }
    } else {
        // ---------------------------------------------------------- softmax
        const uint32_t at = tmem + ((uint32_t)(warp & 3) << 21);  // the warp's 32 rows
        const uint32_t s_at = at + kColS + t * 128, o_at = at + kColO + t * 128;
        const int row_hi = real ? s.first_pos + query + 1 : 0;               // keys [row_lo, row_hi)
        const int row_lo = p.window > 0 ? row_hi - p.window : 0;
        const float v_gs = ld_f32(p.v_gs);
        float m = kNoMax, l = 0.0f;
        for (int j = 0; j < n; ++j) {
            if (!warp_wait(bars.s_full + 8 * (t), j & 1, failed)) break;
            tm_fence_after();
            auto visible = [&](int c) {  // of the tile's columns 32 c ..
                const int first = lo + j * kTile + 32 * c, below = row_hi - first, from = row_lo - first;
                const uint32_t a = below >= 32 ? ~0u : (below <= 0 ? 0u : (1u << below) - 1u);
                const uint32_t z = from <= 0 ? 0u : (from >= 32 ? ~0u : (1u << from) - 1u);
                return a & ~z & sm.seen[j & 3][c];
            };
            uint32_t pk[64];
            float sum[4] = {};
            const float2 s2 = make_float2(scale, scale);
            auto exps = [&](uint32_t (&x)[32], int c) {  // one chunk of P and of the sum
                const uint32_t vis = visible(c);
                if (__any_sync(0xFFFFFFFFu, vis != ~0u)) {
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (!(vis & (1u << k))) x[k] = 0xFF800000u;  // -inf
                }
                // 16 at a time: the exponentials first, then what uses them
                // (this file is compiled with little instruction scheduling,
                // so that they stay apart: the scheduler's own order put each
                // use behind its exponential and took 14 clocks an element of
                // a lone warp where this takes 6.6)
                const float2 nm = make_float2(-m, -m);
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
            auto all_exps = [&]() {  // the next chunk's scores arrive meanwhile
                uint32_t x0[32], x1[32];
                tm_load32(s_at, x0);
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
            };
            if (j > 0) all_exps();  // (the first tile has no maximum yet)
            if (j == 0 || __any_sync(0xFFFFFFFFu, sum[0] + sum[1] + sum[2] + sum[3] > kPMax)) {
                // a row's maximum has risen: take it, rescale, and form P again
                float top = m;
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    uint32_t x[32];
                    tm_load32(s_at + 32 * c, x);
                    tm_wait_ld(x);
                    const uint32_t vis = visible(c);
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (vis & (1u << k)) top = fmaxf(top, __uint_as_float(x[k]) * scale);
                }
                const float f = ex2(m - top);
                m = top;
                l *= f;
                if (j > 0) {
                    if (!warp_wait(bars.pv_done + 8 * (t), (j - 1) & 1, failed)) break;
                    tm_fence_after();
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t x[32];
                        tm_load32(o_at + 32 * c, x);
                        tm_wait_ld(x);
#pragma unroll
                        for (int k = 0; k < 32; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) * f);
                        tm_store32(o_at + 32 * c, x);
                    }
                }
                sum[0] = sum[1] = sum[2] = sum[3] = 0.0f;
                all_exps();
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
#pragma unroll
            for (int c = 0; c < 4; ++c) tm_store16(s_at + 16 * c, pk + 16 * c);
            tm_wait_st();
            tm_fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(bars.p_full + 8 * (t));
        }
        // ---------------------------------------------------------- last step
        if (n > 0) {
            warp_wait(bars.pv_done + 8 * (t), (n - 1) & 1, failed);
            tm_fence_after();
        }
        // through the tile's place of Q, so that a row's 256 bytes leave together
        const bool bad = *failed;
        const float inv = bad ? __uint_as_float(0x7FC00000u) : out_factor(l, v_gs);
        const uint32_t tile = smem_addr(smem) + kQ + t * kTileBytes;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            uint32_t x[32] = {};
            if (n > 0) {
                tm_load32(o_at + 32 * c, x);
                tm_wait_ld(x);
            }
#pragma unroll
            for (int k = 0; k < 32; k += 8) {
                float e[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) e[i] = l == 0.0f && !bad ? 0.0f : __uint_as_float(x[k + i]) * inv;
                const uint4 v = pack8<DT>(e);
                const int chunk = 4 * c + k / 8;
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};"
                             :: "r"(tile + (chunk >> 3) * (kTileBytes / 2) + r * 128 + (((chunk & 7) ^ (r & 7)) << 4)),
                                "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
            }
        }
        __syncwarp();
        const int64_t mine = real ? out_row : -1;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int64_t to = __shfl_sync(0xFFFFFFFFu, mine, 2 * i + (lane >> 4));
            const int from = (warp & 3) * 32 + 2 * i + (lane >> 4);
            uint4 v;
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                         : "r"(tile + ((lane >> 3) & 1) * (kTileBytes / 2) + from * 128 +
                               (((lane & 7) ^ (from & 7)) << 4)) : "memory");
            if (to >= 0) st16(static_cast<uint8_t *>(p.out) + to * (kD * 2) + (lane & 15) * 16, v);
        }
        if (real && p.lse != nullptr) p.lse[out_row] = bad ? __uint_as_float(0x7FC00000u) : lse_of(m, l);
    }
    // ---------------------------------------------------------------- leave
    tm_fence_before();
    __syncthreads();
    if (warp == 12) {
        tm_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" :: "r"(tmem) : "memory");
    }
}

}  // namespace

template <typename DT>
cudaError_t launch_paged_attn_tc(const PagedAttnParams &p, cudaStream_t stream)
{
    static std::atomic<int> ready[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    auto kern = paged_attn_tc_kernel<DT>;
    if (dev >= 64 || !ready[dev].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready[dev].store(1, std::memory_order_relaxed);
    }
    // every sequence has a part of a row block at most beside its full ones
    const int64_t rows = p.n_tokens * p.per;
    const int64_t blocks = rows / kRows + (rows / (p.few + 1) < p.n_seqs ? rows / (p.few + 1) : p.n_seqs);
    if (blocks * p.hk > INT32_MAX) return cudaErrorInvalidConfiguration;
    return blocks > 0 ? launch_pdl(kern, (unsigned)(blocks * p.hk), kThreads, kSmemBytes, stream, p) : cudaSuccess;
}

template cudaError_t launch_paged_attn_tc<BF16>(const PagedAttnParams &, cudaStream_t);
template cudaError_t launch_paged_attn_tc<FP16>(const PagedAttnParams &, cudaStream_t);

}  // namespace rq
