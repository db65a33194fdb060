// rq_paged_attn.cu -- attention over the paged NVFP4 cache for few queries a
// sequence (single-token decode, drafted tokens): the keys of a sequence are
// split over CTAs, each CTA's share over its warps, and the parts joined.
//
// Mathematics.  With x_j = scale log2(e) q . k_j, a part of the keys gives
//   l = sum 2^(x_j - m),  O = sum 2^(x_j - m) v_j
// for any m, and parts join by (m, l, O) -> sum of 2^(m_i - m) (l_i, O_i).  m is
// a maximum when it was last looked at: when a step's sum of exponentials
// passes kPMax (so that fp16 holds each of them).  Most steps need no maximum
// and no reduction over lanes.
//
// What bounds it: 144 bytes a key and KV head have to come from HBM; at 6.8
// TB/s an SM gets one every 6.1 clocks.  The products run on mma.sync with
// keys (then channels) as its 16 rows and queries as its 8 columns: the 2
// clocks a key that this takes at 8 columns lie under the memory time, and a
// key's codes go from shared memory to registers as the operand itself.
// (tcgen05 would want the decoded tile written to shared memory first, 512
// bytes a key: 4 clocks.)  Decoding (e2m1x2 -> f16x2, times the scale, exact)
// and the rest issue about 14 warp instructions a key, 3.5 clocks.
//
// Tokens of a group of 16 are laid over the fragments so that no value moves
// between lanes: lane (g, c) = (lane / 4, lane % 4) holds
//   K (16 tokens x 128, A operand): tokens row g and g + 8, channels 32 c ..
//     32 c + 31 (16 bytes of codes, 2 scales) over the 8 products;
//   V^T (128 x 16 tokens, A operand): channels 16 g .. 16 g + 15 (8 bytes of
//     codes, 1 scale) of tokens c, 4 + c, 8 + c, 12 + c; the nibbles of two
//     tokens are interleaved before the conversion, which then yields token
//     pairs;
//   S^T rows are the tokens, turned into the B operand of the second product
//     by movmatrix.  Row r of the first product is token tok(r) below.
#include "rq_paged_attn.cuh"

#include <atomic>
#include <climits>
#include <type_traits>

namespace rq {

namespace {

// Four warps a CTA, four CTAs an SM (registers): a CTA's warps meet at each
// item's end, so fewer of them wait less (measured with 8, 4 and 2 warps:
// 64 ragged sequences up to 4096 keys 48, 45 and 48 us, 32 sequences of 16
// query columns 40, 34 and 35, one of 1000 keys 9.6, 9.1 and 9.6, 128 x 8192
// keys 228, 228 and 237).
constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kChunkGroups = 2, kChunk = kChunkGroups * 16;  // keys of one step of a warp
constexpr int kStages = 3;
// An item's overhead (queries, first copies, join) in chunks, for the cut into
// shares (0, 4, 8, 16, 32: 56, 52, 46, 45, 49 us for the ragged sequences).
constexpr int kStart = 16;
constexpr int kBatch = 32 / kChunkGroups;  // chunks whose places a warp holds
constexpr uint32_t kAll = (1u << kChunkGroups) - 1u;
constexpr int kChunkBytes = kChunkGroups * kKVGroupBytes;
constexpr int kSmem = kWarps * kStages * kChunkBytes;
// Queries x heads of a KV head up to which a sequence is taken here and not by
// the tensor-memory kernel.
constexpr int kFewColumns = 32;
constexpr int kCluster = 8, kParts = kCluster * kWarps;
constexpr int kMaxCtas = 1024;     // grid limit (workspace slots)

// A part: O [8 NT][128], m [8 NT], l [8 NT].
template <int NT>
constexpr int kPartFloats = 8 * NT * (128 + 2);

// What the CTA left for the join, two slots each: slot 0 a part that continues
// an item begun by an earlier CTA (last: it ends it), slot 1 the first part of
// an item that later CTAs continue.
struct PartInfo {
    int valid, last, seq, head, block;
};

static_assert(kSharedBlocks * kSharedPartBytes <= (size_t)kMaxCtas * 2 * kPartFloats<2> * sizeof(float),
              "the parts of the other kernel lie where this one's are");

constexpr size_t kInfoBytes = ((size_t)kMaxCtas * 2 * sizeof(PartInfo) + 15) / 16 * 16;

// Shared memory at a 32-bit address plus a constant (an address that goes
// through a generic pointer costs three more instructions a load).
template <int OFF>
__device__ __forceinline__ uint4 lds16_at(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4 + %5];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a), "n"(OFF) : "memory");
    return v;
}
template <int OFF>
__device__ __forceinline__ uint2 lds8_at(uint32_t a)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2 + %3];" : "=r"(v.x), "=r"(v.y) : "r"(a), "n"(OFF) : "memory");
    return v;
}
template <int OFF>
__device__ __forceinline__ uint32_t lds2_at(uint32_t a)
{
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1 + %2];" : "=h"(v) : "r"(a), "n"(OFF) : "memory");
    return v;
}
template <int OFF>
__device__ __forceinline__ uint32_t lds1_at(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1 + %2];" : "=r"(v) : "r"(a), "n"(OFF) : "memory");
    return v;
}
template <int DST, int SRC>
__device__ __forceinline__ void cp16_at(uint32_t dst, const uint8_t *src)
{
    asm volatile("cp.async.cg.shared.global [%0 + %1], [%2 + %3], 16;"
                 :: "r"(dst), "n"(DST), "l"(src), "n"(SRC) : "memory");
}

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                    uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                 "{%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v)
{
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
    return d;
}

// Token of row r of the first product (r < 8; r + 8 is 8 tokens further), and
// its inverse: where a token's 64 bytes of K codes are put, so that a warp's
// 16-byte reads by row are consecutive.
__device__ __forceinline__ int tok_of_row(int r) { return (r & 1) * 4 + (r >> 1); }
__device__ __forceinline__ int row_of_tok(int t) { return (t >> 3) * 8 + (t & 3) * 2 + ((t >> 2) & 1); }

// How a sequence's work is cut: blocks of 8 NT query columns, tiles of kChunk
// keys.  Sequences of more than p.few columns are left to the other kernel.
struct Cut {
    int blocks, tiles;
};

template <int NT>
__device__ __forceinline__ Cut cut(const PagedAttnParams &p, const Seq &s)
{
    const int cols = s.nq * p.per;
    return Cut{cols > p.few ? 0 : (cols + 8 * NT - 1) / (8 * NT),
               s.hi > s.lo ? (s.hi - s.lo + kChunk - 1) / kChunk : 1};
}

template <int NT>
__device__ __forceinline__ int64_t seq_units(const PagedAttnParams &p, const Seq &s)
{
    const Cut c = cut<NT>(p, s);
    return (int64_t)p.hk * c.blocks * (c.tiles + kStart);
}

// a / b for a >= 0: a 64-bit division is some 150 instructions, and a is
// nearly always short.
__device__ __forceinline__ int64_t div_small(int64_t a, int b)
{
    return a >> 32 == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// Column of a sequence -> query and head of the group (one query: no division).
__device__ __forceinline__ int query_of(const PagedAttnParams &p, const Seq &s, int col)
{
    return s.nq == 1 ? 0 : (int)((uint32_t)col / (uint32_t)p.per);
}

// Barrier of the cluster; an address of another CTA's shared memory, and a load
// from it.
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_addr(const void *mine, int rank)
{
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(mine)), "r"(rank));
    return a;
}
__device__ __forceinline__ float ld_cluster(uint32_t a)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

// Stores 8 NT columns' results: out (and lse) of column col from its sums.
template <typename DT, int VALS>
__device__ __forceinline__ void store_out(const PagedAttnParams &p, const Seq &s, int head, int col,
                                          int d0, float (&v)[VALS], float m, float l, float v_gs)
{
    const int i = query_of(p, s, col), h = head * p.per + col - i * p.per;
    const int64_t row = ((int64_t)(s.q0 + i) * p.hq + h);
    const float inv = out_factor(l, v_gs);
    uint8_t *dst = static_cast<uint8_t *>(p.out) + (row * 128 + d0) * 2;
#pragma unroll
    for (int k = 0; k < VALS; k += 4)
        *reinterpret_cast<uint2 *>(dst + 2 * k) =
            make_uint2(DT::pack(v[k] * inv, v[k + 1] * inv), DT::pack(v[k + 2] * inv, v[k + 3] * inv));
    if (p.lse != nullptr && d0 == 0)
        p.lse[row] = lse_of(m, l);
}

// Where a lane's pieces of a group go in its warp's ring and where it reads them.
struct WarpRing {
    uint32_t kdst, vdst, fdst, kread, vread, ksread, vsread;
    float *o;  // the same memory, for the warp's part of O at the end

    __device__ __forceinline__ explicit WarpRing(uint8_t *mem)
    {
        const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
        const uint32_t ring = smem_addr(mem);
        // the 16-byte pieces of a group (the fifth: lanes 0-15)
        kdst = ring + row_of_tok(lane >> 2) * 64 + (lane & 3) * 16;  // + 512: tokens 8-15
        vdst = ring + kKVCodesV + (lane >> 2) * 64 + (((lane & 3) ^ ((lane >> 3) & 1) * 2) * 16);
        fdst = ring + kKVScalesK + lane * 16;
        kread = ring + g * 64 + c * 16;
        vread = ring + kKVCodesV + c * 64 + (((g >> 1) ^ ((c >> 1) & 1) * 2) * 16) + (g & 1) * 8;
        ksread = ring + kKVScalesK + tok_of_row(g) * 8 + 2 * c;
        vsread = ring + kKVScalesV + c * 8 + g;
        o = reinterpret_cast<float *>(mem);
    }
};

// A warp's part of an item: columns col0 .. col0 + cols - 1 of a sequence and KV
// head over the chunks first, first + step, .. of the keys from t0 (up to end
// and to what the columns see).  Leaves O [8 NT][128] in the warp's ring and m
// and the sum l of the columns in stats [8 NT].
template <typename DT, int NT>
__device__ __forceinline__ void attend(const PagedAttnParams &p, const Seq &s, int b, int head, int col0, int cols,
                                       int t0, int end, int first, int step, float inv_kgs, const WarpRing &w,
                                       float2 *stats)
{
    static_assert(kStages * kChunkBytes >= 8 * NT * 128 * 4, "a warp's ring holds its part of O at the end");
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    // keys that the block's columns see: all of [need_lo, need_hi) by every
    // one, nothing from blk_hi on by any
    const int i_first = query_of(p, s, col0), i_last = query_of(p, s, col0 + cols - 1);
    const int blk_hi = s.first_pos + i_last + 1;
    const int need_hi = s.first_pos + i_first + 1;
    const int need_lo = p.window > 0 ? blk_hi - p.window : 0;
    const int t1 = min(blk_hi, end);  // may lie before t0: nothing to do
    const int chunks =
        t1 > t0 + first * kChunk ? (t1 - t0 - first * kChunk + step * kChunk - 1) / (step * kChunk) : 0;

    // ---- queries' loads: columns nt * 8 + g (past the last: the first
    // again; a load under a condition would be waited for at once),
    // channels 32 c .. + 31
    uint4 qv[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int col = col0 + (nt * 8 + g < cols ? nt * 8 + g : 0);
        const int i = query_of(p, s, col), h = head * p.per + col - i * p.per;
        const uint8_t *src =
            static_cast<const uint8_t *>(p.q) + ((s.q0 + i) * p.q_stride + (int64_t)h * 128 + 32 * c) * 2;
#pragma unroll
        for (int k = 0; k < 4; ++k) qv[nt][k] = ld_keep16(src + 16 * k);
    }

    // ---- groups of the warp's chunks, 32 groups at a time: lane kChunkGroups
    // i + j holds where group j of chunk i lies in the cache (-1: nowhere)
    auto token_of = [&](int batch) {
        return t0 + (first + step * (batch * kBatch + lane / kChunkGroups)) * kChunk + lane % kChunkGroups * 16;
    };
    // the page id of the batch's token, or of the part's first token where
    // it has none; and the place, once the id is there
    auto find = [&](int batch) {
        const int token = token_of(batch);
        return ld_s32(p.table + (int64_t)b * p.table_stride + ((token < t1 ? token : t0) >> 4) / p.groups);
    };
    auto place = [&](int batch, int id) {
        const int token = token_of(batch), slot = token >> 4;
        return token < t1 && id >= 0 && id < p.num_pages
                   ? (int)(((int64_t)id * p.hk + head) * p.groups + slot % p.groups)
                   : -1;
    };
    auto fetch = [&](int i, int from, uint32_t stage) {  // starts the copies of chunk i
#pragma unroll
        for (int gr = 0; gr < kChunkGroups; ++gr) {
            const int at = __shfl_sync(0xFFFFFFFFu, from, i % kBatch * kChunkGroups + gr);
            if (at >= 0 && i < chunks) {
                const uint8_t *src = p.pool + (int64_t)at * kKVGroupBytes + lane * 16;
                const uint32_t d = stage + gr * kKVGroupBytes;
                cp16_at<0, 0>(d + w.kdst, src);
                cp16_at<512, 512>(d + w.kdst, src);
                cp16_at<0, 1024>(d + w.vdst, src);
                cp16_at<512, 1536>(d + w.vdst, src);
                if (lane < 16) cp16_at<0, 2048>(d + w.fdst, src);
            }
        }
        cp_async_commit();
    };
    int near_id = -1, far_id = -1;
    if (t1 > t0) {
        near_id = find(0);
        far_id = find(1);
    }
    int near = place(0, near_id);
    for (int i = 0; i < kStages - 1; ++i) fetch(i, near, i * kChunkBytes);
    uint32_t near_ok = __ballot_sync(0xFFFFFFFFu, near >= 0);
    int far = -1;  // from the chunk on whose fetch needs it
    uint32_t stage = 0, filled = (kStages - 1) * kChunkBytes;  // of chunk it, of the next to fetch

    // ---- queries as the B operand; each row by a power of two so that fp16
    // holds it
    uint32_t qf[NT][16];
    float cs[NT][2], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        uint4 (&v)[4] = qv[nt];
        float f = 1.0f, back = 1.0f;
        if (std::is_same<DT, BF16>::value) {
            float a = 0.0f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float e[8];
                unpack8<DT>(v[k], e);
#pragma unroll
                for (int j = 0; j < 8; ++j) a = fmaxf(a, fabsf(e[j]));
            }
            a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, 1));
            a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, 2));
            const float2 pw = row_power(a);
            f = pw.x;
            back = pw.y;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (std::is_same<DT, BF16>::value) {
                float e[8];
                unpack8<DT>(v[k], e);
#pragma unroll
                for (int j = 0; j < 8; ++j) e[j] *= f;
                v[k] = pack8<FP16>(e);
            }
            qf[nt][4 * k] = v[k].x;
            qf[nt][4 * k + 1] = v[k].y;
            qf[nt][4 * k + 2] = v[k].z;
            qf[nt][4 * k + 3] = v[k].w;
        }
        const float scale = fmaxf(p.scale * inv_kgs * back, kLeastScale);
        cs[nt][0] = __shfl_sync(0xFFFFFFFFu, scale, 8 * c);
        cs[nt][1] = __shfl_sync(0xFFFFFFFFu, scale, 8 * c + 4);
        m[nt][0] = m[nt][1] = kNoMax;
        l[nt][0] = l[nt][1] = 0.0f;
    }
    float o[NT][8][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nt][j][e] = 0.0f;

    for (int it = 0; it < chunks; ++it) {
        cp_async_wait<kStages - 2>();
        __syncwarp();  // everyone's copies have landed; everyone is done with the stage before
        if (it > 0 && it % kBatch == 0) {
            near = far;
            far_id = find(it / kBatch + 1);
            near_ok = __ballot_sync(0xFFFFFFFFu, near >= 0);
        }
        if (it % kBatch == kBatch - kStages + 1) far = place(it / kBatch + 1, far_id);
        fetch(it + kStages - 1, it % kBatch + kStages - 1 < kBatch ? near : far, filled);
        const int tok0 = t0 + (first + step * it) * kChunk;
        const uint32_t here = near_ok >> (it % kBatch * kChunkGroups);  // bit gr: the group is readable
        const bool full = tok0 >= need_lo && tok0 + kChunk <= need_hi && (here & kAll) == kAll;

        // ---- S^T = K Q^T, the two groups' chains of products side by side
        float x[kChunkGroups][NT][4];
        uint4 ka[kChunkGroups], kb[kChunkGroups];
        uint32_t sa[kChunkGroups], sb[kChunkGroups];
#pragma unroll
        for (int gr = 0; gr < kChunkGroups; ++gr) {
            const uint32_t base = stage + gr * kKVGroupBytes;
            ka[gr] = lds16_at<0>(base + w.kread);
            kb[gr] = lds16_at<512>(base + w.kread);
            sa[gr] = lds2_at<0>(base + w.ksread);
            sb[gr] = lds2_at<64>(base + w.ksread);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[gr][nt][e] = 0.0f;
        }
#pragma unroll
        for (int gr = 0; gr < kChunkGroups; ++gr) {
            sa[gr] = e4m3_pair(sa[gr]);
            sb[gr] = e4m3_pair(sb[gr]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
#pragma unroll
            for (int gr = 0; gr < kChunkGroups; ++gr) {
                const uint32_t wa = k == 0 ? ka[gr].x : k == 1 ? ka[gr].y : k == 2 ? ka[gr].z : ka[gr].w;
                const uint32_t wb = k == 0 ? kb[gr].x : k == 1 ? kb[gr].y : k == 2 ? kb[gr].z : kb[gr].w;
                const uint32_t fa = __byte_perm(sa[gr], sa[gr], k < 2 ? 0x1010 : 0x3232);
                const uint32_t fb = __byte_perm(sb[gr], sb[gr], k < 2 ? 0x1010 : 0x3232);
                uint32_t u[8] = {e2m1_pair<0>(wa), e2m1_pair<0>(wb), e2m1_pair<1>(wa), e2m1_pair<1>(wb),
                                 e2m1_pair<2>(wa), e2m1_pair<2>(wb), e2m1_pair<3>(wa), e2m1_pair<3>(wb)};
#pragma unroll
                for (int i = 0; i < 8; ++i) u[i] = FP16::mul2(u[i], i & 1 ? fb : fa);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma(x[gr][nt], u[0], u[1], u[2], u[3], qf[nt][4 * k], qf[nt][4 * k + 1]);
                    mma(x[gr][nt], u[4], u[5], u[6], u[7], qf[nt][4 * k + 2], qf[nt][4 * k + 3]);
                }
            }
        }

        // ---- probabilities 2^(x - m)
        uint32_t hidden = 0;  // bit (gr, nt, e): the key is not seen by the column
        if (!full) {
#pragma unroll
            for (int gr = 0; gr < kChunkGroups; ++gr)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int t = tok0 + gr * 16 + tok_of_row(g) + (e >> 1) * 8;
                        const int col = nt * 8 + 2 * c + (e & 1);
                        const int pos = s.first_pos + query_of(p, s, col0 + col);
                        const bool seen = (here >> gr & 1u) && col < cols && t <= pos &&
                                          (p.window == 0 || t > pos - p.window);
                        hidden |= (uint32_t)!seen << ((gr * NT + nt) * 4 + e);
                    }
        }
        float y[kChunkGroups][NT][4], sum[NT][2];
        bool high = false;
        auto exps = [&](int nt) {
#pragma unroll
            for (int gr = 0; gr < kChunkGroups; ++gr)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    y[gr][nt][e] = fmaf(x[gr][nt][e], cs[nt][e & 1], -m[nt][e & 1]);
            if (!full) {
#pragma unroll
                for (int gr = 0; gr < kChunkGroups; ++gr)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (hidden & (1u << ((gr * NT + nt) * 4 + e))) y[gr][nt][e] = -INFINITY;
            }
            sum[nt][0] = sum[nt][1] = 0.0f;
#pragma unroll
            for (int gr = 0; gr < kChunkGroups; ++gr)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    y[gr][nt][e] = ex2(y[gr][nt][e]);
                    sum[nt][e & 1] += y[gr][nt][e];
                }
            high |= sum[nt][0] > kPMax || sum[nt][1] > kPMax;
        };
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) exps(nt);
        if (__any_sync(0xFFFFFFFFu, high)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float top = kNoMax;
#pragma unroll
                    for (int gr = 0; gr < kChunkGroups; ++gr)
#pragma unroll
                        for (int e = k; e < 4; e += 2)
                            if (!(hidden & (1u << ((gr * NT + nt) * 4 + e))))
                                top = fmaxf(top, x[gr][nt][e] * cs[nt][k]);
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
                    const float now = fmaxf(m[nt][k], top);
                    const float f = ex2(m[nt][k] - now);
                    m[nt][k] = now;
                    l[nt][k] *= f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        o[nt][j][k] *= f;
                        o[nt][j][k + 2] *= f;
                    }
                }
                exps(nt);
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            l[nt][0] += sum[nt][0];
            l[nt][1] += sum[nt][1];
        }
        uint32_t pf[kChunkGroups][NT][2];
#pragma unroll
        for (int gr = 0; gr < kChunkGroups; ++gr)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                pf[gr][nt][0] = transpose8x8(FP16::pack(y[gr][nt][0], y[gr][nt][1]));
                pf[gr][nt][1] = transpose8x8(FP16::pack(y[gr][nt][2], y[gr][nt][3]));
            }

        // ---- O^T += V^T P^T
#pragma unroll
        for (int gr = 0; gr < kChunkGroups; ++gr) {
            const uint32_t base = stage + gr * kKVGroupBytes;
            const uint2 v0 = lds8_at<0>(base + w.vread), v1 = lds8_at<256>(base + w.vread);
            const uint2 v2 = lds8_at<512>(base + w.vread), v3 = lds8_at<768>(base + w.vread);
            uint32_t f01 = lds1_at<0>(base + w.vsread) | (lds1_at<32>(base + w.vsread) << 8);
            uint32_t f23 = lds1_at<64>(base + w.vsread) | (lds1_at<96>(base + w.vsread) << 8);
            if (!full) {  // bytes of keys that nobody sees may be anything
                const int t = tok0 + gr * 16 + c;
                const int blk_lo = p.window > 0 ? max(0, need_hi - p.window) : 0;
                const uint32_t n = here >> gr & 1u ? blk_hi - blk_lo : 0, at = t - blk_lo;
                if (at >= n) f01 &= 0xFF00u;
                if (at + 4 >= n) f01 &= 0x00FFu;
                if (at + 8 >= n) f23 &= 0xFF00u;
                if (at + 12 >= n) f23 &= 0x00FFu;
            }
            const uint32_t sa = e4m3_pair(f01), sb = e4m3_pair(f23);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t w0 = k ? v0.y : v0.x, w1 = k ? v1.y : v1.x;
                const uint32_t w2 = k ? v2.y : v2.x, w3 = k ? v3.y : v3.x;
                const uint32_t lo = 0x0F0F0F0Fu;
                const uint32_t ea = (w0 & lo) | ((w1 << 4) & ~lo), oa = ((w0 >> 4) & lo) | (w1 & ~lo);
                const uint32_t eb = (w2 & lo) | ((w3 << 4) & ~lo), ob = ((w2 >> 4) & lo) | (w3 & ~lo);
                uint32_t u[16] = {e2m1_pair<0>(ea), e2m1_pair<0>(oa), e2m1_pair<0>(eb), e2m1_pair<0>(ob),
                                  e2m1_pair<1>(ea), e2m1_pair<1>(oa), e2m1_pair<1>(eb), e2m1_pair<1>(ob),
                                  e2m1_pair<2>(ea), e2m1_pair<2>(oa), e2m1_pair<2>(eb), e2m1_pair<2>(ob),
                                  e2m1_pair<3>(ea), e2m1_pair<3>(oa), e2m1_pair<3>(eb), e2m1_pair<3>(ob)};
#pragma unroll
                for (int i = 0; i < 16; ++i) u[i] = FP16::mul2(u[i], i & 2 ? sb : sa);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma(o[nt][4 * k + i], u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3], pf[gr][nt][0],
                            pf[gr][nt][1]);
            }
        }
        stage = stage == (kStages - 1) * kChunkBytes ? 0 : stage + kChunkBytes;
        filled = filled == (kStages - 1) * kChunkBytes ? 0 : filled + kChunkBytes;
    }

    // ---- join the warps: O of column k in the warp's ring, 512 bytes each
    cp_async_wait<0>();
    __syncwarp();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float sum = l[nt][k];
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
            const int col = nt * 8 + 2 * c + k;
            if (g == 0) stats[col] = make_float2(m[nt][k], sum);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                *reinterpret_cast<float2 *>(w.o + col * 128 + 16 * g + 2 * j) =
                    make_float2(o[nt][j][k], o[nt][j][k + 2]);
        }
}

template <typename DT, int NT>
__global__ void __launch_bounds__(kThreads, (NT == 1 ? 16 : 8) / kWarps)
paged_attn_split_kernel(const PagedAttnParams p)
{
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int64_t scan[kWarps];
    __shared__ int start_seq;
    __shared__ int64_t start_rem;
    __shared__ float2 stats[kWarps][8 * NT];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    PartInfo *info = reinterpret_cast<PartInfo *>(p.workspace + kTakenBytes) + 2 * blockIdx.x;
    float *parts = reinterpret_cast<float *>(p.workspace + kTakenBytes + kInfoBytes) +
                   (int64_t)blockIdx.x * 2 * kPartFloats<NT>;

    // ---- this CTA's share: units (head, block, chunk of keys) of all
    // sequences in order, each item (head, block) begun by kStart units that
    // stand for its overhead, cut into equal runs.  Thread t adds up the units of
    // its run of sequences; the thread whose run holds the first unit finds it.
    const int per_thread = (p.n_seqs + kThreads - 1) / kThreads;
    const int b0 = min(p.n_seqs, (int)threadIdx.x * per_thread), b1 = min(p.n_seqs, b0 + per_thread);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) mine += seq_units<NT>(p, load_seq(p, b));
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) scan[warp] = upto;
    __syncthreads();
    int64_t total = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w == warp) upto += total;
        total += scan[w];
    }
    // at least a chunk per warp, where there is enough
    const int n = (int)max((int64_t)1, min((int64_t)gridDim.x, total / kWarps));
    const int64_t i0 = blockIdx.x, each = div_small(total, n), more = total - each * n;
    int64_t u = i0 < n ? each * i0 + min(i0, more) : total;
    const int64_t u_end = i0 < n ? u + each + (i0 < more) : total;
    if (upto - mine <= u && u < upto) {
        int64_t rem = u - (upto - mine);
        int b = b0;
        for (;; ++b) {
            const int64_t w = seq_units<NT>(p, load_seq(p, b));
            if (rem < w) break;
            rem -= w;
        }
        start_seq = b;
        start_rem = rem;
    }
    if (threadIdx.x < 2) info[threadIdx.x].valid = 0;
    if (blockIdx.x == 0)
        for (size_t i = threadIdx.x; i < kTakenBytes / 4; i += kThreads) reinterpret_cast<unsigned *>(p.workspace)[i] = 0;
    __syncthreads();
    if (u >= u_end) return;
    int b = start_seq;
    int64_t rem = start_rem;

    const WarpRing ring(smem + warp * (kStages * kChunkBytes));
    const float inv_kgs = 1.0f / ld_f32(p.k_gs);

    Seq s = load_seq(p, b);
    Cut ct = cut<NT>(p, s);
    while (u < u_end) {
        const int cost = ct.tiles + kStart;
        const int64_t all = (int64_t)p.hk * ct.blocks * cost;
        if (rem >= all) {
            rem -= all;
            s = load_seq(p, ++b);
            ct = cut<NT>(p, s);
            continue;
        }
        const int item = (int)div_small(rem, cost), from = (int)(rem - (int64_t)item * cost);
        const int take = (int)min((int64_t)(cost - from), u_end - u);
        u += take;
        rem += take;
        const int tile0 = max(0, from - kStart), ntile = from + take - kStart - tile0;
        if (ntile <= 0) continue;  // no more than the item's overhead
        const int head = item / ct.blocks, block = item - head * ct.blocks;
        const int col0 = block * 8 * NT, cols = min(8 * NT, s.nq * p.per - col0);
        const int t0 = s.lo + tile0 * kChunk;
        const float v_gs = ld_f32(p.v_gs);
        attend<DT, NT>(p, s, b, head, col0, cols, t0, t0 + ntile * kChunk, warp, kWarps, inv_kgs, ring, stats[warp]);
        __syncthreads();
        constexpr int kPerCol = kThreads / (8 * NT), kVals = 128 / kPerCol;
        const int col = threadIdx.x / kPerCol, d0 = (threadIdx.x % kPerCol) * kVals;
        if (col < cols) {
            float top = kNoMax, sum = 0.0f, v[kVals] = {};
#pragma unroll
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, stats[w][col].x);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = ex2(stats[w][col].x - top);
                sum += f * stats[w][col].y;
                const float *src = reinterpret_cast<const float *>(smem + w * (kStages * kChunkBytes) +
                                                                   col * 512) + d0;
#pragma unroll
                for (int k = 0; k < kVals; ++k) v[k] = fmaf(f, src[k], v[k]);
            }
            if (ntile == ct.tiles) {
                store_out<DT, kVals>(p, s, head, col0 + col, d0, v, top, sum, v_gs);
            } else {
                float *part = parts + (tile0 == 0 ? kPartFloats<NT> : 0);
#pragma unroll
                for (int k = 0; k < kVals; ++k) part[col * 128 + d0 + k] = v[k];
                if (d0 == 0) {
                    part[8 * NT * 128 + col] = top;
                    part[8 * NT * 129 + col] = sum;
                }
            }
        }
        if (threadIdx.x == 0 && ntile != ct.tiles)
            info[tile0 == 0] = PartInfo{1, tile0 + ntile == ct.tiles, b, head, block};
        __syncthreads();
    }
}

// The same for calls that are short: a cluster of kCluster CTAs takes an item, its
// warps the item's chunks in turn, and the parts join through the cluster's
// shared memory, in one launch.  What bounds it is latency: 1 sequence of 1000
// keys (a chunk a warp) 5.1 us in a graph.
template <typename DT, int NT>
__global__ void __launch_bounds__(kThreads, (NT == 1 ? 16 : 8) / kWarps)
paged_attn_cluster_kernel(const PagedAttnParams p)
{
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float2 stats[kWarps][8 * NT];
    pdl_trigger();
    pdl_wait();
    const int warp = threadIdx.x >> 5, rank = blockIdx.x % kCluster;
    const int pair = blockIdx.x / kCluster, b = pair / p.hk, head = pair - b * p.hk;
    const Seq s = load_seq(p, b);
    const float inv_kgs = 1.0f / ld_f32(p.k_gs), v_gs = ld_f32(p.v_gs);
    const WarpRing ring(smem + warp * (kStages * kChunkBytes));
    const int columns = s.nq * p.per;
    for (int col0 = 0; col0 < columns; col0 += 8 * NT) {
        const int cols = min(8 * NT, columns - col0);
        attend<DT, NT>(p, s, b, head, col0, cols, s.lo, s.hi, rank * kWarps + warp, kCluster * kWarps, inv_kgs, ring,
                       stats[warp]);
        cluster_sync();
        // column rank (and rank + 8): a thread a channel over all warps' parts
        for (int col = rank; col < cols; col += kCluster) {
            float m[kParts], l[kParts], o[kParts], top = kNoMax, sum = 0.0f, v = 0.0f;
#pragma unroll
            for (int i = 0; i < kParts; ++i) {
                const uint32_t at = cluster_addr(&stats[i % kWarps][col], i / kWarps);
                m[i] = ld_cluster(at);
                l[i] = ld_cluster(at + 4);
            }
#pragma unroll
            for (int i = 0; i < kParts; ++i)
                o[i] = ld_cluster(cluster_addr(smem + i % kWarps * (kStages * kChunkBytes), i / kWarps) +
                                  (col * 128 + threadIdx.x) * 4);
#pragma unroll
            for (int i = 0; i < kParts; ++i) top = fmaxf(top, m[i]);
#pragma unroll
            for (int i = 0; i < kParts; ++i) {
                const float f = ex2(m[i] - top);
                sum = fmaf(f, l[i], sum);
                v = fmaf(f, o[i], v);
            }
            const int at = col0 + col, i = query_of(p, s, at);
            const int64_t row = (int64_t)(s.q0 + i) * p.hq + head * p.per + at - i * p.per;
            const float x = v * out_factor(sum, v_gs);
            static_cast<uint16_t *>(p.out)[row * 128 + threadIdx.x] = (uint16_t)DT::pack(x, 0.0f);
            if (p.lse != nullptr && threadIdx.x == 0) p.lse[row] = lse_of(top, sum);
        }
        cluster_sync();  // the parts have been read
    }
}

// Joins the parts of items that CTAs of the kernel above share.  CTA i looks
// at the item whose first part CTA i of that kernel left, if any, and at the
// parts of the CTAs after it up to the one that ends the item.  A warp takes
// columns of the item, a lane 4 channels.
template <typename DT, int NT>
__global__ void __launch_bounds__(256)
paged_attn_join_kernel(const PagedAttnParams p, int ctas)
{
    __shared__ int last;
    pdl_trigger();
    pdl_wait();
    const PartInfo *info = reinterpret_cast<const PartInfo *>(p.workspace + kTakenBytes);
    const int i = blockIdx.x;
    const PartInfo me = info[2 * i + 1];
    if (!me.valid) return;
    if (threadIdx.x == 0) last = ctas - 1;
    __syncthreads();
    for (int j = i + 1 + threadIdx.x; j < ctas; j += blockDim.x)
        if (info[2 * j].valid && info[2 * j].last) atomicMin(&last, j);
    __syncthreads();
    const int end = last, n = end - i + 1;
    const float *parts = reinterpret_cast<const float *>(p.workspace + kTakenBytes + kInfoBytes);
    auto part = [&](int k) {  // the k-th part of the item
        return parts + ((int64_t)(i + k) * 2 + (k == 0)) * kPartFloats<NT>;
    };
    const Seq s = load_seq(p, me.seq);
    const float v_gs = ld_f32(p.v_gs);
    const int lane = threadIdx.x & 31, d0 = lane * 4;
    for (int col = threadIdx.x >> 5; col < 8 * NT; col += 8) {
        const int at = me.block * 8 * NT + col;
        if (at >= s.nq * p.per) break;
        float top = kNoMax;
        for (int k = lane; k < n; k += 32) top = fmaxf(top, part(k)[8 * NT * 128 + col]);
        top = group_max<32>(top);
        float sum = 0.0f, v[4] = {};
        constexpr int kU = 8;
        for (int k0 = 0; k0 < n; k0 += kU) {
            float4 a[kU];
            float f[kU], ll[kU];
#pragma unroll
            for (int k = 0; k < kU; ++k) {
                const float *src = part(min(k0 + k, n - 1));
                a[k] = *reinterpret_cast<const float4 *>(src + col * 128 + d0);
                f[k] = src[8 * NT * 128 + col];
                ll[k] = src[8 * NT * 129 + col];
            }
#pragma unroll
            for (int k = 0; k < kU; ++k) {
                const float w = k0 + k < n ? ex2(f[k] - top) : 0.0f;
                sum = fmaf(w, ll[k], sum);
                v[0] = fmaf(w, a[k].x, v[0]);
                v[1] = fmaf(w, a[k].y, v[1]);
                v[2] = fmaf(w, a[k].z, v[2]);
                v[3] = fmaf(w, a[k].w, v[3]);
            }
        }
        store_out<DT, 4>(p, s, me.head, at, d0, v, top, sum, v_gs);
    }
}

template <typename DT, int NT>
cudaError_t launch_split(const PagedAttnParams &p, int dev, cudaStream_t stream)
{
    static std::atomic<int> occ_cache[64];
    auto kern = paged_attn_split_kernel<DT, NT>;
    int per_sm = dev < 64 ? occ_cache[dev].load(std::memory_order_relaxed) : 0;
    if (per_sm <= 0) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e == cudaSuccess)
            e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kThreads, kSmem);
        if (e != cudaSuccess) return e;
        if (per_sm < 1) return cudaErrorInvalidConfiguration;
        if (dev < 64) occ_cache[dev].store(per_sm, std::memory_order_relaxed);
    }
    const int full = device_sms(dev) * per_sm, grid = full < kMaxCtas ? full : kMaxCtas;
    cudaError_t e = launch_pdl(kern, grid, kThreads, kSmem, stream, p);
    if (e != cudaSuccess) return e;
    return launch_pdl(paged_attn_join_kernel<DT, NT>, grid, 256, 0, stream, p, grid);
}

template <typename DT, int NT>
cudaError_t launch_cluster(const PagedAttnParams &p, int dev, cudaStream_t stream)
{
    static_assert(kThreads == 128, "the join takes a thread a channel");
    static std::atomic<int> ready[64];
    auto kern = paged_attn_cluster_kernel<DT, NT>;
    if (dev >= 64 || !ready[dev].load(std::memory_order_relaxed)) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready[dev].store(1, std::memory_order_relaxed);
    }
    return launch_pdl_cluster(kern, (unsigned)(p.n_seqs * p.hk), kCluster, kThreads, kSmem, stream, p);
}

// Whether the cluster form is taken: all its CTAs run at once, and the table has
// no room for sequences so long that cutting them finer pays.  Measured, with the
// split form in brackets.  8 KV heads of 2 queries: 1 sequence of 100, 1000, 4000,
// 16,000 and 32,000 keys 5.3, 5.3, 7.8, 18.2 and 31.7 us (6.9, 9.0, 11.3, 18.5
// and 21.8), 4 of 1000, 8000 and 16,000 7.7, 18.8 and 31.8 (10.5, 18.3 and 24.6),
// 9 of 100, 1000, 4000 and 16,000 8.7, 9.0, 13.4 and 36 (7.2, 12.6, 19.0 and 45).
// 1 KV head of 8, 72 sequences of 100, 1000 and 16,000 12.4, 13.6 and 39 (7.3,
// 14.1 and 47).  2 KV heads of 16: 9 sequences of 100, 1000, 4000 and 16,000 10.2,
// 11.0, 13.8 and 28.5 (8.7, 14.7, 18.9 and 26.8), 18 of 1000 and 4000 16.6 and
// 22.0 (15.9 and 20.9).  So to 8000 keys it wins but for the very short ones; at
// 16,000 it is 0.8 to 1.5 times as fast, and the limit is a table's room, that
// most sequences do not fill.  The lengths are on the device: the host cannot
// choose by them.
template <int NT>
bool is_short(const PagedAttnParams &p, int dev)
{
    return (int64_t)p.n_seqs * p.hk * kCluster <= (NT == 1 ? 4 : 1) * device_sms(dev) && p.max_keys <= 16384;
}

// Whether the tensor-memory kernel is faster for the runs of queries.  Both
// kernels' times go with the keys: here a block of 16 columns takes 35 ps a key,
// spread over every SM, there one of 256 rows 11.7 ns on one SM or, where blocks
// are few, on up to 8 (the join 3 us a part).  Measured (here, there) in us: 4
// sequences of 30,000 keys, 2 KV heads and 48, 128, 256 and 512 columns 42, 82, 148
// and 280 (91, 90, 80 and 81), 8 heads and 48, 128, 256 and 512 116, 281, 542 and
// 1066 (147, 141, 129 and 217); 16 of 1000 keys, 8 heads and the same 37, 73, 132
// and 248 (28, 28, 27 and 46); 1 of 4000 keys, 8 heads and 512 columns 58 (41).
// The keys are the table's room, up to 8192: most sequences do not fill a wider
// one.
bool runs_pay(const PagedAttnParams &p, int sms)
{
    const int64_t rows = (int64_t)p.per * p.n_tokens;
    double keys = p.max_keys < 8192 ? p.max_keys : 8192;
    if (p.window > 0 && keys > p.window + p.max_q) keys = p.window + p.max_q;
    const double blocks16 = (double)(rows / 16 + p.n_seqs) * p.hk, blocks = (double)(rows / 256 + p.n_seqs) * p.hk;
    double parts = kSharedBlocks / blocks < 8 ? kSharedBlocks / blocks : 8;
    if (parts > keys / 1024) parts = keys / 1024;
    const double waves = blocks > sms ? blocks / sms : 1;
    const double there = parts >= 2 ? 15 + 0.0117 * keys / parts + 3 * parts : 15 + 0.0117 * keys * waves;
    return there < 14 + 3.5e-5 * blocks16 * keys;
}

}  // namespace

size_t paged_attn_workspace_bytes(int, int)
{
    return kTakenBytes + kInfoBytes + (size_t)kMaxCtas * 2 * kPartFloats<2> * sizeof(float);
}

template <typename DT>
cudaError_t launch_paged_attn(const PagedAttnParams &p, cudaStream_t stream)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    // 8 columns hold the queries of a KV head, or 16 do (one pass over the
    // keys instead of two)
    const int64_t cols = (int64_t)p.per * p.max_q;
    PagedAttnParams few = p;
    few.few = INT_MAX;
    if (cols <= 8)
        return is_short<1>(few, dev) ? launch_cluster<DT, 1>(few, dev, stream) : launch_split<DT, 1>(few, dev, stream);
    if (p.q_starts == nullptr || cols <= kFewColumns || !runs_pay(p, device_sms(dev)))
        return cols <= 16 && is_short<2>(few, dev) ? launch_cluster<DT, 2>(few, dev, stream)
                                                : launch_split<DT, 2>(few, dev, stream);
    few.few = kFewColumns;
    e = launch_split<DT, 2>(few, dev, stream);
    return e != cudaSuccess ? e : launch_paged_attn_tc<DT>(few, kInfoBytes, stream);
}

template cudaError_t launch_paged_attn<BF16>(const PagedAttnParams &, cudaStream_t);
template cudaError_t launch_paged_attn<FP16>(const PagedAttnParams &, cudaStream_t);

}  // namespace rq
