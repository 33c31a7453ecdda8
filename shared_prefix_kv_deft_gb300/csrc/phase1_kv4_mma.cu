// phase1_kv4_mma.cu -- phase-1 partial attention over a 4-bit KV cache on
// tcgen05 tensor cores, for work items with 16 to 64 rows and head_dim 128
// (the other units: phase1_kv4.cu, with the mathematics that both share).
//
// Tokens on the MMA's M, rows on its N, as in the bf16 kernel:
//     S^T[128 tok x RP]  = K_tile . Q^T            (TMEM, fp32)
//     O^T[128 d   x RP] += V_tile^T . P^T          (TMEM, fp32)
// RP = 32 or 64.  The cache's 4 bits become fp16 once for all rows, K's in
// TMEM (the first operand of its product may lie there) and V's in shared
// memory: a thread takes half a row of K and of V of every tile (32 bytes and
// four scales each, fetched a tile ahead straight into registers), 128 rows a
// tile from wherever the chunk's tokens lie, none beside them.  At 64 rows a
// token costs a thread its unpacking (some 90 instructions for 64 elements of
// K and as many of V) and 32 exponentials; mma.sync, at an eighth of the
// tensor rate and with every fragment unpacked again for each 32 rows, took
// 182 us where this takes 99 (the step on a document of 32768 tokens with 64
// branches of 64 to 8192, 32/8 heads: 36 GFLOP), 44 where 30 (32 branches of
// 256 tokens on a prompt of 4096, 32/32 heads).
//
// A CTA of eight warps takes one unit, and two CTAs share an SM: one unpacks
// and exponentiates while the other waits.  All warps do the same work.  For
// tile t they unpack K(t + 1), read S(t) and take its exponents; one thread
// starts S(t + 1) into S's other buffer, all warps' K being there by then;
// they write P(t) once P(t - 1).V(t - 1) is done, unpack V(t), and vote at the
// tile's one barrier whether a column's maximum has to be raised (when a logit
// passes it by more than 2^4: O and the sums are then rescaled and P(t) is
// made again, before anything has used it); P(t).V(t) is started.  Sums of
// the weights stay with the threads until the end.  Every wait is bounded.
//
// S is read in the fragments of an MMA's rows (16x256b): a thread has four
// rows at RP / 8 columns, so that a column's sums, factors and maxima take a
// fourth of the registers and reads that a row a thread would take, and S is
// read once.
//
// What bounds it is the tile's chain: 2.1 us for 128 tokens of a unit, two
// units an SM (hardly less for one alone), of which the tensor products are a
// fifth and the issue slots under half: 516 instructions a warp and tile, 128
// of them the conversions and products of the unpacking.  Measured and left:
// one CTA an SM with twice the registers (155 us where two had 109), 512
// threads with a quarter row each (231: 64 registers spill), fewer registers
// than 128, for room beside the other launch (111 to 126), S's read under K's
// unpacking (107 where 99: eight spilled words), the rows through asynchronous
// copies in shared memory (106 to 109), the products started by other warps
// than the first (99).
#include <cfloat>

#include "kv4.cuh"
#include "kv4_internal.h"
#include "merge.cuh"
#include "tcgen05.cuh"

namespace deft {
namespace {

constexpr int kThreads = 256;
constexpr int kD = 128, kTile = 128;
constexpr unsigned kAll = 0xffffffffu;
constexpr uint32_t kRowGroup = 2048;    // 8 tokens x 128 dims of fp16: two 1 KB swizzle atoms (d halves)
constexpr uint32_t kTileBytes = 16 * kRowGroup;
constexpr uint32_t kTmemCols = 256;     // S at 0 and 64, O at 128, K's tile (fp16 pairs) at 192

template <int RP>
struct Cfg {
    static constexpr uint32_t v = 0;                            // [16 groups][d half][8 tok][128 B]
    static constexpr uint32_t p = v + kTileBytes;               // [128 tok][128 B]
    static constexpr uint32_t q_half = RP * 128;
    static constexpr uint32_t q = p + kTile * 128;              // [d half][RP rows][128 B]
    static constexpr uint32_t col = q + 2 * q_half;             // [RP / 2] two columns' factors, their lift - maximum
    static constexpr uint32_t red = col + RP * 8;               // [4 warps][RP]
    static constexpr uint32_t seg = red + 4 * RP * 4;           // [256] position, page, begin; [256] mask (8 B)
    static constexpr uint32_t misc = seg + kMaxSegsPerChunk * 20;   // TMEM base
    static constexpr uint32_t bars = misc + 16;                 // S, O, K, end
    static constexpr uint32_t total = bars + 32;
    static constexpr uint32_t alloc = total + 1024;
    static_assert(q % 1024 == 0 && p % 1024 == 0, "128-byte-swizzle atoms");
    static_assert(2 * (alloc + 1024) <= 228 * 1024, "two CTAs an SM");
};

// kind::f16 with fp16 A and B, fp32 D.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int a_mn, int b_mn)
{
    return tc::idesc_bf16(M, N, a_mn, b_mn) & ~((1u << 7) | (1u << 10));
}

// tc::tmem_st16 without the wait.
__device__ __forceinline__ void tmem_put(uint32_t addr, const float (&v)[16])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
                 "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]), "f"(v[10]),
                 "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
                 : "memory");
}

// Half a token's row: 64 elements and their scales.
struct HalfRow {
    uint4 w[2];
    uint32_t s;
    // row: the half row's place; tok: of the page.
    __device__ __forceinline__ void load(const uint8_t *row, int tok, int half)
    {
        using P = kv4::Page<kD>;
        w[0] = __ldg(reinterpret_cast<const uint4 *>(row));
        w[1] = __ldg(reinterpret_cast<const uint4 *>(row) + 1);
        const uint8_t *sc = row + (P::kScales - tok * (P::kRow - P::kScaleRow) - half * (P::kRow - P::kScaleRow) / 2);
        s = __ldg(reinterpret_cast<const uint32_t *>(sc));
    }
    // Words 4 b .. 4 b + 3 as fp16, eight elements each.
    template <typename F>
    __device__ __forceinline__ void each(int b, F f) const
    {
        const uint32_t x[4] = {w[b].x, w[b].y, w[b].z, w[b].w};
        const uint32_t a = kv4::scales2(b == 0 ? s : s >> 16);
        const uint32_t sc[2] = {__byte_perm(a, 0, 0x1010), __byte_perm(a, 0, 0x3232)};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t h[4];
            kv4::unpack8(x[i], h);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                h[k] = kv4::hmul2(h[k], sc[i / 2]);
            f(i, h);
        }
    }
    // Into the swizzled row at `dst` (row r of its group of eight).
    __device__ __forceinline__ void to_smem(uint8_t *dst, int r) const
    {
#pragma unroll
        for (int b = 0; b < 2; ++b)
            each(b, [&](int i, const uint32_t (&h)[4]) {
                *reinterpret_cast<uint4 *>(dst + (((4 * b + i) ^ r) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
            });
    }
    // Into 32 columns of the thread's TMEM lane.
    __device__ __forceinline__ void to_tmem(uint32_t addr) const
    {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            float v[16];
            each(b, [&](int i, const uint32_t (&h)[4]) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    v[4 * i + k] = __uint_as_float(h[k]);
            });
            tmem_put(addr + 16 * b, v);
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
    }
};

// D[tmem] (+)= A[tmem] . B[smem], kind::f16.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile("{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
                 "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
                 : "memory");
}

// Lanes 0-15 of the warp's 32, from `addr` on: lane (g, t) = (lane / 4, lane %
// 4) gets rows g and g + 8 at columns 8 j + 2 t and + 1: v[4 j], v[4 j + 1],
// v[4 j + 2], v[4 j + 3].  Valid after tmem_got.
__device__ __forceinline__ void tmem_get(uint32_t addr, float (&v)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]),
                   "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
                 : "r"(addr));
}
__device__ __forceinline__ void tmem_get(uint32_t addr, float (&v)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "r"(addr));
}
__device__ __forceinline__ void tmem_got(float (&v)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]),
                   "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_got(float (&v)[8])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7])
                 :
                 : "memory");
}

// Four 8x8 blocks of fp16, a pair of row lane / 4 a lane in each: lane i has
// the address of row i of the 32 (16 bytes).
__device__ __forceinline__ void store_rows(uint32_t addr, const uint32_t (&w)[4])
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                 : "memory");
}

// The largest (a NaN counts for nothing).
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

template <int RP>
__global__ void __launch_bounds__(kThreads, 2) phase1_kv4_mma_kernel(Kv4Args ka, DevPartition p)
{
    using C = Cfg<RP>;
    using P = kv4::Page<kD>;
    constexpr int NC = RP / 2;      // columns of a warp
    constexpr int NJ = NC / 8;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw);
    const AttnArgs &a = ka.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int half = warp >> 2, row = (warp & 3) * 32 + lane, g = lane >> 2, t4 = lane & 3;    // tile row, half of its dims and of the columns
    float *col = reinterpret_cast<float *>(smem + C::col);
    // Column c's factor (logits in base 2 from S's numbers) and lift - maximum.
    auto col_f = [&](int c) -> float & { return col[2 * (c & ~1) + (c & 1)]; };
    auto col_y = [&](int c) -> float & { return col[2 * (c & ~1) + 2 + (c & 1)]; };
    float *red = reinterpret_cast<float *>(smem + C::red);
    int32_t *seg_pos = reinterpret_cast<int32_t *>(smem + C::seg), *seg_page = seg_pos + kMaxSegsPerChunk,
            *seg_begin = seg_page + kMaxSegsPerChunk;
    uint64_t *seg_mask = reinterpret_cast<uint64_t *>(seg_begin + kMaxSegsPerChunk);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::misc);
    const uint32_t bar_s = base + C::bars, bar_o = bar_s + 8, bar_k = bar_s + 16, bar_end = bar_s + 24;

    if (warp == 0) {
        tc::tmem_alloc(smem_u32(tmem_slot), kTmemCols);
        tc::tmem_relinquish();
    }
    if (tid == 0) {
        tc::mbar_init(bar_s, 1);
        tc::mbar_init(bar_o, 1);
        tc::mbar_init(bar_k, kThreads / 32);
        tc::mbar_init(bar_end, 1);
        tc::fence_mbar_init();
    }
    __syncthreads();
    if (a.wait_prior)
        grid_dep_wait();
    grid_dep_launch();

    // ---- the unit ----
    const int Hkv = a.num_kv_heads, Hq = a.num_q_heads, G = a.gqa_group;
    const int it = blockIdx.x / Hkv, h = blockIdx.x - it * Hkv, item = ka.first + it;
    const int32_t *triple = p.mma_items + 3 * (size_t)item;
    const int c = triple[0], qb = triple[1], R = (triple[2] - qb) * G;
    const int rm0 = p.mma_rmask_off[item];
    const int cq0 = p.chunk_q_off[c] + qb, T = p.chunk_tokens[c];
    const int sb = p.chunk_seg_off[c], nseg = p.chunk_seg_off[c + 1] - sb;
    for (int s = tid; s < nseg; s += kThreads) {
        const int tb = p.seg_tok_begin[sb + s];
        seg_pos[s] = p.seg_chunk_pos[sb + s];
        seg_page[s] = a.node_page_off[p.seg_node[sb + s]] + tb / kPageSize;
        seg_begin[s] = tb % kPageSize;
        const uint4 w = reinterpret_cast<const uint4 *>(p.mma_rmask)[rm0 + s];
        seg_mask[s] = (uint64_t)w.x | (uint64_t)w.z << (item < ka.mma_narrow ? 16 : 32);
    }
    // The thread's piece of a row of Q, on its way while the pages are looked up.
    constexpr int TPR = kThreads / RP, DT = kD / TPR;   // threads of a row, dims of a thread
    const int q_row = tid / TPR, piece = tid % TPR;
    uint32_t qw[DT / 2];
#pragma unroll
    for (int i = 0; i < DT / 2; ++i)
        qw[i] = 0u;
    if (q_row < R) {
        const int k = q_row / G;
        const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.q) +
                                                           ((size_t)p.chunk_q[cq0 + k] * Hq + h * G + (q_row - k * G)) * kD + piece * DT);
#pragma unroll
        for (int i = 0; i < DT / 8; ++i) {
            const uint4 x = src[i];
            qw[4 * i] = x.x, qw[4 * i + 1] = x.y, qw[4 * i + 2] = x.z, qw[4 * i + 3] = x.w;
        }
    }
    __syncthreads();    // the segments

    // ---- rows of the chunk ----
    const int ntiles = (T + kTile - 1) / kTile;
    const uint8_t *k4 = static_cast<const uint8_t *>(a.k_pages) + half * (P::kRow / 2);
    const uint8_t *v4 = static_cast<const uint8_t *>(a.v_pages) + half * (P::kRow / 2);
    struct Where {
        int page;
        int meta;           // segment x 16 + token of the page
    };
    // Of the chunk's token at the thread's row of tile t (past the last: the
    // last, which has no weight there).
    auto where = [&](int t) {
        const int x = min(t * kTile + row, T - 1);
        int seg = 0, hi = nseg;
        while (hi - seg > 1) {
            const int mid = (seg + hi) >> 1;
            if (seg_pos[mid] <= x)
                seg = mid;
            else
                hi = mid;
        }
        const int j = x - seg_pos[seg] + seg_begin[seg];
        Where w;
        w.page = a.page_id[seg_page[seg] + j / kPageSize];
        w.meta = seg * kPageSize + j % kPageSize;
        return w;
    };
    auto load = [&](HalfRow &x, const uint8_t *pool, const Where &w) {
        const int tok = w.meta % kPageSize;
        const uint32_t at = (uint32_t)w.page * (uint32_t)Hkv + h;   // (the step is refused where this could pass 32 bits)
        x.load(pool + ((size_t)at * P::kBytes + tok * P::kRow), tok, half);
    };
    HalfRow kr, vr;
    Where w0 = where(0), w1 = where(1), w2;     // of tiles t, t + 1, t + 2
    load(kr, k4, w0);
    load(vr, v4, w0);
    // ---- Q^T: bf16 -> fp16 times a power of two ----
    {
        float big = 0.f;            // the row's largest finite magnitude
        bool inf = false;
#pragma unroll
        for (int i = 0; i < DT / 2; ++i) {
            const float2 x = bf16x2_to_float2(qw[i] & 0x7fff7fffu);
            big = x.x < INFINITY ? fmaxf(big, x.x) : big;
            big = x.y < INFINITY ? fmaxf(big, x.y) : big;
            inf |= x.x == INFINITY || x.y == INFINITY;
        }
#pragma unroll
        for (int o = 1; o < TPR; o <<= 1)
            big = fmaxf(big, __shfl_xor_sync(kAll, big, o));
        const int e = big > 0.f ? 14 - ilogbf(big) : 0;
        // 2^e in two factors: e reaches from -113 to 147.
        const int e1 = e / 2, e2 = e - e1;
        // Infinities become NaN (with the elements beside them), so that a
        // logit of -inf is a masked one.
        const float up1 = inf ? kv4::nan() : kv4::pow2(e1), up2 = kv4::pow2(e2);
#pragma unroll
        for (int i = 0; i < DT / 8; ++i) {
            uint32_t x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 y = bf16x2_to_float2(qw[4 * i + j]);
                x[j] = kv4::f16x2(y.x * up1 * up2, y.y * up1 * up2);
            }
            const int chunk = piece * (DT / 8) + i;         // of the row's sixteen
            *reinterpret_cast<uint4 *>(smem + C::q + (chunk >> 3) * C::q_half + q_row * 128 + (((chunk & 7) ^ (q_row & 7)) << 4)) =
                make_uint4(x[0], x[1], x[2], x[3]);
        }
        // A column of no row has weights of 0: 2^(f * 0 - inf).
        if (piece == 0) {
            // (A factor past fp32, for a row near its end, leaves logits of 0.)
            col_f(q_row) = fminf(a.scale_log2 * kv4::pow2(-e1) * ka.k_scale * kv4::pow2(-e2), FLT_MAX);
            col_y(q_row) = q_row < R ? INFINITY : -INFINITY;
        }
    }
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const uint32_t tm_s = tmem + ((uint32_t)(warp & 3) << 21) + half * NC, tm_o = tm_s + 128;

    uint8_t *row_v = smem + C::v + (row >> 3) * kRowGroup + half * 1024 + (row & 7) * 128;
    const uint32_t tm_k = tmem + ((uint32_t)(warp & 3) << 21) + 192 + half * 32;
    const uint32_t row_bits = R >= RP ? 0xffffffffu >> (32 - NC)
                                      : (uint32_t)((((1ull << R) - 1) >> (half * NC)) & (0xffffffffu >> (32 - NC)));

    // Of S a thread holds columns 8 j + 2 t4 and + 1 (of the warp's) for rows
    // 16 h + 8 q + g: with a row a thread, the sums of 32 columns would take 32
    // registers and S would have to be read twice.
    float l[2 * NJ], x[2][2][2 * NJ];
#pragma unroll
    for (int j = 0; j < 2 * NJ; ++j)
        l[j] = 0.f;
    const float4 *my_col = reinterpret_cast<const float4 *>(col + half * 2 * NC + 4 * t4);
    const uint32_t p_row = base + C::p + row * 128;
    bool ok = true;
    kr.to_tmem(tm_k);
    load(kr, k4, w1);
    w2 = where(2);
    tc::fence_proxy_async();
    tc::fence_before_sync();
    __syncthreads();
    constexpr uint32_t idesc_s = idesc_f16(kTile, RP, 0, 0), idesc_o = idesc_f16(kD, RP, 1, 1);
    auto issue_s = [&](int t) {
        const uint64_t dq = tc::smem_desc(base + C::q, 16, 1024);
#pragma unroll
        for (int s = 0; s < 8; ++s)
            mma_ts(tmem + (t & 1) * 64, tmem + 192 + 8 * s, dq + (((s >> 2) * C::q_half + (s & 3) * 32) >> 4), idesc_s,
                   s > 0 ? 1u : 0u);
        tc::mma_commit(bar_s);
    };
    if (tid == 0) {
        tc::fence_after_sync();
        issue_s(0);
    }
    for (int t = 0; t < ntiles; ++t) {
        // ---- S(t) is there, and has been read from K's buffer: K(t + 1) ----
        if (ok)
            ok = tc::mbar_wait(bar_s, t & 1);
        tc::fence_after_sync();
        __syncwarp();
        if (t + 1 < ntiles) {
            kr.to_tmem(tm_k);
            load(kr, k4, w2);
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0)
                tc::mbar_arrive(bar_k);
        }
        const Where w3 = where(t + 3);      // (its page is looked up while the tile is worked on)
        uint32_t seen = 0;          // the thread's tile row's, by column
        if (t * kTile + row < T)
            seen = (uint32_t)(seg_mask[w0.meta / kPageSize] >> (half * NC)) & row_bits;
        const bool whole = __all_sync(kAll, seen == row_bits);
        const uint32_t tm_st = tm_s + (t & 1) * 64;
        auto read = [&]() {
            float v[2][4 * NJ];
            tmem_get(tm_st, v[0]);
            tmem_get(tm_st + (16u << 16), v[1]);
#pragma unroll
            for (int h2 = 0; h2 < 2; ++h2) {
                tmem_got(v[h2]);
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        x[h2][q][2 * j] = v[h2][4 * j + 2 * q];
                        x[h2][q][2 * j + 1] = v[h2][4 * j + 2 * q + 1];
                    }
            }
        };
        auto hide = [&]() {
#pragma unroll
            for (int h2 = 0; h2 < 2; ++h2)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const uint32_t bits = __shfl_sync(kAll, seen, 16 * h2 + 8 * q + g) >> (2 * t4);
#pragma unroll
                    for (int j = 0; j < 2 * NJ; ++j)
                        x[h2][q][j] = (bits >> (8 * (j / 2) + (j & 1))) & 1u ? x[h2][q][j] : -INFINITY;
                }
        };
        // The weights are taken with the maxima so far; where that is seen to
        // have been too little (and for the first tile), the maxima are raised
        // and they are taken again, before P is used.
        float ln[2 * NJ];
        bool raise = t == 0;
        for (;;) {
            if (raise) {
                read();
                hide();
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    float2 big = make_float2(-INFINITY, -INFINITY);     // (the factors are positive)
#pragma unroll
                    for (int h2 = 0; h2 < 2; ++h2)
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            big.x = fmaxf(big.x, x[h2][q][2 * j]);
                            big.y = fmaxf(big.y, x[h2][q][2 * j + 1]);
                        }
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) {
                        big.x = fmaxf(big.x, __shfl_xor_sync(kAll, big.x, o));
                        big.y = fmaxf(big.y, __shfl_xor_sync(kAll, big.y, o));
                    }
                    if (g == 0)
                        *reinterpret_cast<float2 *>(red + (warp & 3) * RP + half * NC + 8 * j + 2 * t4) = big;
                }
                __syncthreads();
                float now = 0.f, alpha = 1.f;
                if (tid < RP) {
                    const float was = col_y(tid);       // lift - maximum; -inf: no row
                    const float big = fmaxf(fmaxf(red[tid], red[RP + tid]), fmaxf(red[2 * RP + tid], red[3 * RP + tid]));
                    now = was == -INFINITY || big == -INFINITY ? was : fminf(was, kv4::kLift - big * col_f(tid));
                    if (now == -INFINITY && was != -INFINITY)
                        now = kv4::nan();         // a logit past fp32: for good, through the sums
                    alpha = now == was ? 1.f : tc::ex2(now - was);
                }
                __syncthreads();
                if (tid < RP) {
                    col_y(tid) = now;
                    red[tid] = alpha;
                }
                __syncthreads();
#pragma unroll
                for (int j = 0; j < 2 * NJ; ++j)
                    l[j] *= red[half * NC + 8 * (j / 2) + 2 * t4 + (j & 1)];
                if (t > 0) {
#pragma unroll
                    for (int c = 0; c < NC; c += 16) {
                        float o[16];
                        tc::tmem_ld16(tm_o + c, o);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            o[i] *= red[half * NC + c + i];
                        tc::tmem_st16(tm_o + c, o);
                    }
                }
            }
            // ---- exponents ----
            read();
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const float4 z = my_col[4 * j];
                const f32x2 f = f2_pack(z.x, z.y), y = f2_pack(z.z, z.w);
#pragma unroll
                for (int h2 = 0; h2 < 2; ++h2)
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const float2 u = f2_unpack(f2_fma(f2_pack(x[h2][q][2 * j], x[h2][q][2 * j + 1]), f, y));
                        x[h2][q][2 * j] = u.x;
                        x[h2][q][2 * j + 1] = u.y;
                    }
            }
            if (!whole)
                hide();
            float top = -INFINITY;
#pragma unroll
            for (int h2 = 0; h2 < 2; ++h2)
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int j = 0; j < 2 * NJ; j += 2)
                        top = max3(top, x[h2][q][j], x[h2][q][j + 1]);
            // One thread starts S(t + 1): by now the other warps' K is there.
            if (tid == 0 && t + 1 < ntiles && (t == 0 || !raise)) {
                if (ok)
                    ok = tc::mbar_wait(bar_k, t & 1);
                tc::fence_after_sync();
                issue_s(t + 1);
            }
            // ---- P(t), V(t), once P(t - 1).V(t - 1) is done ----
            if (t > 0 && !raise && ok)
                ok = tc::mbar_wait(bar_o, (t - 1) & 1);
            __syncwarp();
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                uint32_t w[4];
                float l0 = l[2 * j], l1 = l[2 * j + 1];
#pragma unroll
                for (int h2 = 0; h2 < 2; ++h2)
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const float y0 = tc::ex2(x[h2][q][2 * j]), y1 = tc::ex2(x[h2][q][2 * j + 1]);
                        l0 += y0;
                        l1 += y1;
                        w[2 * h2 + q] = kv4::f16x2(y0, y1);
                    }
                ln[2 * j] = l0;
                ln[2 * j + 1] = l1;
                store_rows(p_row + (((half * NJ + j) ^ (row & 7)) << 4), w);
            }
            if (t == 0 || !raise) {
                vr.to_smem(row_v, row & 7);
                load(vr, v4, w1);
                w0 = w1;
                w1 = w2;
                w2 = w3;
            }
            tc::fence_proxy_async();
            tc::fence_before_sync();
            const bool over = __syncthreads_or(top > kv4::kLift + kv4::kUp);
            tc::fence_after_sync();
            if (raise || !over)
                break;
            raise = true;
        }
#pragma unroll
        for (int j = 0; j < 2 * NJ; ++j)
            l[j] = ln[j];
        if (tid == 0) {
            const uint64_t dv = tc::smem_desc(base + C::v, 1024, kRowGroup), dp = tc::smem_desc(base + C::p, kTile * 128, 1024);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                tc::mma_bf16(tmem + 128, dv + ((k * 2 * kRowGroup) >> 4), dp + ((k * 2048) >> 4), idesc_o, t > 0 || k > 0 ? 1u : 0u);
            tc::mma_commit(bar_o);
        }
    }
    // ---- out ----
    if (ok)
        ok = tc::mbar_wait(bar_o, (ntiles - 1) & 1);
    tc::fence_after_sync();
    {
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            float2 sum = make_float2(l[2 * j], l[2 * j + 1]);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                sum.x += __shfl_xor_sync(kAll, sum.x, o);
                sum.y += __shfl_xor_sync(kAll, sum.y, o);
            }
            if (g == 0)
                *reinterpret_cast<float2 *>(red + (warp & 3) * RP + half * NC + 8 * j + 2 * t4) = sum;
        }
    }
    const bool failed = __syncthreads_or(!ok);
    if (failed && tid == 0) {
        report_failure(p.status, 402);
        // The products still under way end before their operands' places and
        // TMEM are given back: a barrier of their own, whose first phase ends
        // with the last of them (S's and O's may be some phases behind).
        tc::mma_commit(bar_end);
        tc::mbar_wait(bar_end, 0);
    }
    if (tid < RP && tid < R) {
        float sum = (red[tid] + red[RP + tid]) + (red[2 * RP + tid] + red[3 * RP + tid]);
        if (failed)
            sum = kv4::nan();
        // sum is 0 where the row attends no token, NaN where a logit was.
        const float lse2 = sum == 0.f ? -INFINITY : log2f(sum) - col_y(tid);
        const int k = tid / G;
        // (+inf, so that the merge's weight for it is NaN and not 0)
        a.lse_part[(size_t)(cq0 + k) * Hq + h * G + (tid - k * G)] = lse2 == lse2 ? lse2 : INFINITY;
        col_f(tid) = sum == 0.f ? 0.f : ka.v_scale / sum;
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < NC; c += 16) {
        float o[16];
        tc::tmem_ld16(tm_o + c, o);
        const int r = half * NC + c;
        int k = r / G, j = r - k * G;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (r + i < R)
                a.o_part[((size_t)(cq0 + k) * Hq + h * G + j) * kD + row] = o[i] * col_f(r + i);
            if (++j == G) {
                j = 0;
                ++k;
            }
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 0)
        tc::tmem_dealloc(tmem, kTmemCols);
    if (ka.last && blockIdx.x == gridDim.x - 1)
        grid_dep_wait();
}

template <int RP>
int launch(const Kv4Args &ka, const DevPartition &p, cudaStream_t st)
{
    const int64_t ctas = (int64_t)ka.n * ka.a.num_kv_heads;
    if (ctas > INT32_MAX)
        return (int)cudaErrorInvalidConfiguration;
    auto *kernel = phase1_kv4_mma_kernel<RP>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<RP>::alloc);
    if (e != cudaSuccess)
        return (int)e;
    return (int)launch_dependent(kernel, dim3((unsigned)ctas), dim3(kThreads), Cfg<RP>::alloc, st, ka, p);
}

}  // namespace

int launch_phase1_kv4_mma(const Kv4Args &ka, const DevPartition &p, int rows, void *stream)
{
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return rows <= 32 ? launch<32>(ka, p, st) : launch<64>(ka, p, st);
}

}  // namespace deft
