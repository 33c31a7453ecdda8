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
// 182 us where this takes 106 (the step on a document of 32768 tokens with 64
// branches of 64 to 8192, 32/8 heads: 36 GFLOP), 44 where 32 (32 branches of
// 256 tokens on a prompt of 4096, 32/32 heads).
//
// What bounds it is the tile's chain: 2.3 us for 128 tokens of a unit, two
// units an SM, of which the tensor products are a fifth; the rest is issue
// slots, the stores and reads of V, P and S, and two barriers.  One CTA an SM
// with twice the registers: 155 us for the 106; 512 threads with a quarter
// row each: 231 (64 registers spill); fewer registers than 128, for room
// beside the other launch: 111 to 126.
//
// A CTA of eight warps takes one unit, and two CTAs share an SM: one unpacks
// and exponentiates while the other waits.  All warps do the same work.  For
// tile t they unpack K(t + 1), read S(t) (a thread a token and half the
// columns) and vote at a barrier whether a column's maximum has to be raised
// (when a logit passes it by more than 2^4); one thread issues S(t + 1) into
// S's other buffer; they write P(t), unpack V(t), and at a second barrier
// P(t).V(t) is issued.  Both products so run while the next operand is
// unpacked.  Sums of the weights stay with the threads until the end.  Every
// wait is bounded.
#include <cfloat>

#include "kv4.cuh"
#include "kv4_internal.h"
#include "merge.cuh"
#include "tcgen05.cuh"

namespace deft {
namespace {

constexpr int kThreads = 256;
constexpr int kD = 128, kTile = 128;
constexpr float kUp = 4.f, kLift = 11.f;
#define kNaN __int_as_float(0x7fffffff)
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
    static constexpr uint32_t col = q + 2 * q_half;             // [RP] factor, [RP] lift - maximum
    static constexpr uint32_t red = col + RP * 8;               // [4 warps][RP]
    static constexpr uint32_t seg = red + 4 * RP * 4;           // [256] position, page, begin; [256] mask (8 B)
    static constexpr uint32_t misc = seg + kMaxSegsPerChunk * 20;   // TMEM base, extremes of the rows' exponents
    static constexpr uint32_t bars = misc + 16;                 // S, O
    static constexpr uint32_t total = bars + 16;
    static constexpr uint32_t alloc = total + 1024;
    static_assert(q % 1024 == 0 && p % 1024 == 0, "128-byte-swizzle atoms");
    static_assert(2 * (alloc + 1024) <= 228 * 1024, "two CTAs an SM");
};

// kind::f16 with fp16 A and B, fp32 D.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int a_mn, int b_mn)
{
    return tc::idesc_bf16(M, N, a_mn, b_mn) & ~((1u << 7) | (1u << 10));
}

__device__ __forceinline__ uint32_t f16x2(float lo, float hi)
{
    const __half2 r = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&r);
}

__device__ __forceinline__ float pow2(int e)   // -126 <= e <= 127
{
    return __int_as_float((127 + e) << 23);
}

// Half a token's row: 64 elements and their scales.
struct HalfRow {
    uint4 w[2];
    uint32_t s;
    __device__ __forceinline__ void zero()
    {
        w[0] = w[1] = make_uint4(0, 0, 0, 0);
        s = 0;
    }
    __device__ __forceinline__ void load(const uint8_t *page, int tok, int half, bool sectors)
    {
        using P = kv4::Page<kD>;
        const uint4 *src = reinterpret_cast<const uint4 *>(page + tok * P::kRow) + 2 * half;
        if (sectors) {
            asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                         : "=r"(w[0].x), "=r"(w[0].y), "=r"(w[0].z), "=r"(w[0].w), "=r"(w[1].x), "=r"(w[1].y), "=r"(w[1].z), "=r"(w[1].w)
                         : "l"(src));
        } else {
            w[0] = __ldg(src);
            w[1] = __ldg(src + 1);
        }
        s = __ldg(reinterpret_cast<const uint32_t *>(page + P::kScales + tok * P::kScaleRow) + half);
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
            tc::tmem_st16(addr + 16 * b, v);
        }
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

// Column i's reduction over the warp's lanes, to lanes i and i + 16.
template <bool kMax>
__device__ __forceinline__ float reduce_columns(float (&v)[16], int lane)
{
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float y = __shfl_xor_sync(kAll, v[i], 16);
        v[i] = kMax ? fmaxf(v[i], y) : v[i] + y;
    }
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) {
        const bool upper = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float send = upper ? v[i] : v[i + o], keep = upper ? v[i + o] : v[i];
            const float y = __shfl_xor_sync(kAll, send, o);
            v[i] = kMax ? fmaxf(keep, y) : keep + y;
        }
    }
    return v[0];
}

template <int RP>
__global__ void __launch_bounds__(kThreads, 2) phase1_kv4_mma_kernel(Kv4Args ka, DevPartition p)
{
    using C = Cfg<RP>;
    using P = kv4::Page<kD>;
    constexpr int NC = RP / 2;      // columns of a thread
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw);
    const AttnArgs &a = ka.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int half = warp >> 2, row = (warp & 3) * 32 + lane;      // tile row, half of its dims and of the columns
    float *col_f = reinterpret_cast<float *>(smem + C::col), *col_y = col_f + RP;
    float *red = reinterpret_cast<float *>(smem + C::red);
    int32_t *seg_pos = reinterpret_cast<int32_t *>(smem + C::seg), *seg_page = seg_pos + kMaxSegsPerChunk,
            *seg_begin = seg_page + kMaxSegsPerChunk;
    uint64_t *seg_mask = reinterpret_cast<uint64_t *>(seg_begin + kMaxSegsPerChunk);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::misc);
    int *ext = reinterpret_cast<int *>(smem + C::misc) + 1;     // least, greatest exponent of a row
    const uint32_t bar_s = base + C::bars, bar_o = bar_s + 8;

    if (warp == 0) {
        tc::tmem_alloc(smem_u32(tmem_slot), kTmemCols);
        tc::tmem_relinquish();
    }
    if (tid == 0) {
        tc::mbar_init(bar_s, 1);
        tc::mbar_init(bar_o, 1);
        tc::fence_mbar_init();
        ext[0] = 1000;
        ext[1] = -1000;
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
    const uint8_t *k4 = static_cast<const uint8_t *>(a.k_pages) + (size_t)h * P::kBytes;
    const uint8_t *v4 = static_cast<const uint8_t *>(a.v_pages) + (size_t)h * P::kBytes;
    const size_t page_step = (size_t)Hkv * P::kBytes;
    struct Where {
        int page, meta;     // page -1: no token; segment x 16 + place in the page
    };
    auto where = [&](int t) {
        Where w{-1, 0};
        const int x = t * kTile + row;
        if (x < T) {
            int seg = 0, hi = nseg;
            while (hi - seg > 1) {
                const int mid = (seg + hi) >> 1;
                if (seg_pos[mid] <= x)
                    seg = mid;
                else
                    hi = mid;
            }
            const int j = x - seg_pos[seg] + seg_begin[seg];
            w.page = a.page_id[seg_page[seg] + j / kPageSize];
            w.meta = seg * kPageSize + j % kPageSize;
        }
        return w;
    };
    // (A half row is one 32-byte sector where the pools are aligned so.)
    const bool sectors = (((uintptr_t)a.k_pages | (uintptr_t)a.v_pages) & 31u) == 0;
    auto load = [&](HalfRow &x, const uint8_t *pool, const Where &w) {
        if (w.page >= 0)
            x.load(pool + (size_t)w.page * page_step, w.meta % kPageSize, half, sectors);
        else
            x.zero();
    };
    HalfRow kr, vr;
    Where w0 = where(0), w1 = where(1), w2{-1, 0};      // of tiles t, t + 1, t + 2
    load(kr, k4, w0);
    load(vr, v4, w0);
    // ---- Q^T: bf16 -> fp16 times a power of two ----
    bool uniform;
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
        int e = big > 0.f ? 14 - ilogbf(big) : 1 << 20;        // (a row of zeros takes any)
        // Rows within 2^8 of one another share the power of two, and with it
        // the factor of their logits: fp16 holds the smallest one's elements
        // down to 2^-31 of its largest.
        if (piece == 0 && e < 1 << 20) {
            atomicMin(ext, e);
            atomicMax(ext + 1, e);
        }
        __syncthreads();
        uniform = ext[1] - ext[0] <= 8;
        if (uniform || e == 1 << 20)
            e = ext[0] == 1000 ? 0 : ext[0];
        // 2^e in two factors: e reaches from -113 to 147.
        const int e1 = e / 2, e2 = e - e1;
        // Infinities become NaN (with the elements beside them), so that a
        // logit of -inf is a masked one.
        const float up1 = inf ? kNaN : pow2(e1), up2 = pow2(e2);
#pragma unroll
        for (int i = 0; i < DT / 8; ++i) {
            uint32_t x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 y = bf16x2_to_float2(qw[4 * i + j]);
                x[j] = f16x2(y.x * up1 * up2, y.y * up1 * up2);
            }
            const int chunk = piece * (DT / 8) + i;         // of the row's sixteen
            *reinterpret_cast<uint4 *>(smem + C::q + (chunk >> 3) * C::q_half + q_row * 128 + (((chunk & 7) ^ (q_row & 7)) << 4)) =
                make_uint4(x[0], x[1], x[2], x[3]);
        }
        // A column of no row has weights of 0: 2^(f * 0 - inf).
        if (piece == 0) {
            // (A factor past fp32, for a row near its end, leaves logits of 0.)
            col_f[q_row] = fminf(a.scale_log2 * pow2(-e1) * ka.k_scale * pow2(-e2), FLT_MAX);
            col_y[q_row] = q_row < R ? INFINITY : -INFINITY;
        }
    }
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const uint32_t tm_s = tmem + ((uint32_t)(warp & 3) << 21) + half * NC, tm_o = tm_s + 128;

    uint8_t *row_v = smem + C::v + (row >> 3) * kRowGroup + half * 1024 + (row & 7) * 128;
    const uint32_t tm_k = tmem + ((uint32_t)(warp & 3) << 21) + 192 + half * 32;
    const f32x2 common = f2_pack(col_f[0], col_f[0]);
    const uint32_t row_bits = R >= RP ? 0xffffffffu >> (32 - NC)
                                      : (uint32_t)((((1ull << R) - 1) >> (half * NC)) & (0xffffffffu >> (32 - NC)));

    f32x2 l[NC / 2];
#pragma unroll
    for (int i = 0; i < NC / 2; ++i)
        l[i] = f2_pack(0.f, 0.f);
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
        // ---- S(t) has been read from K's buffer: K(t + 1) ----
        if (ok)
            ok = tc::mbar_wait(bar_s, t & 1);
        tc::fence_after_sync();
        __syncwarp();
        if (t + 1 < ntiles) {
            kr.to_tmem(tm_k);
            load(kr, k4, w2);
        }
        // ---- exponents of the weights ----
        // Sixteen columns at a time, read from TMEM again where they are
        // needed again: all of them would not fit beside the sums and the rows
        // that are on their way.
        const uint32_t tm_st = tm_s + (t & 1) * 64;
        f32x2 x[8];
        auto read = [&](uint32_t from) {
            float v[16];
            tc::tmem_ld16(from, v);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[i] = f2_pack(v[2 * i], v[2 * i + 1]);
        };
        uint32_t seen = 0;
        if (t * kTile + row < T)
            seen = (uint32_t)(seg_mask[w0.meta / kPageSize] >> (half * NC)) & row_bits;
        const bool whole = __all_sync(kAll, seen == row_bits);
        auto hide = [&](int c) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 v = f2_unpack(x[i]);
                x[i] = f2_pack((seen >> (c + 2 * i)) & 1u ? v.x : -INFINITY, (seen >> (c + 2 * i + 1)) & 1u ? v.y : -INFINITY);
            }
        };
        auto exponents = [&](int c) {       // of columns c .. c + 15
            read(tm_st + c);
            const ulonglong2 *cf = reinterpret_cast<const ulonglong2 *>(col_f + half * NC + c),
                             *cy = reinterpret_cast<const ulonglong2 *>(col_y + half * NC + c);
            if (uniform) {
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const ulonglong2 y = cy[i / 2];
                    x[i] = f2_fma(x[i], common, y.x);
                    x[i + 1] = f2_fma(x[i + 1], common, y.y);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const ulonglong2 f = cf[i / 2], y = cy[i / 2];
                    x[i] = f2_fma(x[i], f.x, y.x);
                    x[i + 1] = f2_fma(x[i + 1], f.y, y.y);
                }
            }
            if (!whole)
                hide(c);
        };
        float top = -INFINITY;
#pragma unroll
        for (int c = 0; c < NC; c += 16) {
            exponents(c);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 v = f2_unpack(x[i]);
                top = fmaxf(top, fmaxf(v.x, v.y));
            }
        }
        tc::fence_proxy_async();
        tc::fence_before_sync();
        const bool raise = __syncthreads_or(top > kLift + kUp);
        if (tid == 0 && t + 1 < ntiles) {
            tc::fence_after_sync();
            issue_s(t + 1);
        }
        // P(t - 1).V(t - 1) is done: P, V and O are free.
        if (t > 0 && ok)
            ok = tc::mbar_wait(bar_o, (t - 1) & 1);
        __syncwarp();
        if (raise) {
            // Maxima over the tile, from S again.
            tc::fence_after_sync();
#pragma unroll
            for (int c = 0; c < NC; c += 16) {
                read(tm_st + c);
                hide(c);
                float v[16];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 y = f2_unpack(x[i]);
                    v[2 * i] = y.x;
                    v[2 * i + 1] = y.y;
                }
                const float big = reduce_columns<true>(v, lane);        // (factors are positive)
                if (lane < 16)
                    red[(warp & 3) * RP + half * NC + c + lane] = big;
            }
            __syncthreads();
            float now = 0.f, alpha = 1.f;
            if (tid < RP) {
                const float was = col_y[tid];       // lift - maximum; -inf: no row
                const float big = fmaxf(fmaxf(red[tid], red[RP + tid]), fmaxf(red[2 * RP + tid], red[3 * RP + tid]));
                now = was == -INFINITY || big == -INFINITY ? was : fminf(was, kLift - big * col_f[tid]);
                if (now == -INFINITY && was != -INFINITY)
                    now = kNaN;         // a logit past fp32: for good, through the sums
                alpha = now == was ? 1.f : tc::ex2(now - was);
            }
            __syncthreads();
            if (tid < RP) {
                col_y[tid] = now;
                red[tid] = alpha;
            }
            __syncthreads();
#pragma unroll
            for (int c = 0; c < NC; c += 16) {
                const f32x2 *al = reinterpret_cast<const f32x2 *>(red + half * NC + c);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    l[c / 2 + i] = f2_mul(l[c / 2 + i], al[i]);
                if (t > 0) {
                    read(tm_o + c);
                    float v[16];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 y = f2_unpack(f2_mul(x[i], al[i]));
                        v[2 * i] = y.x;
                        v[2 * i + 1] = y.y;
                    }
                    tc::tmem_st16(tm_o + c, v);
                }
            }
        }
        // ---- P(t), V(t) ----
        uint8_t *dst = smem + C::p + row * 128;
#pragma unroll
        for (int c = 0; c < NC; c += 16) {
            if (NC > 16 || raise)
                exponents(c);
#pragma unroll
            for (int i = 0; i < 16; i += 8) {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 y = f2_unpack(x[i / 2 + j]);
                    const float y0 = tc::ex2(y.x), y1 = tc::ex2(y.y);
                    l[(c + i) / 2 + j] = f2_add(l[(c + i) / 2 + j], f2_pack(y0, y1));
                    w[j] = f16x2(y0, y1);
                }
                *reinterpret_cast<uint4 *>(dst + ((((half * NC + c + i) >> 3) ^ (row & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        vr.to_smem(row_v, row & 7);
        load(vr, v4, w1);
        w0 = w1;
        w1 = w2;
        w2 = where(t + 3);
        tc::fence_proxy_async();
        tc::fence_before_sync();
        __syncthreads();
        if (tid == 0) {
            tc::fence_after_sync();
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
        for (int c = 0; c < NC; c += 16) {
            float v[16];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 y = f2_unpack(l[c / 2 + i]);
                v[2 * i] = y.x;
                v[2 * i + 1] = y.y;
            }
            const float sum = reduce_columns<false>(v, lane);
            if (lane < 16)
                red[(warp & 3) * RP + half * NC + c + lane] = sum;
        }
    }
    const bool failed = __syncthreads_or(!ok);
    if (failed && tid == 0)
        report_failure(p.status, 402);
    if (tid < RP && tid < R) {
        float sum = (red[tid] + red[RP + tid]) + (red[2 * RP + tid] + red[3 * RP + tid]);
        if (failed)
            sum = kNaN;
        // sum is 0 where the row attends no token, NaN where a logit was.
        const float lse2 = sum == 0.f ? -INFINITY : log2f(sum) - col_y[tid];
        const int k = tid / G;
        // (+inf, so that the merge's weight for it is NaN and not 0)
        a.lse_part[(size_t)(cq0 + k) * Hq + h * G + (tid - k * G)] = lse2 == lse2 ? lse2 : INFINITY;
        col_f[tid] = sum == 0.f ? 0.f : ka.v_scale / sum;
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
                a.o_part[((size_t)(cq0 + k) * Hq + h * G + j) * kD + row] = o[i] * col_f[r + i];
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
