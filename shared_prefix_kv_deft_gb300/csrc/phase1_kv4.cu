// phase1_kv4.cu -- phase-1 partial attention of a tree step over a 4-bit KV
// cache (kv4.cuh), for every row count and both head sizes.
//
// A unit is (work item, KV head), as in the bf16 kernels: for the unit's rows
// r (a query and a member of its head group) over the chunk's tokens j that
// the row attends,
//     s_rj = (q_r . k_j) * scale,  o_r = softmax_j(s_r) . v,  L_r = lse(s_r),
// stored as an fp32 partial (o_r, L_r in base 2) in the row's slot, or in out
// / lse where the query has this one slot.
//
// Tokens are the MMA's M, rows its N (mma.sync m16n8k16, fp16 operands, fp32
// accumulators), a page of 16 tokens at a time:
//     S^T[16 tok x 8 NT] = K . Q^T,     O^T[D x 8 NT] += V^T . P^T.
// Both products' A operand is the cache itself, unpacked from 4 bits straight
// into the registers that the MMA reads: K with a lane's dims contiguous
// (the order of the contracted dims is free as long as Q's agrees), V with
// two tokens' nibbles put side by side first, so that one conversion makes a
// pair along the tokens.  c * s is exact in fp16, and so is Q once each row
// is multiplied by a power of two that puts its largest element in [2^14,
// 2^15) (what falls below fp16 there is 2^-39 of the row's largest).  S^T's
// layout becomes P^T's by a transposition of 8x8 blocks between lanes.
//
// P is held as 2^11 * 2^(s - m), m a maximum that is raised only when a logit
// passes it by more than 2^4: at most 2^15, and weights down to 2^-35 of the
// largest count.
//
// A CTA of four warps takes a unit.  Rows beyond 16 go to further warps;
// the warps of 16 rows deal the unit's pages among themselves, each with its
// own ring of bulk copies, and join their states in shared memory at the end.
// Every wait is bounded.
#include "kv4.cuh"
#include "merge.cuh"
#include "tcgen05.cuh"

namespace deft {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kStages = 4;
constexpr int kRowsMax = 64;
constexpr float kUp = 4.f, kLift = 11.f;
constexpr unsigned kAll = 0xffffffffu;

struct Kv4Args {
    AttnArgs a;
    float k_scale, v_scale;
    int32_t n_mma, n_fma;      // items of the partition's two lists
    int32_t mma_narrow;        // tensor-core items below this have their row masks split at 16
};

template <int D>
struct Cfg {
    using P = kv4::Page<D>;
    static constexpr uint32_t kStage = 2 * P::kBytes;                     // K, then V, of one page
    static constexpr uint32_t kQRow = 2 * D + 16;                        // bytes of a row of Q, padded
    static constexpr uint32_t ring = 0;                                   // [warp][stage]; at the end [warp][16][D] fp32
    static constexpr uint32_t ring_bytes = kWarps * kStages * kStage > kWarps * 16 * D * 4 ? kWarps * kStages * kStage
                                                                                            : kWarps * 16 * D * 4;
    static constexpr uint32_t q = ring + ring_bytes;                      // [64] rows
    static constexpr uint32_t qf = q + kRowsMax * kQRow;                  // [64] what a row's S is multiplied by
    static constexpr uint32_t ml = qf + kRowsMax * 4;                     // [warp][16] m, l
    static constexpr uint32_t seg = ml + kWarps * 16 * 8;                 // [256] mask (8 B), page, begin, len; [257] first slice
    static constexpr uint32_t bars = seg + kMaxSegsPerChunk * 24 + 8;
    static constexpr uint32_t total = bars + kWarps * kStages * 8 + 16;
    static_assert(kStage % 16 == 0 && q % 16 == 0 && seg % 8 == 0 && bars % 8 == 0, "alignment");
};

struct Slice {
    int page, seg, lo, hi;   // tokens lo .. hi - 1 of the page
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// An 8x8 block of fp16, two of a row's elements a lane, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

__device__ __forceinline__ uint32_t f16x2(float lo, float hi)
{
    const __half2 r = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&r);
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads) phase1_kv4_kernel(Kv4Args ka, DevPartition p)
{
    using C = Cfg<D>;
    using P = kv4::Page<D>;
    constexpr int KW = D / 32;      // words of a lane's K elements: dims (D / 4) t ..
    constexpr int VW = D / 64;      // words of a lane's V elements: dims (D / 8) g ..
    extern __shared__ __align__(128) uint8_t smem[];
    const AttnArgs &a = ka.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const uint32_t base = smem_u32(smem);
    uint64_t *seg_mask = reinterpret_cast<uint64_t *>(smem + C::seg);
    int32_t *seg_page = reinterpret_cast<int32_t *>(smem + C::seg + kMaxSegsPerChunk * 8);   // first page's index in page_id
    int32_t *seg_begin = seg_page + kMaxSegsPerChunk, *seg_len = seg_begin + kMaxSegsPerChunk;
    int32_t *seg_first = seg_len + kMaxSegsPerChunk;                                         // [257] slices before the segment
    float *qf = reinterpret_cast<float *>(smem + C::qf);
    float2 *ml = reinterpret_cast<float2 *>(smem + C::ml);
    const uint32_t bars = base + C::bars + warp * kStages * 8;

    if (lane == 0) {
        for (int s = 0; s < kStages; ++s)
            tc::mbar_init(bars + s * 8, 1);
        tc::fence_mbar_init();
    }
    grid_dep_wait();
    grid_dep_launch();

    // ---- the unit ----
    const int Hkv = a.num_kv_heads, Hq = a.num_q_heads, G = a.gqa_group;
    const int unit = blockIdx.x, it = unit / Hkv, h = unit - it * Hkv;
    const bool wide = it < ka.n_mma;
    const int item = wide ? it : it - ka.n_mma;
    const int32_t *triple = (wide ? p.mma_items : p.fma_items) + 3 * (size_t)item;
    const int c = triple[0], qb = triple[1], R = (triple[2] - qb) * G;
    const int cq0 = p.chunk_q_off[c] + qb;
    const int sb = p.chunk_seg_off[c], nseg = p.chunk_seg_off[c + 1] - sb;
    const uint32_t direct = !wide && a.direct ? p.fma_direct[item] : 0u;
    const int rm0 = wide ? p.mma_rmask_off[item] : p.fma_rmask_off[item];
    for (int s = tid; s < nseg; s += kThreads) {
        const int len = p.seg_tok_len[sb + s], tb = p.seg_tok_begin[sb + s];
        seg_page[s] = a.node_page_off[p.seg_node[sb + s]] + tb / kPageSize;
        seg_begin[s] = tb % kPageSize;
        seg_len[s] = len;
        seg_first[s + 1] = (tb % kPageSize + len + kPageSize - 1) / kPageSize;
        if (wide) {
            const uint4 w = reinterpret_cast<const uint4 *>(p.mma_rmask)[rm0 + s];
            seg_mask[s] = (uint64_t)w.x | (uint64_t)w.z << (item < ka.mma_narrow ? 16 : 32);
        } else {
            seg_mask[s] = p.fma_rmask[rm0 + s];
        }
    }
    if (tid == 0)
        seg_first[0] = 0;
    // ---- Q, a row a warp: bf16 -> fp16 times a power of two ----
    const int groups = R <= 8 * NT ? 1 : R <= 16 * NT ? 2 : 4;     // warps' worth of rows
    for (int r = warp; r < groups * 8 * NT; r += kWarps) {
        float x[D / 32];
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
            x[i] = 0.f;
        if (r < R) {
            const int head = h * G + r % G;
            const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(a.q) +
                                       ((size_t)p.chunk_q[cq0 + r / G] * Hq + head) * D + lane * (D / 32);
#pragma unroll
            for (int i = 0; i < D / 32; i += 2) {
                const float2 v = bf16x2_to_float2(*reinterpret_cast<const uint32_t *>(src + i));
                x[i] = v.x;
                x[i + 1] = v.y;
            }
        }
        float big = 0.f;   // the largest finite magnitude
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
            if (fabsf(x[i]) < INFINITY)
                big = fmaxf(big, fabsf(x[i]));
        big = warp_max(big);
        // 2^e in two factors: e reaches from -113 to 147.
        const int e = big > 0.f ? 14 - ilogbf(big) : 0, e1 = e / 2, e2 = e - e1;
        const float up1 = __int_as_float((127 + e1) << 23), up2 = __int_as_float((127 + e2) << 23);
#pragma unroll
        for (int i = 0; i < D / 32; i += 2)
            *reinterpret_cast<uint32_t *>(smem + C::q + r * C::kQRow + (lane * (D / 32) + i) * 2) =
                f16x2(x[i] * up1 * up2, x[i + 1] * up1 * up2);
        if (lane == 0)
            qf[r] = a.scale_log2 * __int_as_float((127 - e1) << 23) * ka.k_scale * __int_as_float((127 - e2) << 23);
    }
    __syncthreads();
    if (warp == 0) {
        // Slices before each segment: an inclusive scan of the counts.
        int before = 0;
        for (int s0 = 0; s0 < nseg; s0 += 32) {
            int n = s0 + lane < nseg ? seg_first[s0 + lane + 1] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(kAll, n, o);
                if (lane >= o)
                    n += y;
            }
            if (s0 + lane < nseg)
                seg_first[s0 + lane + 1] = before + n;
            before += __shfl_sync(kAll, n, 31);
        }
    }
    __syncthreads();

    // ---- the warp's rows and slices ----
    const int rg = warp % groups, ts = warp / groups, TS = kWarps / groups;
    const int row0 = rg * 8 * NT;
    const int total = seg_first[nseg];
    const int mine = total > ts && row0 < R ? (total - ts + TS - 1) / TS : 0;
    uint32_t qa[NT][KW * 4];        // Q^T fragments: two registers a step of 16 dims
    float f[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const uint8_t *src = smem + C::q + (row0 + 8 * n + g) * C::kQRow + t * (D / 2);
#pragma unroll
        for (int i = 0; i < KW; ++i) {
            const uint4 w = *reinterpret_cast<const uint4 *>(src + 16 * i);
            qa[n][4 * i] = w.x, qa[n][4 * i + 1] = w.y, qa[n][4 * i + 2] = w.z, qa[n][4 * i + 3] = w.w;
        }
        f[n][0] = qf[row0 + 8 * n + 2 * t];
        f[n][1] = qf[row0 + 8 * n + 2 * t + 1];
    }
    // Slice i of the warp, by lane i % 32 for the batch it lies in.
    Slice batch{0, 0, 0, 0};
    auto fill_batch = [&](int b) {
        const int i = b * 32 + lane;
        if (i < mine) {
            const int x = ts + i * TS;
            int lo = 0, hi = nseg;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (seg_first[mid] <= x)
                    lo = mid;
                else
                    hi = mid;
            }
            const int j = x - seg_first[lo];
            batch.page = a.page_id[seg_page[lo] + j];
            batch.seg = lo;
            batch.lo = max(0, seg_begin[lo] - j * kPageSize);
            batch.hi = min(kPageSize, seg_begin[lo] + seg_len[lo] - j * kPageSize);
        }
    };
    const uint8_t *k4 = static_cast<const uint8_t *>(a.k_pages), *v4 = static_cast<const uint8_t *>(a.v_pages);
    const uint64_t pol = tc::l2_kv_policy(false);
    const uint32_t ring = base + C::ring + warp * kStages * C::kStage;
    auto copy = [&](int i, int page) {   // lane 0
        const uint32_t dst = ring + (i % kStages) * C::kStage, bar = bars + (i % kStages) * 8;
        const size_t at = ((size_t)page * Hkv + h) * P::kBytes;
        tc::mbar_arrive_expect_tx(bar, C::kStage);
        tc::bulk_load(dst, k4 + at, P::kBytes, bar, pol);
        tc::bulk_load(dst + P::kBytes, v4 + at, P::kBytes, bar, pol);
    };
    fill_batch(0);
    // The next batch's slices are taken when its first copy is due.
    Slice next = batch;
    int issued = 0, next_batch = 0;
    auto issue = [&](int i) {
        if (i / 32 != next_batch) {
            const Slice keep = batch;
            next_batch = i / 32;
            fill_batch(next_batch);
            next = batch;
            batch = keep;
        }
        const int page = __shfl_sync(kAll, next.page, i & 31);
        if (lane == 0)
            copy(i, page);
    };
    for (; issued < mine && issued < kStages; ++issued)
        issue(issued);

    float o[D / 16][NT][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
            o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.f;
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.f;
    }
    const uint64_t row_bits = R >= 64 ? ~0ull : (1ull << R) - 1;
    const uint64_t my_rows = (row_bits >> row0) & ((1ull << (8 * NT)) - 1);
    bool ok = true;
    for (int i = 0; i < mine; ++i) {
        if (i > 0 && (i & 31) == 0)
            batch = next;      // (issue() is at most kStages ahead: it has filled this batch)
        const int seg = __shfl_sync(kAll, batch.seg, i & 31);
        const int lo = __shfl_sync(kAll, batch.lo, i & 31), hi = __shfl_sync(kAll, batch.hi, i & 31);
        if (!__all_sync(kAll, tc::mbar_wait(bars + (i % kStages) * 8, (i / kStages) & 1))) {
            ok = false;
            break;
        }
        const uint8_t *ks = smem + C::ring + (warp * kStages + i % kStages) * C::kStage, *vs = ks + P::kBytes;
        // ---- S^T ----
        float s[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
            s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
        {
            uint32_t w0[KW], w1[KW], sc0[D / 64], sc1[D / 64];
            if constexpr (D == 128) {
                const uint4 x = *reinterpret_cast<const uint4 *>(ks + g * P::kRow + t * 16);
                const uint4 y = *reinterpret_cast<const uint4 *>(ks + (g + 8) * P::kRow + t * 16);
                w0[0] = x.x, w0[1] = x.y, w0[2] = x.z, w0[3] = x.w;
                w1[0] = y.x, w1[1] = y.y, w1[2] = y.z, w1[3] = y.w;
                const uint32_t u = kv4::scales2(*reinterpret_cast<const uint16_t *>(ks + P::kScales + g * P::kScaleRow + t * 2));
                const uint32_t v = kv4::scales2(*reinterpret_cast<const uint16_t *>(ks + P::kScales + (g + 8) * P::kScaleRow + t * 2));
                sc0[0] = __byte_perm(u, 0, 0x1010), sc0[1] = __byte_perm(u, 0, 0x3232);
                sc1[0] = __byte_perm(v, 0, 0x1010), sc1[1] = __byte_perm(v, 0, 0x3232);
            } else {
                const uint2 x = *reinterpret_cast<const uint2 *>(ks + g * P::kRow + t * 8);
                const uint2 y = *reinterpret_cast<const uint2 *>(ks + (g + 8) * P::kRow + t * 8);
                w0[0] = x.x, w0[1] = x.y;
                w1[0] = y.x, w1[1] = y.y;
                const uint32_t u = ks[P::kScales + g * P::kScaleRow + t], v = ks[P::kScales + (g + 8) * P::kScaleRow + t];
                sc0[0] = kv4::scales2(u | u << 8);
                sc1[0] = kv4::scales2(v | v << 8);
            }
#pragma unroll
            for (int w = 0; w < KW; ++w) {
                uint32_t x[4], y[4];
                kv4::unpack8(w0[w], x);
                kv4::unpack8(w1[w], y);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    x[k] = kv4::hmul2(x[k], sc0[w / 2]);
                    y[k] = kv4::hmul2(y[k], sc1[w / 2]);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    mma16816(s[n], x[0], y[0], x[1], y[1], qa[n][4 * w], qa[n][4 * w + 1]);
                    mma16816(s[n], x[2], y[2], x[3], y[3], qa[n][4 * w + 2], qa[n][4 * w + 3]);
                }
            }
        }
        // ---- softmax ----
        const uint64_t rows = (seg_mask[seg] >> row0) & my_rows;
        const bool whole = hi - lo == kPageSize && rows == my_rows;
        bool grow = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[n][j] *= f[n][j & 1];
                if (!whole) {
                    const int tok = g + (j >> 1) * 8, row = 8 * n + 2 * t + (j & 1);
                    if (tok < lo || tok >= hi || !((rows >> row) & 1))
                        s[n][j] = -INFINITY;
                }
                grow |= s[n][j] > m[n][j & 1] + kUp;
            }
        }
        if (__any_sync(kAll, grow)) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float x = fmaxf(s[n][j], s[n][j + 2]);
                    x = fmaxf(x, __shfl_xor_sync(kAll, x, 4));
                    x = fmaxf(x, __shfl_xor_sync(kAll, x, 8));
                    x = fmaxf(x, __shfl_xor_sync(kAll, x, 16));
                    x = fmaxf(m[n][j], x);
                    const float alpha = x == -INFINITY ? 1.f : tc::ex2(m[n][j] - x);
                    m[n][j] = x;
                    l[n][j] *= alpha;
#pragma unroll
                    for (int d = 0; d < D / 16; ++d) {
                        o[d][n][j] *= alpha;
                        o[d][n][j + 2] *= alpha;
                    }
                }
            }
        }
        uint32_t pb[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float m0 = m[n][0] == -INFINITY ? 0.f : m[n][0] - kLift, m1 = m[n][1] == -INFINITY ? 0.f : m[n][1] - kLift;
            const float p0 = tc::ex2(s[n][0] - m0), p1 = tc::ex2(s[n][1] - m1);
            const float p2 = tc::ex2(s[n][2] - m0), p3 = tc::ex2(s[n][3] - m1);
            l[n][0] += p0 + p2;
            l[n][1] += p1 + p3;
            pb[n][0] = transpose8(f16x2(p0, p1));
            pb[n][1] = transpose8(f16x2(p2, p3));
        }
        // ---- O^T ----
        {
            uint32_t sv[2];     // scales of tokens (2t, 2t + 1) and (2t + 8, 2t + 9)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int tok = 2 * t + 8 * q;
                const uint8_t *src = vs + P::kScales + tok * P::kScaleRow + (D == 128 ? g : g >> 1);
                uint32_t x = src[0], y = src[P::kScaleRow];
                if (!whole) {   // (what a page holds beside the segment's tokens may be anything)
                    x = tok >= lo && tok < hi ? x : 0u;
                    y = tok + 1 >= lo && tok + 1 < hi ? y : 0u;
                }
                sv[q] = kv4::scales2(x | y << 8);
            }
#pragma unroll
            for (int w = 0; w < VW; ++w) {
                uint32_t e[2][4], od[2][4];   // even and odd dims of the word, by token pair
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const uint8_t *src = vs + (2 * t + 8 * q) * P::kRow + g * (D / 16) + 4 * w;
                    const uint32_t x = *reinterpret_cast<const uint32_t *>(src);
                    const uint32_t y = *reinterpret_cast<const uint32_t *>(src + P::kRow);
                    kv4::unpack8((x & 0x0f0f0f0fu) | (y << 4 & 0xf0f0f0f0u), e[q]);
                    kv4::unpack8((x >> 4 & 0x0f0f0f0fu) | (y & 0xf0f0f0f0u), od[q]);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        e[q][k] = kv4::hmul2(e[q][k], sv[q]);
                        od[q][k] = kv4::hmul2(od[q][k], sv[q]);
                    }
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mma16816(o[4 * w + k][n], e[0][k], od[0][k], e[1][k], od[1][k], pb[n][0], pb[n][1]);
            }
        }
        // The stage is free once every lane has read it.
        __syncwarp();
        if (issued < mine) {
            issue(issued);
            ++issued;
        }
    }
    if (!ok) {
        // A copy that never landed: give the others their time, and say so.
        for (int i = 0; i < kStages; ++i)
            tc::mbar_wait(bars + i * 8, 0);
        if (lane == 0)
            report_failure(p.status, 401);
#pragma unroll
        for (int n = 0; n < NT; ++n)
            l[n][0] = l[n][1] = __int_as_float(0x7fffffff);
    }

    // ---- the warps' states, joined ----
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float x = l[n][j];
            x += __shfl_xor_sync(kAll, x, 4);
            x += __shfl_xor_sync(kAll, x, 8);
            x += __shfl_xor_sync(kAll, x, 16);
            if (g == 0)
                ml[warp * 16 + 8 * n + 2 * t + j] = make_float2(m[n][j], x);
        }
    __syncthreads();   // every warp's copies have been read
    float *os = reinterpret_cast<float *>(smem + C::ring);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float *dst = os + (warp * 16 + 8 * n + 2 * t + j) * D + g * (D / 8);
#pragma unroll
            for (int i = 0; i < D / 16; i += 2)
                *reinterpret_cast<float4 *>(dst + 2 * i) =
                    make_float4(o[i][n][j], o[i][n][j + 2], o[i + 1][n][j], o[i + 1][n][j + 2]);
        }
    __syncthreads();
    for (int r = warp; r < R; r += kWarps) {
        const int grp = r / (8 * NT), in = r - grp * 8 * NT;
        float M = -INFINITY;
        for (int k = 0; k < TS; ++k)
            M = fmaxf(M, ml[(grp + k * groups) * 16 + in].x);
        float sum = 0.f, acc[D / 32];
#pragma unroll
        for (int e = 0; e < D / 32; ++e)
            acc[e] = 0.f;
        for (int k = 0; k < TS; ++k) {
            const int w = grp + k * groups;
            const float2 s = ml[w * 16 + in];
            const float wt = M == -INFINITY ? 1.f : tc::ex2(s.x - M);
            sum = fmaf(wt, s.y, sum);
            const float *src = os + (w * 16 + in) * D + lane * (D / 32);
#pragma unroll
            for (int e = 0; e < D / 32; ++e)
                acc[e] = fmaf(wt, src[e], acc[e]);
        }
        // sum is 0 where the row attends no token, NaN where a logit was.
        const float inv = sum == 0.f ? 0.f : ka.v_scale / sum;
        const float lse2 = sum == 0.f ? -INFINITY : M + log2f(sum) - kLift;
        const int k = r / G, head = h * G + r % G;
        if (r < 32 && ((direct >> r) & 1u)) {
            const size_t row = (size_t)p.chunk_q[cq0 + k] * Hq + head;
#pragma unroll
            for (int e = 0; e < D / 32; ++e)
                store_out(a, row, lane * (D / 32) + e, D, acc[e] * inv);
            if (lane == 0)
                a.lse_out[row] = direct_lse(lse2);
        } else {
            const size_t row = (size_t)(cq0 + k) * Hq + head;
#pragma unroll
            for (int e = 0; e < D / 32; ++e)
                a.o_part[row * D + lane * (D / 32) + e] = acc[e] * inv;
            // (+inf, so that the merge's weight for it is NaN and not 0)
            if (lane == 0)
                a.lse_part[row] = lse2 == lse2 ? lse2 : INFINITY;
        }
    }
}

template <int D>
int launch(const Kv4Args &ka, const DevPartition &p, cudaStream_t st)
{
    constexpr int NT = 2;
    const int64_t units = (int64_t)(ka.n_mma + ka.n_fma) * ka.a.num_kv_heads;
    if (units == 0)
        return 0;
    if (units > INT32_MAX)
        return (int)cudaErrorInvalidConfiguration;
    auto *kernel = phase1_kv4_kernel<D, NT>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::total);
    if (e != cudaSuccess)
        return (int)e;
    return (int)launch_dependent(kernel, dim3((unsigned)units), dim3(kThreads), Cfg<D>::total, st, ka, p);
}

}  // namespace

int dispatch_step4(const AttnArgs &a, const DevPartition &dp, const Partition &hp, float k_scale, float v_scale, void *stream,
                   const LaunchTracer &trace)
{
    const Kv4Args ka{a, k_scale, v_scale, dp.num_mma_items, dp.num_fma_items, hp.mma_bucket_off[1]};
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (ka.n_mma + ka.n_fma > 0) {
        const int r = trace({DEFT_K_PHASE1_KV4, 0, 0, 0, ka.n_mma + ka.n_fma, 0.f}, stream,
                            [&] { return a.head_dim == 128 ? launch<128>(ka, dp, st) : launch<64>(ka, dp, st); });
        if (r)
            return r;
    }
    const int32_t nq = a.direct ? dp.num_merge_q : dp.num_queries;
    if (nq == 0)
        return 0;
    const int32_t *qlist = nq < dp.num_queries ? dp.merge_q : nullptr;
    return trace({DEFT_K_PHASE2, 0, 0, 0, nq, 0.f}, stream, [&] { return launch_phase2(a, dp, qlist, nq, stream); });
}

}  // namespace deft
