// phase1_kv4.cu -- phase-1 partial attention of a tree step over a 4-bit KV
// cache (kv4.cuh) on mma.sync, for units of up to 15 rows, and at head_dim 64
// for all (phase1_kv4_mma.cu: 16 to 64 rows at head_dim 128); the merge of
// the partials; the step's launches.
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
// 2^15) (elements under 2^-31 of the row's largest are off by at most 2^-39 of
// it).  S^T's layout becomes P^T's by a transposition of 8x8 blocks between lanes.
//
// P is held as 2^11 * 2^(s - m), m a maximum that is raised only when a logit
// passes it by more than 2^4: at most 2^15, and weights down to 2^-35 of the
// largest count.
//
// A warp takes a unit, fed by its own ring of bulk copies (four pages), and a
// CTA of four warps the KV heads of an item, which share its tables; where
// that leaves SMs idle (heads_per_cta), two or four warps deal a unit's pages
// among themselves and join their states in shared memory at the end.  Up to
// 8 rows a step takes two pages, so that two chains of products and
// exponentials overlap.  Every wait is bounded.
//
// What bounds it is the units' latency: 64 requests of 64 to 8192 tokens,
// 32/8 heads of 128, a step of 36.1 us for 115 MB (17 us at the measured copy
// rate).  Of a unit's 10 us, 4 are the chain of look-ups from its item to its
// first page (five loads, each waiting for the one before), and in the other 6
// each scheduler issues an instruction in two cycles from its four warps, some
// 300 a page and warp: 64 conversions and 64 products of the unpacking, the
// rest for V's nibbles, the softmax, the look-ups and the copies.  Leaving out
// any one of these (in a copy for measurement) gains 5% at most.  Measured and
// left: bytes put apart by mul.hi, pairs made by integer arithmetic (44.7, 48.4
// us where 37.9), five CTAs an SM with fewer registers (39.1 where 37.9); a conversion
// takes any byte of its operand at no cost.
#include <cfloat>

#include "kv4.cuh"
#include "kv4_internal.h"
#include "merge.cuh"
#include "tcgen05.cuh"

namespace deft {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr unsigned kAll = 0xffffffffu;

template <int D, int NT>
struct Cfg {
    using P = kv4::Page<D>;
    static constexpr bool kQSmem = NT > 2;                                // Q^T fragments in shared memory
    static constexpr int kPages = NT == 1 ? 2 : 1;                        // pages of a step
    static constexpr int kStages = 4 / kPages;
    static constexpr uint32_t kPage = 2 * P::kBytes;                      // K, then V
    static constexpr uint32_t kStage = kPages * kPage;
    static constexpr uint32_t kState = NT * (1 + D / 16) * 512;           // a warp's state when warps join
    static constexpr uint32_t ring_raw = kWarps * kStages * kStage;       // [warp][stage]; at the end two states
    static constexpr uint32_t ring_bytes = ring_raw > 2 * kState ? ring_raw : (2 * kState + 127) / 128 * 128;
    static constexpr uint32_t q = ring_bytes;                             // [warp][NT * D / 32][lane] 16 bytes
    static constexpr uint32_t seg = q + (kQSmem ? kWarps * NT * (D / 32) * 512 : 0);
    static constexpr uint32_t bars = seg + kMaxSegsPerChunk * 24 + 8;     // [256] mask (8 B), page, begin, len; [257] first slice
    static constexpr uint32_t total = bars + kWarps * kStages * 8;
    static constexpr int kCtas = NT == 1 ? 4 : NT == 2 ? 3 : 2;           // that an SM is to hold
    static_assert(kStage % 16 == 0 && q % 16 == 0 && seg % 8 == 0 && bars % 8 == 0, "alignment");
    static_assert((total + 1024) * kCtas <= 228 * 1024, "shared memory of an SM");
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
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

// The exponent of the power of two that puts a row's largest finite
// magnitude in [2^14, 2^15): N pairs of bf16 in each of the row's LANES
// neighbouring lanes (-113 to 147; 0 for a row of zeros).  Infinities become
// NaN, so that a logit of -inf is a masked one.
template <int N, int LANES>
__device__ __forceinline__ int row_exponent(uint32_t (&w)[N])
{
    uint32_t big = 0;               // magnitudes order as integers
#pragma unroll
    for (int i = 0; i < N; ++i)
        big = __vmaxu2(big, w[i] & 0x7fff7fffu);
    big = max(big & 0xffffu, big >> 16);
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1)
        big = max(big, __shfl_xor_sync(kAll, big, o));
    if (__any_sync(kAll, big >= 0x7f80u)) {     // infinities, NaN: without them
        big = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t lo = w[i] & 0x7fffu, hi = w[i] >> 16 & 0x7fffu;
            big = max(big, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
            w[i] |= (lo == 0x7f80u ? 0x40u : 0u) | (hi == 0x7f80u ? 0x400000u : 0u);
        }
#pragma unroll
        for (int o = 1; o < LANES; o <<= 1)
            big = max(big, __shfl_xor_sync(kAll, big, o));
    }
    return big == 0 ? 0 : big >= 0x80u ? 14 + 127 - (int)(big >> 7) : 14 + 133 - (31 - __clz((int)big));
}

// A slice: the tokens of one page that belong to one segment.  `desc` holds
// tokens lo .. hi - 1 of the page and the segment; bit 31: all 16 tokens, for
// all of the warp's rows.
__device__ __forceinline__ uint32_t slice_desc(int seg, int lo, int hi, bool whole)
{
    return (whole ? 1u << 31 : 0u) | (uint32_t)seg << 16 | (uint32_t)lo << 8 | (uint32_t)hi;
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, Cfg<D, NT>::kCtas) phase1_kv4_kernel(Kv4Args ka, DevPartition p)
{
    using C = Cfg<D, NT>;
    using P = kv4::Page<D>;
    constexpr int KW = D / 32;      // words of a lane's K elements: dims (D / 4) t ..
    constexpr int VW = D / 64;      // words of a lane's V elements: dims (D / 8) g ..
    constexpr int NR = 8 * NT;      // rows of a warp
    constexpr int PP = C::kPages, kStages = C::kStages, kBatch = 32 / PP;
    extern __shared__ __align__(128) uint8_t smem[];
    const AttnArgs &a = ka.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const uint32_t base = smem_u32(smem);
    uint64_t *seg_mask = reinterpret_cast<uint64_t *>(smem + C::seg);
    int32_t *seg_page = reinterpret_cast<int32_t *>(smem + C::seg + kMaxSegsPerChunk * 8);   // first page's index in page_id
    int32_t *seg_begin = seg_page + kMaxSegsPerChunk, *seg_len = seg_begin + kMaxSegsPerChunk;
    int32_t *seg_first = seg_len + kMaxSegsPerChunk;                                         // [257] slices before the segment
    const uint32_t bars = base + C::bars + warp * kStages * 8;

    if (lane == 0) {
        for (int s = 0; s < kStages; ++s)
            tc::mbar_init(bars + s * 8, 1);
        tc::fence_mbar_init();
    }
    if (a.wait_prior)
        grid_dep_wait();
    grid_dep_launch();

    // ---- the item ----
    const int Hkv = a.num_kv_heads, Hq = a.num_q_heads, G = a.gqa_group;
    const int it = blockIdx.x / ka.head_groups, hg = blockIdx.x - it * ka.head_groups;
    const int item = ka.first + it;
    const int32_t *triple = (ka.wide ? p.mma_items : p.fma_items) + 3 * (size_t)item;
    const int c = triple[0], qb = triple[1], R = (triple[2] - qb) * G;
    const int rm0 = (ka.wide ? p.mma_rmask_off : p.fma_rmask_off)[item];
    const uint32_t direct = !ka.wide && a.direct ? p.fma_direct[item] : 0u;
    const int cq0 = p.chunk_q_off[c] + qb;
    const int sb = p.chunk_seg_off[c], nseg = p.chunk_seg_off[c + 1] - sb;
    auto row_mask = [&](int s) -> uint64_t {
        if (!ka.wide)
            return p.fma_rmask[rm0 + s];
        const uint4 w = reinterpret_cast<const uint4 *>(p.mma_rmask)[rm0 + s];
        return (uint64_t)w.x | (uint64_t)w.z << (item < ka.mma_narrow ? 16 : 32);
    };
    // The warp's part: rows [row0, row0 + NR) of KV head h; of the slices, PP
    // a step, steps ts, ts + TS, ...
    const int groups = R <= NR ? 1 : 2;                 // (a CTA's share of heads leaves room for both)
    const int TS = kWarps / (ka.heads * groups);
    const int ts = warp % TS, rg = warp / TS % groups, h = hg * ka.heads + warp / (TS * groups);
    const int row0 = rg * NR;

    // The rows of Q, on their way while the slices are looked up: lane (g, t)
    // takes dims (D / 4) t .. of row g of eight.
    uint32_t qw[NT][KW * 4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int r = row0 + 8 * n + g;
#pragma unroll
        for (int i = 0; i < KW * 4; ++i)
            qw[n][i] = 0u;
        if (r < R) {
            const int k = r / G;
            const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.q) +
                                                               ((size_t)p.chunk_q[cq0 + k] * Hq + h * G + (r - k * G)) * D) +
                               t * KW;
#pragma unroll
            for (int i = 0; i < KW; ++i) {
                const uint4 v = src[i];
                qw[n][4 * i] = v.x, qw[n][4 * i + 1] = v.y, qw[n][4 * i + 2] = v.z, qw[n][4 * i + 3] = v.w;
            }
        }
    }

    // One segment (a piece of a longer node) is the common case; the table of
    // several is made by the CTA.
    uint64_t mask0 = 0;
    int page0 = 0, begin0 = 0, len0 = 0, total;
    if (nseg == 1) {
        len0 = p.seg_tok_len[sb];
        const int tb = p.seg_tok_begin[sb];
        page0 = a.node_page_off[p.seg_node[sb]] + tb / kPageSize;
        begin0 = tb % kPageSize;
        mask0 = row_mask(0);
        total = (begin0 + len0 + kPageSize - 1) / kPageSize;
    } else {
        for (int s = tid; s < nseg; s += kThreads) {
            const int len = p.seg_tok_len[sb + s], tb = p.seg_tok_begin[sb + s];
            seg_page[s] = a.node_page_off[p.seg_node[sb + s]] + tb / kPageSize;
            seg_begin[s] = tb % kPageSize;
            seg_len[s] = len;
            seg_first[s + 1] = (tb % kPageSize + len + kPageSize - 1) / kPageSize;
            seg_mask[s] = row_mask(s);
        }
        if (tid == 0)
            seg_first[0] = 0;
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
        total = seg_first[nseg];
    }
    const int steps = (total + PP - 1) / PP, mine = steps > ts ? (steps - ts + TS - 1) / TS : 0;
    const uint64_t row_bits = R >= 64 ? ~0ull : (1ull << R) - 1;
    const uint32_t my_rows = (uint32_t)(row_bits >> row0) & (uint32_t)((1ull << NR) - 1);

    // ---- slices: 32 at a time, each held (and its copy issued) by a lane ----
    const uint64_t pol = tc::l2_kv_policy(false);
    const uint32_t ring = base + warp * kStages * C::kStage;
    // The lane's slice of the batch of steps from `first` on.
    auto get_slice = [&](int first, const uint8_t *&k, const uint8_t *&v, uint32_t &desc) {
        const int i = first + lane / PP, x = (ts + i * TS) * PP + lane % PP;
        desc = 0;               // no token
        if (i >= mine || x >= total)
            return;
        int seg = 0, j = x, pg = page0, begin = begin0, len = len0;
        uint64_t mask = mask0;
        if (nseg > 1) {
            int hi = nseg;
            while (hi - seg > 1) {
                const int mid = (seg + hi) >> 1;
                if (seg_first[mid] <= x)
                    seg = mid;
                else
                    hi = mid;
            }
            j = x - seg_first[seg];
            pg = seg_page[seg], begin = seg_begin[seg], len = seg_len[seg], mask = seg_mask[seg];
        }
        const size_t at = ((size_t)a.page_id[pg + j] * Hkv + h) * P::kBytes;
        k = static_cast<const uint8_t *>(a.k_pages) + at;
        v = static_cast<const uint8_t *>(a.v_pages) + at;
        const int lo = max(0, begin - j * kPageSize), hi = min(kPageSize, begin + len - j * kPageSize);
        desc = slice_desc(seg, lo, hi, hi - lo == kPageSize && ((uint32_t)(mask >> row0) & my_rows) == my_rows);
    };
    const uint8_t *next_k = nullptr, *next_v = nullptr;
    uint32_t cur = 0, next = 0;     // the batch in hand, and the one whose copies go out
    get_slice(0, next_k, next_v, next);
    cur = next;
    const uint32_t lane_ring = ring + lane % PP * C::kPage;
    auto issue = [&](int i) {
        const int first = i % kBatch * PP;
        if (first == 0 && i > 0)
            get_slice(i, next_k, next_v, next);
        const uint32_t bar = bars + (i % kStages) * 8;
        if (lane == first)
            tc::mbar_arrive_expect_tx(bar, min(PP, total - (ts + i * TS) * PP) * C::kPage);
        __syncwarp();
        if (lane / PP == i % kBatch && next != 0) {
            const uint32_t to = lane_ring + (i % kStages) * C::kStage;
            tc::bulk_load(to, next_k, P::kBytes, bar, pol);
            tc::bulk_load(to + P::kBytes, next_v, P::kBytes, bar, pol);
        }
    };
    __syncwarp();   // the barriers are there
    int issued = 0;
    for (; issued < mine && issued < kStages; ++issued)
        issue(issued);

    // ---- Q^T fragments ----
    uint32_t qa[C::kQSmem ? 1 : NT][KW * 4];
    uint4 *qs = reinterpret_cast<uint4 *>(smem + C::q) + warp * NT * KW * 32 + lane;
    float f[NT][2];                 // what rows 2t and 2t + 1 of S are multiplied by
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        uint32_t (&w)[KW * 4] = qw[n];
        // 2^e, in two factors for rows below 2^-112 (e reaches 147).
        const int e = row_exponent<KW * 4, 4>(w), e1 = min(e, 126), e2 = e - e1;
        // (A factor past fp32, for a row near its end, leaves logits of 0.)
        const float up = kv4::pow2(e1), fr = fminf(a.scale_log2 * kv4::pow2(-e1) * ka.k_scale * kv4::pow2(-e2), FLT_MAX);
        f[n][0] = __shfl_sync(kAll, fr, 8 * t);
        f[n][1] = __shfl_sync(kAll, fr, 8 * t + 4);
        if (e2 == 0) {
#pragma unroll
            for (int i = 0; i < KW * 4; ++i) {
                const float2 v = bf16x2_to_float2(w[i]);
                w[i] = kv4::f16x2(v.x * up, v.y * up);
            }
        } else {
            const float up2 = kv4::pow2(e2);
#pragma unroll
            for (int i = 0; i < KW * 4; ++i) {
                const float2 v = bf16x2_to_float2(w[i]);
                w[i] = kv4::f16x2(v.x * up * up2, v.y * up * up2);
            }
        }
        if constexpr (C::kQSmem) {
#pragma unroll
            for (int i = 0; i < KW; ++i)
                qs[(n * KW + i) * 32] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < KW * 4; ++i)
                qa[n][i] = w[i];
        }
    }

    float o[D / 16][NT][4];
    float m[NT][2], l[NT][2];       // maxima less kLift, sums
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
            o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.f;
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.f;
    }
    // MMA row r holds token r ^ (r >> 1 & 1) of the page: then the eight lanes
    // of a 16-byte read of K and the sixteen of an 8-byte read of V, whose
    // rows are 64 bytes, meet the fewest bank conflicts (24 reads of
    // shared memory a page, not 40).
    const int kg = g ^ (g >> 1 & 1);
    const int vx = 2 * t + (t & 1), vy = 2 * t + 1 - (t & 1);
    auto landed = [&](int stage, uint32_t parity) { return tc::mbar_wait(bars + stage * 8, parity); };
    int failed = -1;                // the step whose copy did not land in time
    for (int i = 0; i < mine; ++i) {
        if (i > 0 && i % kBatch == 0)
            cur = next;      // (issue() is at most kStages ahead: it has filled this batch)
        uint32_t desc[PP];
        bool whole = true;
#pragma unroll
        for (int p2 = 0; p2 < PP; ++p2) {
            desc[p2] = __shfl_sync(kAll, cur, i % kBatch * PP + p2);
            whole &= desc[p2] >> 31 != 0;
        }
        if (!__all_sync(kAll, ring_wait(i, kStages, landed))) {
            failed = i;
            break;
        }
        uint8_t *stage = smem + (warp * kStages + i % kStages) * C::kStage;
        // ---- S^T ----
        float s[PP][NT][4];
#pragma unroll
        for (int p2 = 0; p2 < PP; ++p2) {
            const uint8_t *ks = stage + p2 * C::kPage;
#pragma unroll
            for (int n = 0; n < NT; ++n)
                s[p2][n][0] = s[p2][n][1] = s[p2][n][2] = s[p2][n][3] = 0.f;
            uint32_t w0[KW], w1[KW], sc0[KW / 2], sc1[KW / 2];
            if constexpr (D == 128) {
                const uint4 x = *reinterpret_cast<const uint4 *>(ks + kg * P::kRow + t * 16);
                const uint4 y = *reinterpret_cast<const uint4 *>(ks + (kg + 8) * P::kRow + t * 16);
                w0[0] = x.x, w0[1] = x.y, w0[2] = x.z, w0[3] = x.w;
                w1[0] = y.x, w1[1] = y.y, w1[2] = y.z, w1[3] = y.w;
                const uint32_t u = kv4::scales2(*reinterpret_cast<const uint16_t *>(ks + P::kScales + kg * P::kScaleRow + t * 2));
                const uint32_t v = kv4::scales2(*reinterpret_cast<const uint16_t *>(ks + P::kScales + (kg + 8) * P::kScaleRow + t * 2));
                sc0[0] = __byte_perm(u, 0, 0x1010), sc0[1] = __byte_perm(u, 0, 0x3232);
                sc1[0] = __byte_perm(v, 0, 0x1010), sc1[1] = __byte_perm(v, 0, 0x3232);
            } else {
                const uint2 x = *reinterpret_cast<const uint2 *>(ks + kg * P::kRow + t * 8);
                const uint2 y = *reinterpret_cast<const uint2 *>(ks + (kg + 8) * P::kRow + t * 8);
                w0[0] = x.x, w0[1] = x.y;
                w1[0] = y.x, w1[1] = y.y;
                const uint32_t u = ks[P::kScales + kg * P::kScaleRow + t], v = ks[P::kScales + (kg + 8) * P::kScaleRow + t];
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
                    uint4 q;
                    if constexpr (C::kQSmem)
                        q = qs[(n * KW + w) * 32];
                    else
                        q = make_uint4(qa[n][4 * w], qa[n][4 * w + 1], qa[n][4 * w + 2], qa[n][4 * w + 3]);
                    mma16816(s[p2][n], x[0], y[0], x[1], y[1], q.x, q.y);
                    mma16816(s[p2][n], x[2], y[2], x[3], y[3], q.z, q.w);
                }
            }
        }
        // ---- softmax ----
        // The weights' exponents: s f - m + kLift; above kLift + kUp (an m of
        // -inf, as at the start, among them) the maxima are raised first.
        float x[PP][NT][4];
        bool grow = false;
        auto exponents = [&]() {
#pragma unroll
            for (int p2 = 0; p2 < PP; ++p2)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        x[p2][n][j] = fmaf(s[p2][n][j], f[n][j & 1], -m[n][j & 1]);
        };
        exponents();
        if (!whole) {
#pragma unroll
            for (int p2 = 0; p2 < PP; ++p2) {
                const int lo = desc[p2] >> 8 & 255, hi = desc[p2] & 255;
                const uint32_t rows = (uint32_t)((nseg > 1 ? seg_mask[desc[p2] >> 16 & 0x7fff] : mask0) >> row0);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int tok = kg + (j >> 1) * 8, row = 8 * n + 2 * t + (j & 1);
                        if (tok < lo || tok >= hi || !((rows >> row) & 1)) {
                            s[p2][n][j] = -INFINITY;    // (f is positive)
                            x[p2][n][j] = -INFINITY;
                        }
                    }
                // What a page holds beside the segment's tokens may be
                // anything: V's scales there become 0.
                constexpr int kWords = P::kScaleRow / 4;        // of a token's scales
                uint32_t *sc = reinterpret_cast<uint32_t *>(stage + p2 * C::kPage + P::kBytes + P::kScales);
                if (lane < kPageSize * kWords && (lane / kWords < lo || lane / kWords >= hi))
                    sc[lane] = 0u;
            }
            tc::fence_proxy_async();    // (the stage's next page is a bulk copy)
            __syncwarp();
        }
#pragma unroll
        for (int p2 = 0; p2 < PP; ++p2)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    grow |= x[p2][n][j] > kv4::kLift + kv4::kUp;
        if (__any_sync(kAll, grow)) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float y = -INFINITY;
#pragma unroll
                    for (int p2 = 0; p2 < PP; ++p2)
                        y = fmaxf(y, fmaxf(s[p2][n][j] * f[n][j], s[p2][n][j + 2] * f[n][j]));
                    y = fmaxf(y, __shfl_xor_sync(kAll, y, 4));
                    y = fmaxf(y, __shfl_xor_sync(kAll, y, 8));
                    y = fmaxf(y, __shfl_xor_sync(kAll, y, 16));
                    y = fmaxf(m[n][j], y - kv4::kLift);
                    y = y == INFINITY ? kv4::nan() : y;       // a logit past fp32: for good, through l
                    const float alpha = y == m[n][j] ? 1.f : tc::ex2(m[n][j] - y);
                    m[n][j] = y;
                    l[n][j] *= alpha;
#pragma unroll
                    for (int d = 0; d < D / 16; ++d) {
                        o[d][n][j] *= alpha;
                        o[d][n][j + 2] *= alpha;
                    }
                }
            }
            exponents();
            // A masked place, also in a row whose maximum is still -inf.
#pragma unroll
            for (int p2 = 0; p2 < PP; ++p2)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        x[p2][n][j] = s[p2][n][j] == -INFINITY ? -INFINITY : x[p2][n][j];
        }
        uint32_t pb[PP][NT][2];
#pragma unroll
        for (int p2 = 0; p2 < PP; ++p2)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float p0 = tc::ex2(x[p2][n][0]), p1 = tc::ex2(x[p2][n][1]);
                const float p3 = tc::ex2(x[p2][n][3]), q0 = tc::ex2(x[p2][n][2]);
                l[n][0] += p0 + q0;
                l[n][1] += p1 + p3;
                pb[p2][n][0] = transpose8(kv4::f16x2(p0, p1));
                pb[p2][n][1] = transpose8(kv4::f16x2(q0, p3));
            }
        // ---- O^T ----
#pragma unroll
        for (int p2 = 0; p2 < PP; ++p2) {
            const uint8_t *vs = stage + p2 * C::kPage + P::kBytes;
            uint32_t sv[2], vw[2][2][VW];     // by token pair: scales, words of both tokens
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const uint8_t *sx = vs + P::kScales + (D == 128 ? g : g >> 1);
                const uint32_t x = sx[(vx + 8 * q) * P::kScaleRow], y = sx[(vy + 8 * q) * P::kScaleRow];
                sv[q] = kv4::scales2(x | y << 8);
                const uint8_t *rx = vs + (vx + 8 * q) * P::kRow + g * (D / 16), *ry = vs + (vy + 8 * q) * P::kRow + g * (D / 16);
                if constexpr (D == 128) {
                    const uint2 u = *reinterpret_cast<const uint2 *>(rx), v = *reinterpret_cast<const uint2 *>(ry);
                    vw[q][0][0] = u.x, vw[q][0][1] = u.y;
                    vw[q][1][0] = v.x, vw[q][1][1] = v.y;
                } else {
                    vw[q][0][0] = *reinterpret_cast<const uint32_t *>(rx);
                    vw[q][1][0] = *reinterpret_cast<const uint32_t *>(ry);
                }
            }
#pragma unroll
            for (int w = 0; w < VW; ++w) {
                uint32_t e[2][4], od[2][4];   // even and odd dims of the word, by token pair
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const uint32_t x = vw[q][0][w], y = vw[q][1][w];
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
                        mma16816(o[4 * w + k][n], e[0][k], od[0][k], e[1][k], od[1][k], pb[p2][n][0], pb[p2][n][1]);
            }
        }
        // The stage is free once every lane has read it.
        __syncwarp();
        if (issued < mine) {
            issue(issued);
            ++issued;
        }
    }
    if (failed >= 0) {
        // A copy that did not land: time for it and for those behind it, before
        // the ring is used for the states or freed, and say so.
        ring_drain(failed, issued, kStages, landed);
        if (lane == 0)
            report_failure(p.status, 401);
#pragma unroll
        for (int n = 0; n < NT; ++n)
            l[n][0] = l[n][1] = kv4::nan();
    }

    // ---- the states of the warps that shared the slices, joined by halves:
    // the upper half writes its state, lane by lane, the lower takes it in ----
    if (TS > 1) {
        for (int half = TS / 2; half >= 1; half /= 2) {
            __syncthreads();   // the ring, or the states before, have been read
            const int pair = (warp / TS) * half + (ts & (half - 1));
            float *st = reinterpret_cast<float *>(smem) + (size_t)pair * (C::kState / 4);
            if (ts >= half && ts < 2 * half) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    reinterpret_cast<float4 *>(st)[n * 32 + lane] = make_float4(m[n][0], m[n][1], l[n][0], l[n][1]);
#pragma unroll
                    for (int d = 0; d < D / 16; ++d)
                        reinterpret_cast<float4 *>(st)[(NT + n * (D / 16) + d) * 32 + lane] =
                            make_float4(o[d][n][0], o[d][n][1], o[d][n][2], o[d][n][3]);
                }
            }
            __syncthreads();
            if (ts < half) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float4 x = reinterpret_cast<const float4 *>(st)[n * 32 + lane];
                    const float mj[2] = {x.x, x.y}, lj[2] = {x.z, x.w};
                    float wa[2], wb[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float M = fmaxf(m[n][j], mj[j]);
                        wa[j] = M == -INFINITY ? 1.f : tc::ex2(m[n][j] - M);
                        wb[j] = M == -INFINITY ? 1.f : tc::ex2(mj[j] - M);
                        m[n][j] = M;
                        l[n][j] = l[n][j] * wa[j] + lj[j] * wb[j];
                    }
#pragma unroll
                    for (int d = 0; d < D / 16; ++d) {
                        const float4 y = reinterpret_cast<const float4 *>(st)[(NT + n * (D / 16) + d) * 32 + lane];
                        o[d][n][0] = o[d][n][0] * wa[0] + y.x * wb[0];
                        o[d][n][1] = o[d][n][1] * wa[1] + y.y * wb[1];
                        o[d][n][2] = o[d][n][2] * wa[0] + y.z * wb[0];
                        o[d][n][3] = o[d][n][3] * wa[1] + y.w * wb[1];
                    }
                }
            }
        }
    }

    // ---- out: lane (g, t) holds dims (D / 8) g .. of rows 2t and 2t + 1 ----
    if (ts == 0) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float sum = l[n][j];
                sum += __shfl_xor_sync(kAll, sum, 4);
                sum += __shfl_xor_sync(kAll, sum, 8);
                sum += __shfl_xor_sync(kAll, sum, 16);
                const int r = row0 + 8 * n + 2 * t + j;
                if (r >= R)
                    continue;
                // sum is 0 where the row attends no token, NaN where a logit was.
                const float inv = sum == 0.f ? 0.f : ka.v_scale / sum;
                const float lse2 = sum == 0.f ? -INFINITY : m[n][j] + log2f(sum);
                const int k = r / G, head = h * G + (r - k * G);
                const bool straight = r < 32 && ((direct >> r) & 1u);
                const size_t row = (size_t)(straight ? p.chunk_q[cq0 + k] : cq0 + k) * Hq + head;
                const size_t at = row * D + g * (D / 8);
                if (straight && a.out_dtype == DEFT_OUT_BF16) {
#pragma unroll
                    for (int d = 0; d < D / 16; d += 4) {
                        uint32_t w[4];
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const __nv_bfloat162 b = __floats2bfloat162_rn(o[d + x][n][j] * inv, o[d + x][n][j + 2] * inv);
                            w[x] = *reinterpret_cast<const uint32_t *>(&b);
                        }
                        reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + at)[d / 4] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                } else {
                    float4 *dst = reinterpret_cast<float4 *>((straight ? static_cast<float *>(a.out) : a.o_part) + at);
#pragma unroll
                    for (int d = 0; d < D / 16; d += 2)
                        dst[d / 2] = make_float4(o[d][n][j] * inv, o[d][n][j + 2] * inv, o[d + 1][n][j] * inv, o[d + 1][n][j + 2] * inv);
                }
                if (g == 0) {
                    if (straight)
                        a.lse_out[row] = direct_lse(lse2);
                    else    // (+inf, so that the merge's weight for it is NaN and not 0)
                        a.lse_part[row] = lse2 == lse2 ? lse2 : INFINITY;
                }
            }
    }
    // The merge waits for this launch alone: its last CTA waits for the ones
    // before.
    if (ka.last && blockIdx.x == gridDim.x - 1)
        grid_dep_wait();
}

template <int D, int NT>
int launch(Kv4Args ka, const DevPartition &p, cudaStream_t st)
{
    ka.head_groups = ka.a.num_kv_heads / ka.heads;      // (heads divides them: every warp has a unit)
    const int64_t ctas = (int64_t)ka.n * ka.head_groups;
    if (ctas > INT32_MAX)
        return (int)cudaErrorInvalidConfiguration;
    auto *kernel = phase1_kv4_kernel<D, NT>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D, NT>::total);
    if (e != cudaSuccess)
        return (int)e;
    return (int)launch_dependent(kernel, dim3((unsigned)ctas), dim3(kThreads), Cfg<D, NT>::total, st, ka, p);
}

// KV heads that a CTA takes, of the most it can (a unit a warp, or a pair of
// warps for two groups of rows): fewer, several warps then sharing a unit's
// pages, while all CTAs still run at once.
int heads_per_cta(int64_t items, int32_t hkv, int most, int64_t slots)
{
    int heads = most;
    while (heads > 1 && items * (hkv / (heads / 2)) <= slots)
        heads /= 2;
    return heads;
}

// The merge of each row's partials by their lse, as phase2.cu's, with W warps
// a row: a path of many chunks (33 of 256 tokens in 8192) is read by four
// warps at once instead of in a chain of 16 loads and then one after another
// (64 requests of 64 to 8192 tokens in chunks of 256; with at most 8 partials
// a row a warp reads them all at once, and four warps only added a barrier).
// Also, lse is NaN where a logit was.
template <int D, int W>
__global__ void __launch_bounds__(kThreads) merge4_kernel(AttnArgs a, const int32_t *__restrict__ q_slot_off,
                                                          const int32_t *__restrict__ q_slot,
                                                          const int32_t *__restrict__ queries, int32_t nq)
{
    constexpr int E = D / 32, KP = 8;     // elements of a lane, partials loaded at once
    __shared__ float st[kWarps][D + 2];
    grid_dep_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % W;
    const int64_t job = (int64_t)blockIdx.x * (kWarps / W) + warp / W;
    const bool live = job < (int64_t)nq * a.num_q_heads;
    const int i = live ? (int)(job / a.num_q_heads) : 0, h = (int)(job - (int64_t)i * a.num_q_heads);
    const int q = queries ? queries[i] : i;
    const int s0 = q_slot_off[q], n = live ? q_slot_off[q + 1] - s0 : 0;
    float M = -INFINITY, sum = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e)
        acc[e] = 0.f;
    bool waited = false;
    for (int b = part; b < n; b += 32 * W) {
        const int k = b + lane * W, here = min(32, (n - b + W - 1) / W);
        size_t row = 0;
        if (k < n)
            row = (size_t)q_slot[s0 + k] * a.num_q_heads + h;
        if (!waited)
            grid_dep_wait();       // the phase-1 launches have completed
        waited = true;
        const float l = k < n ? a.lse_part[row] : -INFINITY;
        const float top = fmaxf(M, warp_max(l));
        if (top == -INFINITY)
            continue;              // partials that attended nothing
        const float keep = tc::ex2(M - top), w = k < n ? tc::ex2(l - top) : 0.f;
        M = top;
        sum = sum * keep + warp_sum(w);
#pragma unroll
        for (int e = 0; e < E; ++e)
            acc[e] *= keep;
        for (int j0 = 0; j0 < here; j0 += KP) {
            float v[KP][E], wj[KP];
#pragma unroll
            for (int j = 0; j < KP; ++j) {
                const size_t r = __shfl_sync(kAll, row, (j0 + j) & 31);
                wj[j] = __shfl_sync(kAll, w, (j0 + j) & 31);
                const float *src = a.o_part + r * D + lane * E;
                if (j0 + j >= here) {
                    wj[j] = 0.f;
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        v[j][e] = 0.f;
                } else if constexpr (E == 4) {
                    const float4 x = *reinterpret_cast<const float4 *>(src);
                    v[j][0] = x.x, v[j][1] = x.y, v[j][2] = x.z, v[j][3] = x.w;
                } else {
                    const float2 x = *reinterpret_cast<const float2 *>(src);
                    v[j][0] = x.x, v[j][1] = x.y;
                }
            }
#pragma unroll
            for (int j = 0; j < KP; ++j)
#pragma unroll
                for (int e = 0; e < E; ++e)
                    acc[e] = fmaf(wj[j], v[j][e], acc[e]);
        }
    }
    if (!waited)
        grid_dep_wait();
    if constexpr (W > 1) {
#pragma unroll
        for (int e = 0; e < E; ++e)
            st[warp][lane * E + e] = acc[e];
        if (lane == 0) {
            st[warp][D] = M;
            st[warp][D + 1] = sum;
        }
        __syncthreads();
        if (part != 0)
            return;
        float top = M;
        for (int w = 1; w < W; ++w)
            top = fmaxf(top, st[warp + w][D]);
        sum = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e)
            acc[e] = 0.f;
        for (int w = 0; w < W; ++w) {
            const float x = st[warp + w][D] == -INFINITY ? 0.f : tc::ex2(st[warp + w][D] - top);
            sum = fmaf(x, st[warp + w][D + 1], sum);
#pragma unroll
            for (int e = 0; e < E; ++e)
                acc[e] = fmaf(x, st[warp + w][lane * E + e], acc[e]);
        }
        M = top;
    }
    if (!live)
        return;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const size_t row = (size_t)q * a.num_q_heads + h;
#pragma unroll
    for (int e = 0; e < E; ++e)
        acc[e] *= inv;
    if (a.out_dtype == DEFT_OUT_F32) {
        float *o = static_cast<float *>(a.out) + row * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; e += 2)
            *reinterpret_cast<float2 *>(o + e) = make_float2(acc[e], acc[e + 1]);
    } else {
        __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.out) + row * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; e += 2)
            *reinterpret_cast<__nv_bfloat162 *>(o + e) = __floats2bfloat162_rn(acc[e], acc[e + 1]);
    }
    if (lane == 0)
        a.lse_out[row] = sum == 0.f ? -INFINITY : direct_lse(M + log2f(sum));
}

template <int D>
int launch_merge4(const AttnArgs &a, const DevPartition &p, const int32_t *queries, int32_t nq, int32_t slots, cudaStream_t st)
{
    const int64_t rows = (int64_t)nq * a.num_q_heads;
    const int per = slots > 8 ? 1 : kWarps;
    const int64_t ctas = (rows + per - 1) / per;
    if (ctas > INT32_MAX)
        return (int)cudaErrorInvalidConfiguration;
    return (int)launch_dependent(per == 1 ? merge4_kernel<D, kWarps> : merge4_kernel<D, 1>, dim3((unsigned)ctas), dim3(kThreads), 0, st, a,
                                 p.q_slot_off, p.q_slot, queries, nq);
}

}  // namespace

int dispatch_step4(const AttnArgs &a, const DevPartition &dp, const Partition &hp, float k_scale, float v_scale,
                   int32_t max_slots, void *stream, const LaunchTracer &trace)
{
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    Kv4Args ka{};
    ka.a = a;
    ka.k_scale = k_scale, ka.v_scale = v_scale;
    ka.mma_narrow = hp.mma_bucket_off[1];
    // One or two launches for each width, the widest first: 33 to 64 and 16 to
    // 32 rows (the tensor-core list; on mma.sync at head_dim 64), 9 to 15, up
    // to 8.
    struct Part {
        int32_t wide, first, n, rows;
    };
    const int32_t few = hp.fma_bucket_off[4], all = dp.num_fma_items, narrow = hp.mma_bucket_off[1], mma = dp.num_mma_items;
    const bool tc = a.head_dim == 128;
    const Part parts[4] = {{1, tc ? narrow : 0, tc ? mma - narrow : mma, 64}, {1, 0, tc ? narrow : 0, 32}, {0, few, all - few, 16}, {0, 0, few, 8}};
    for (const Part &x : parts) {
        if (x.n == 0)
            continue;
        ka.wide = x.wide;
        // Whole rounds of CTAs with as many heads as they take, and the rest
        // over more CTAs (64 requests: 830 CTAs of four heads are one round
        // of 608 and 222 that would keep the device waiting for their whole
        // length).  The items of one width are sorted by length, so that the
        // rest are the shorter ones; of several widths joined here (1, 2, 4
        // and 8 rows; at head_dim 64 32 and 64) they are sorted by width
        // first, and the rest come from the widest.
        const bool tcgen = x.wide && tc;
        const int64_t slots = (int64_t)(x.rows > 16 ? 2 : x.rows > 8 ? 3 : 4) * num_sms();
        int most = x.rows > 16 ? 2 : 4;
        while (a.num_kv_heads % most != 0)
            most /= 2;
        const int32_t groups = a.num_kv_heads / most;
        int32_t bulk = tcgen ? x.n : (int32_t)((int64_t)x.n * groups / slots * slots / groups);
        for (int32_t done = 0; done < x.n;) {
            const bool rest = done >= bulk;
            ka.first = x.first + done;
            ka.n = rest ? x.n - done : bulk;
            ka.heads = rest ? heads_per_cta(ka.n, a.num_kv_heads, most, slots) : most;
            const int r = trace({DEFT_K_PHASE1_KV4, 0, x.rows, 0, ka.n, 0.f}, stream, [&] {
                if (x.wide)
                    return tc ? launch_phase1_kv4_mma(ka, dp, x.rows, stream) : launch<64, 4>(ka, dp, st);
                if (a.head_dim == 128)
                    return x.rows > 8 ? launch<128, 2>(ka, dp, st) : launch<128, 1>(ka, dp, st);
                return x.rows > 8 ? launch<64, 2>(ka, dp, st) : launch<64, 1>(ka, dp, st);
            });
            if (r)
                return r;
            done += ka.n;
            ka.a.wait_prior = 0;
            ka.last = 1;
        }
    }
    const int32_t nq = a.direct ? dp.num_merge_q : dp.num_queries;
    if (nq == 0)
        return 0;
    const int32_t *qlist = nq < dp.num_queries ? dp.merge_q : nullptr;
    return trace({DEFT_K_PHASE2, 0, 0, 0, nq, 0.f}, stream, [&] {
        return a.head_dim == 128 ? launch_merge4<128>(a, dp, qlist, nq, max_slots, st) : launch_merge4<64>(a, dp, qlist, nq, max_slots, st);
    });
}

}  // namespace deft
