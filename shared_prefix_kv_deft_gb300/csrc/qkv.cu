// qkv.cu -- the attention block's inputs on their way from the projection to
// the cache: head norms and the position rotation of q and k, with k and v
// appended to the paged cache in bf16 (deft_qkv_write) or in 4 bits
// (deft_qkv_write4), and 4-bit pages back as bf16 pages (deft_kv_unpack4).
//
// For a head x of head_dim D at position p, in fp32 throughout:
//     y_i = x_i * r * w_i,  r = 1 / sqrt(sum x_i^2 / D + eps)      (norm)
//     (a, b) -> (a cos - b sin, b cos + a sin)                     (rotation)
// for the pairs (a, b) = (y_i, y_{i + R/2}), or (y_2i, y_2i+1), of the first
// R elements, cos and sin from the caller's table, then one rounding to
// bf16.  In 4 bits (kv4.cuh) that bf16 value is what is quantised.
//
// Every product and sum rounds by itself (no fused multiply-add) and the
// squares are added neighbours first, so that the result does not depend on
// which thread holds what: in 4 bits, a value next to a border between two
// codes would otherwise differ by a whole code from one form of the call to
// another.
//
// Layout.  D / 16 lanes hold a head's row, two 8-element pieces each: pieces
// (j, j + R/16) where the rotation pairs them, so that both elements of a
// pair are in one lane, else (j, j + D/16), so that every access covers whole
// sectors (with neighbouring pieces in a lane the v rows' 16-byte stores left
// half sectors to the L2).  A warp takes one or two rounds of
// 32 / (D / 16) heads of one kind (q, k or v) of one token, all loads ahead
// of the arithmetic; the token's cos and sin stay in registers over them.
// 32768 tokens (32/8 heads of 128, bf16): 136 us, 6.0 TB/s; the 822 MB at
// the measured copy rate take 121.  Bound by the rows in flight: persistent
// CTAs fed by a ring of bulk copies in shared memory took 164 us.
#include <cstdint>

#include "common.cuh"
#include "deft_internal.h"
#include "kv4.cuh"

namespace deft {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr unsigned kAll = 0xffffffffu;
// Heads a group of lanes takes, and the CTAs that an SM is to hold (which sets
// the registers): rows in flight against warps in flight.  32768 tokens of
// bf16, 32/8 heads of 128: 2 and 9 136 us, though some registers spill, 2 and 8
// 142, 2 and 7 151, 2 and 10 160, 3 and 6 162 (CTAs of 256 threads, 2 and 4:
// 145, rows' lines marked for eviction first: 148); 10007 tokens of fp32, 12/4
// heads of 64: 1 and 10 18.4 us, 1 and 9 20.5, 1 and 11 20.5, 2 and 7 21.0.
template <bool kF32>
struct Shape {
    static constexpr int kHeads = kF32 ? 1 : 2, kCtas = kF32 ? 10 : 9;
};

struct QkvArgs {
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;   // elements between tokens
    const int32_t *slot, *position;
    const float *cos_sin;                   // [num_positions][rot_dim]: cos, then sin
    const void *q_norm, *k_norm;            // in the inputs' type, or null
    float eps;
    int32_t num_positions, half;            // half: 8-element pieces of rot_dim / 2
    int32_t split;                          // pairs (i, i + rot_dim / 2), not neighbours
    __nv_bfloat16 *q_out;
    uint8_t *k_pages, *v_pages;
    float k_scale, v_scale, k_six, v_six;   // 4 bits: g and 6 g
    int32_t num_tokens, num_pages, num_q_heads, num_kv_heads;
    int32_t q_tasks, kv_tasks;              // warps of one token for q, and for each of k and v
};

// Eight consecutive elements.
template <bool kF32>
struct Piece {
    uint4 v[kF32 ? 2 : 1];
    __device__ __forceinline__ void zero()
    {
        v[0] = make_uint4(0, 0, 0, 0);
        if constexpr (kF32)
            v[1] = v[0];
    }
    // kKept: of memory that nothing writes while the kernel runs (the rows may
    // be queries in place).
    template <bool kKept = false>
    __device__ __forceinline__ void load(const void *src, int64_t elem)
    {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const char *>(src) + elem * (kF32 ? 4 : 2));
        v[0] = kKept ? __ldg(p) : p[0];
        if constexpr (kF32)
            v[1] = kKept ? __ldg(p + 1) : p[1];
    }
    __device__ __forceinline__ void values(float (&x)[8]) const
    {
        if constexpr (kF32) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                x[4 * i] = __uint_as_float(v[i].x), x[4 * i + 1] = __uint_as_float(v[i].y);
                x[4 * i + 2] = __uint_as_float(v[i].z), x[4 * i + 3] = __uint_as_float(v[i].w);
            }
        } else {
            const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
    }
};

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi)
{
    const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&r);
}

__device__ __forceinline__ float square_sum(const float (&x)[8])
{
    float s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        s[i] = __fadd_rn(__fmul_rn(x[2 * i], x[2 * i]), __fmul_rn(x[2 * i + 1], x[2 * i + 1]));
    return __fadd_rn(__fadd_rn(s[0], s[1]), __fadd_rn(s[2], s[3]));
}

// The lane's two pieces of a row: j and j + half for the lanes j < half (where
// the rotation pairs pieces half apart), 2j and 2j + 1 for the others.
template <int D, bool kWhole>
struct Place {
    static constexpr int kLanes = D / 16;   // lanes of a row; as `half`: no lane is another
    int half;                               // (kWhole: it is that)
    int j;        // lane in the row
    int p0, p1;   // its pieces
    __device__ __forceinline__ Place(int lane, int half_) : half(kWhole ? kLanes : half_), j(lane % kLanes)
    {
        const bool paired = j < half;
        p0 = paired ? j : 2 * j;
        p1 = paired ? j + half : 2 * j + 1;
    }
    // The value that belongs to piece p, of the lanes' (a, b) for their
    // pieces (p0, p1); every lane of the warp calls it.
    __device__ __forceinline__ float of(int p, float a, float b) const
    {
        const bool paired = p < 2 * half;
        const int src = paired ? (p < half ? p : p - half) : p >> 1;
        const bool second = paired ? p >= half : (p & 1) != 0;
        const float x = __shfl_sync(kAll, a, src, kLanes), y = __shfl_sync(kAll, b, src, kLanes);
        return second ? y : x;
    }
    // The row's sum of the pieces' sums, neighbours first.
    __device__ __forceinline__ float row_sum(float a, float b) const
    {
        if (kWhole || half == kLanes) {     // pieces j and j + kLanes: both halves of the row
#pragma unroll
            for (int o = 1; o < kLanes; o <<= 1) {
                a = __fadd_rn(a, __shfl_xor_sync(kAll, a, o));
                b = __fadd_rn(b, __shfl_xor_sync(kAll, b, o));
            }
            return __fadd_rn(a, b);
        }
        float s = __fadd_rn(of(2 * j, a, b), of(2 * j + 1, a, b));
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1)
            s = __fadd_rn(s, __shfl_xor_sync(kAll, s, o));
        return s;
    }
    // The larger of a value over each of the lane's pieces and the other
    // piece of its block.
    __device__ __forceinline__ void block_max(float &a, float &b) const
    {
        const bool whole = kWhole || half == kLanes;    // then the other piece is the neighbouring lane's
        const float x = whole ? __shfl_xor_sync(kAll, a, 1) : of(p0 ^ 1, a, b);
        const float y = whole ? __shfl_xor_sync(kAll, b, 1) : of(p1 ^ 1, a, b);
        a = kv4::max_nan(a, x);
        b = kv4::max_nan(b, y);
    }
};

// kWhole: the rotation turns whole heads, in halves.
template <int D, bool kF32, bool k4, bool kWhole>
__global__ void __launch_bounds__(kThreads, Shape<kF32>::kCtas) qkv_kernel(QkvArgs a)
{
    constexpr int kLanes = D / 16, kRows = 32 / kLanes, C = Shape<kF32>::kHeads;
    const int lane = threadIdx.x & 31, sub = lane / kLanes;
    const uint32_t per_token = (uint32_t)(a.q_tasks + 2 * a.kv_tasks);
    const uint32_t task = blockIdx.x * kWarps + (threadIdx.x >> 5);
    const uint32_t tok = task / per_token;
    if (tok >= (uint32_t)a.num_tokens)
        return;
    int part = (int)(task - tok * per_token);
    const int kind = part < a.q_tasks ? 0 : part < a.q_tasks + a.kv_tasks ? 1 : 2;
    part -= kind == 0 ? 0 : kind == 1 ? a.q_tasks : a.q_tasks + a.kv_tasks;
    const int heads = kind == 0 ? a.num_q_heads : a.num_kv_heads;
    const void *src = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
    const int64_t row0 = (int64_t)tok * (kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride);
    const int32_t slot = kind == 0 ? 0 : a.slot[tok];
    const int half = kind == 2 ? 0 : kWhole ? kLanes : a.half;
    const bool split = kWhole || a.split;
    const Place<D, kWhole> at(lane, split && half > 0 ? half : kLanes);
    const int head0 = part * (C * kRows) + sub;

    // (The position first: the angles wait for it.)
    const int32_t pos = kind == 2 || a.half == 0 ? 0 : a.position[tok];
    Piece<kF32> raw[C][2];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int h = head0 + c * kRows;
        if (h < heads) {
            raw[c][0].load(src, row0 + (int64_t)h * D + at.p0 * 8);
            raw[c][1].load(src, row0 + (int64_t)h * D + at.p1 * 8);
        } else {
            raw[c][0].zero();
            raw[c][1].zero();
        }
    }
    // (After the loads, which so do not wait for it: 148 us where 158.
    // An unsigned comparison: a negative slot is past the end too.)
    if (kind != 0 && (uint32_t)slot >= (uint32_t)a.num_pages * kPageSize)
        return;
    // The lane's eight angles: those of its elements (both pieces' are the
    // same), or four for each piece's pairs of neighbours.
    const bool turns0 = split ? at.j < half : at.p0 < 2 * half, turns1 = split ? turns0 : at.p1 < 2 * half;
    float cs[8], sn[8];
    if (turns0) {
        if ((uint32_t)pos < (uint32_t)a.num_positions) {
            const float4 *t = reinterpret_cast<const float4 *>(a.cos_sin + (int64_t)pos * half * 16);
            const int i0 = split ? 2 * at.j : at.p0, i1 = split ? 2 * at.j + 1 : turns1 ? at.p1 : at.p0;
            const float4 c0 = __ldg(t + i0), c1 = __ldg(t + i1), s0 = __ldg(t + half * 2 + i0), s1 = __ldg(t + half * 2 + i1);
            cs[0] = c0.x, cs[1] = c0.y, cs[2] = c0.z, cs[3] = c0.w, cs[4] = c1.x, cs[5] = c1.y, cs[6] = c1.z, cs[7] = c1.w;
            sn[0] = s0.x, sn[1] = s0.y, sn[2] = s0.z, sn[3] = s0.w, sn[4] = s1.x, sn[5] = s1.y, sn[6] = s1.z, sn[7] = s1.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                cs[i] = sn[i] = __int_as_float(0x7fffffff);
        }
    }
    const void *norm = kind == 0 ? a.q_norm : kind == 1 ? a.k_norm : nullptr;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int h = head0 + c * kRows;
        float x[2][8];
        raw[c][0].values(x[0]);
        raw[c][1].values(x[1]);
        if (norm) {
            const float ss = at.row_sum(square_sum(x[0]), square_sum(x[1]));
            const float r = __frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(ss, 1.f / D), a.eps)));
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                Piece<kF32> wp;
                wp.template load<true>(norm, (p == 0 ? at.p0 : at.p1) * 8);
                float w[8];
                wp.values(w);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    x[p][i] = __fmul_rn(__fmul_rn(x[p][i], r), w[i]);
            }
        }
        if (turns0) {
            if (split) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float u = x[0][i], v = x[1][i];
                    x[0][i] = __fsub_rn(__fmul_rn(u, cs[i]), __fmul_rn(v, sn[i]));
                    x[1][i] = __fadd_rn(__fmul_rn(v, cs[i]), __fmul_rn(u, sn[i]));
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {       // pair i % 4 of piece i / 4, angle i
                    if (i == 4 && !turns1)
                        break;
                    float &u = x[i / 4][2 * (i % 4)], &v = x[i / 4][2 * (i % 4) + 1];
                    const float t = __fsub_rn(__fmul_rn(u, cs[i]), __fmul_rn(v, sn[i]));
                    v = __fadd_rn(__fmul_rn(v, cs[i]), __fmul_rn(u, sn[i]));
                    u = t;
                }
            }
        }
        uint4 o[2];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w[i] = bf16x2(x[p][2 * i], x[p][2 * i + 1]);
            }
            o[p] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        const bool live = h < heads;
        if (kind == 0) {
            if (live) {
                uint4 *dst = reinterpret_cast<uint4 *>(a.q_out + ((int64_t)tok * heads + h) * D);
                dst[at.p0] = o[0];
                dst[at.p1] = o[1];
            }
        } else if constexpr (!k4) {
            if (live) {
                const int64_t line = ((int64_t)(slot / kPageSize) * heads + h) * kPageSize + slot % kPageSize;
                uint4 *dst = reinterpret_cast<uint4 *>(kind == 1 ? a.k_pages : a.v_pages) + line * (D / 8);
                dst[at.p0] = o[0];
                dst[at.p1] = o[1];
            }
        } else {
            float m[2];
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const uint32_t w[4] = {o[p].x, o[p].y, o[p].z, o[p].w};
                m[p] = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 v = bf16x2_to_float2(w[i] & 0x7fff7fffu);
                    m[p] = kv4::max_nan(m[p], kv4::max_nan(v.x, v.y));
                }
            }
            at.block_max(m[0], m[1]);
            using P = kv4::Page<D>;
            const float g = kind == 1 ? a.k_scale : a.v_scale, six = kind == 1 ? a.k_six : a.v_six;
            uint8_t *page = (kind == 1 ? a.k_pages : a.v_pages) + ((int64_t)(slot / kPageSize) * heads + h) * P::kBytes;
            const int line = slot % kPageSize;
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const int piece = p == 0 ? at.p0 : at.p1;
                const uint32_t w[4] = {o[p].x, o[p].y, o[p].z, o[p].w};
                float y[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 v = bf16x2_to_float2(w[i]);
                    y[2 * i] = v.x;
                    y[2 * i + 1] = v.y;
                }
                const uint32_t s = kv4::scale_of(m[p], six);
                const uint32_t codes = kv4::pack8(y, m[p], __fmul_rn(kv4::scale_value(s), g));
                if (live) {
                    *reinterpret_cast<uint32_t *>(page + line * P::kRow + piece * 4) = codes;
                    if ((piece & 1) == 0)
                        page[P::kScales + line * P::kScaleRow + (piece >> 1)] = (uint8_t)s;
                }
            }
        }
    }
}

// Blocks a thread has in flight.  6007 pages of 8 heads of 128 (504 MB, 74 us at
// the measured copy rate): 77.9 us, at 1 block 79.9; with two 16-byte stores in
// place of one of 32 bytes, which leaves half sectors to the L2, 88.1 and more.
constexpr int kUnpack = 4, kUnpackThreads = 256;

struct UnpackArgs {
    const uint8_t *k4, *v4;
    const int32_t *page_id;
    uint4 *k_pages, *v_pages;
    float k_scale, v_scale;
    int32_t num_listed, num_pages, num_kv_heads;
};

// A thread a block of 16 elements: 8 bytes of codes and a scale in, 32 bytes
// out; a CTA's threads go over one page's heads, K and V by blockIdx.y.
template <int D>
__global__ void __launch_bounds__(kUnpackThreads) unpack4_kernel(UnpackArgs a)
{
    using P = kv4::Page<D>;
    const int page = a.page_id[blockIdx.x];
    if ((uint32_t)page >= (uint32_t)a.num_pages)
        return;
    const bool is_v = blockIdx.y != 0;
    const float g = is_v ? a.v_scale : a.k_scale;
    const uint8_t *src = (is_v ? a.v4 : a.k4) + (int64_t)page * a.num_kv_heads * P::kBytes;
    uint4 *dst = (is_v ? a.v_pages : a.k_pages) + (int64_t)blockIdx.x * a.num_kv_heads * (kPageSize * D / 8);
    const int blocks = a.num_kv_heads * D;
    for (int b0 = threadIdx.x; b0 < blocks; b0 += kUnpack * kUnpackThreads) {
        uint2 w[kUnpack];
        uint32_t s[kUnpack];
#pragma unroll
        for (int u = 0; u < kUnpack; ++u) {
            const int b = b0 + u * kUnpackThreads;
            if (b < blocks) {
                const uint8_t *head = src + (int64_t)(b / D) * P::kBytes;
                w[u] = __ldcs(reinterpret_cast<const uint2 *>(head) + b % D);
                s[u] = __ldcs(head + P::kScales + b % D);
            }
        }
#pragma unroll
        for (int u = 0; u < kUnpack; ++u) {
            const int b = b0 + u * kUnpackThreads;
            if (b >= blocks)
                break;
            const uint32_t s2 = kv4::scales2(s[u] | s[u] << 8);
            uint32_t h0[4], h1[4], o[8];
            kv4::unpack8(w[u].x, h0);
            kv4::unpack8(w[u].y, h1);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t t = kv4::hmul2(k < 4 ? h0[k & 3] : h1[k & 3], s2);
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&t));
                o[k] = bf16x2(f.x * g, f.y * g);
            }
            asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst + 2 * b), "r"(o[0]), "r"(o[1]),
                         "r"(o[2]), "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
                         : "memory");
        }
    }
}

template <typename Args>
int launch(void (*kernel)(Args), dim3 grid, int threads, cudaStream_t st, const Args &a)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = st;
    return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess ? DEFT_OK : DEFT_ECUDA;
}

template <int D, bool kF32, bool k4, bool kWhole>
int launch_qkv(QkvArgs a, cudaStream_t st)
{
    constexpr int kRound = Shape<kF32>::kHeads * (32 / (D / 16));   // heads a warp takes
    a.q_tasks = (a.num_q_heads + kRound - 1) / kRound;
    a.kv_tasks = (a.num_kv_heads + kRound - 1) / kRound;
    const int64_t tasks = (int64_t)a.num_tokens * (a.q_tasks + 2 * a.kv_tasks);
    if (tasks > INT32_MAX)
        return DEFT_EUNSUPPORTED;
    return launch(qkv_kernel<D, kF32, k4, kWhole>, dim3((unsigned)((tasks + kWarps - 1) / kWarps)), kThreads, st, a);
}

template <int D, bool k4>
int pick_qkv(const QkvArgs &a, bool f32, cudaStream_t st)
{
    // (With the rotation's place known: 32768 tokens 162 -> 154 us, 16384 into
    // 4 bits and back 116 -> 106 us, when it was added.)
    if (a.split && a.half == D / 16)
        return f32 ? launch_qkv<D, true, k4, true>(a, st) : launch_qkv<D, false, k4, true>(a, st);
    return f32 ? launch_qkv<D, true, k4, false>(a, st) : launch_qkv<D, false, k4, false>(a, st);
}

bool good_scale(float g)
{
    return g >= 0x1p-60f && g <= 0x1p60f;
}

// The argument checks of both append calls; fills `a` but for the pools.
int check_qkv(const void *q, const void *k, const void *v, int32_t in_dtype, int64_t q_stride, int64_t k_stride,
              int64_t v_stride, const int32_t *slot, int32_t num_tokens, const deft_qk_turn *turn, void *q_out,
              const void *k_pool, const void *v_pool, int32_t num_pages, int32_t num_q_heads, int32_t num_kv_heads,
              int32_t head_dim, int32_t page_size, QkvArgs &a)
{
    if (num_tokens < 0 || num_pages < 1 || num_kv_heads < 1 || num_q_heads < 0 || !k_pool || !v_pool ||
        k_pool == v_pool || (in_dtype != DEFT_OUT_BF16 && in_dtype != DEFT_OUT_F32))
        return DEFT_EINVAL;
    const deft_qk_turn none{};
    const deft_qk_turn &t = turn ? *turn : none;
    if (t.rot_dim < 0 || t.rot_dim > head_dim || (t.rot_dim > 0 && (!t.cos_sin || t.num_positions < 1)) ||
        (t.interleaved != 0 && t.interleaved != 1) || ((t.q_norm || t.k_norm) && !(t.eps >= 0.f && t.eps <= 1e30f)))
        return DEFT_EINVAL;
    if ((head_dim != 64 && head_dim != 128) || page_size != kPageSize || num_pages > INT32_MAX / kPageSize ||
        t.rot_dim % 16 != 0)
        return DEFT_EUNSUPPORTED;
    const int64_t q_row = (int64_t)num_q_heads * head_dim, kv_row = (int64_t)num_kv_heads * head_dim;
    const int64_t es = in_dtype == DEFT_OUT_F32 ? 4 : 2;
    if (q_row > (1 << 24) || kv_row > (1 << 24))
        return DEFT_EINVAL;
    if ((int64_t)num_tokens * (num_q_heads + 2 * (int64_t)num_kv_heads) > INT32_MAX)
        return DEFT_EUNSUPPORTED;
    if (num_tokens > 0 && (!k || !v || !slot || (t.rot_dim > 0 && !t.position) || (num_q_heads > 0 && (!q || !q_out))))
        return DEFT_EINVAL;
    uintptr_t all = (uintptr_t)k | (uintptr_t)v | (uintptr_t)k_pool | (uintptr_t)v_pool | (uintptr_t)t.q_norm |
                    (uintptr_t)t.k_norm | (uintptr_t)t.cos_sin;
    if (num_q_heads > 0)
        all |= (uintptr_t)q | (uintptr_t)q_out;
    if (all & 15u)
        return DEFT_EINVAL;
    if (num_tokens > 1) {
        if (k_stride < kv_row || v_stride < kv_row || (k_stride * es) % 16 || (v_stride * es) % 16)
            return DEFT_EINVAL;
        if (num_q_heads > 0 && (q_stride < q_row || (q_stride * es) % 16))
            return DEFT_EINVAL;
    }
    // In place only where every row of q_out is the row that was read.
    if (num_q_heads > 0 && q_out == q && (es != 2 || (num_tokens > 1 && q_stride != q_row)))
        return DEFT_EINVAL;
    a = QkvArgs{};
    a.q = q, a.k = k, a.v = v;
    a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride;
    a.slot = slot;
    a.num_tokens = num_tokens, a.num_pages = num_pages;
    a.num_q_heads = num_q_heads, a.num_kv_heads = num_kv_heads;
    a.q_out = static_cast<__nv_bfloat16 *>(q_out);
    a.q_norm = t.q_norm, a.k_norm = t.k_norm, a.eps = t.eps;
    a.cos_sin = t.cos_sin, a.position = t.position, a.num_positions = t.num_positions;
    a.half = t.rot_dim / 16, a.split = !t.interleaved;
    return DEFT_OK;
}

}  // namespace
}  // namespace deft

extern "C" {

int deft_qkv_write(const void *q, const void *k, const void *v, int32_t in_dtype, int64_t q_stride, int64_t k_stride,
                   int64_t v_stride, const int32_t *slot, int32_t num_tokens, const deft_qk_turn *turn, void *q_out,
                   void *k_pages, void *v_pages, int32_t num_pages, int32_t num_q_heads, int32_t num_kv_heads,
                   int32_t head_dim, int32_t page_size, void *stream)
{
    using namespace deft;
    QkvArgs a;
    const int rc = check_qkv(q, k, v, in_dtype, q_stride, k_stride, v_stride, slot, num_tokens, turn, q_out, k_pages,
                             v_pages, num_pages, num_q_heads, num_kv_heads, head_dim, page_size, a);
    if (rc != DEFT_OK || num_tokens == 0)
        return rc;
    a.k_pages = static_cast<uint8_t *>(k_pages), a.v_pages = static_cast<uint8_t *>(v_pages);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const bool f32 = in_dtype == DEFT_OUT_F32;
    return head_dim == 128 ? pick_qkv<128, false>(a, f32, st) : pick_qkv<64, false>(a, f32, st);
}

int deft_qkv_write4(const void *q, const void *k, const void *v, int32_t in_dtype, int64_t q_stride, int64_t k_stride,
                    int64_t v_stride, const int32_t *slot, int32_t num_tokens, const deft_qk_turn *turn, void *q_out,
                    void *k4_pages, void *v4_pages, float k_scale, float v_scale, int32_t num_pages,
                    int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t page_size, void *stream)
{
    using namespace deft;
    QkvArgs a;
    if (!good_scale(k_scale) || !good_scale(v_scale))
        return DEFT_EINVAL;
    const int rc = check_qkv(q, k, v, in_dtype, q_stride, k_stride, v_stride, slot, num_tokens, turn, q_out, k4_pages,
                             v4_pages, num_pages, num_q_heads, num_kv_heads, head_dim, page_size, a);
    if (rc != DEFT_OK || num_tokens == 0)
        return rc;
    a.k_pages = static_cast<uint8_t *>(k4_pages), a.v_pages = static_cast<uint8_t *>(v4_pages);
    a.k_scale = k_scale, a.v_scale = v_scale, a.k_six = 6.f * k_scale, a.v_six = 6.f * v_scale;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const bool f32 = in_dtype == DEFT_OUT_F32;
    return head_dim == 128 ? pick_qkv<128, true>(a, f32, st) : pick_qkv<64, true>(a, f32, st);
}

size_t deft_kv4_page_bytes(int32_t head_dim)
{
    return head_dim == 64 || head_dim == 128 ? (size_t)deft::kv4::page_bytes(head_dim) : 0;
}

int deft_kv_unpack4(const void *k4_pages, const void *v4_pages, float k_scale, float v_scale, int32_t num_pages,
                    const int32_t *page_id, int32_t num_listed, void *k_pages, void *v_pages, int32_t num_kv_heads,
                    int32_t head_dim, int32_t page_size, void *stream)
{
    using namespace deft;
    if (!k4_pages || !v4_pages || num_pages < 1 || num_listed < 0 || num_kv_heads < 1 || num_kv_heads > (1 << 18) ||
        !good_scale(k_scale) || !good_scale(v_scale))
        return DEFT_EINVAL;
    if ((head_dim != 64 && head_dim != 128) || page_size != kPageSize)
        return DEFT_EUNSUPPORTED;
    if (num_listed == 0)
        return DEFT_OK;
    if (!page_id || !k_pages || !v_pages || k_pages == v_pages || k_pages == k4_pages || k_pages == v4_pages ||
        v_pages == k4_pages || v_pages == v4_pages ||
        (((uintptr_t)k4_pages | (uintptr_t)v4_pages) & 15u) || (((uintptr_t)k_pages | (uintptr_t)v_pages) & 31u))
        return DEFT_EINVAL;
    UnpackArgs a{static_cast<const uint8_t *>(k4_pages), static_cast<const uint8_t *>(v4_pages), page_id,
                 static_cast<uint4 *>(k_pages), static_cast<uint4 *>(v_pages), k_scale, v_scale,
                 num_listed, num_pages, num_kv_heads};
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const dim3 grid((unsigned)num_listed, 2);
    return head_dim == 128 ? launch(unpack4_kernel<128>, grid, kUnpackThreads, st, a) : launch(unpack4_kernel<64>, grid, kUnpackThreads, st, a);
}

}  // extern "C"
