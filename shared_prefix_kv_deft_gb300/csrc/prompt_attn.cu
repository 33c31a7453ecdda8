// prompt_attn.cu -- attention of whole prompts over the paged cache on
// tcgen05 tensor cores (deft_prompt_attn), head_dim 64 and 128.
//
// Formulation: query rows on the MMA's M dimension, KV tokens on N in tiles
// of 128 (eight pages of the path, whichever nodes they belong to):
//     S[128 rows x 128 tok]  = Q . K_tile^T          (TMEM, fp32)
//     O[128 rows x d]       += P . V_tile            (TMEM, fp32; P bf16 in TMEM)
// A row is a (token, head of the group) pair, token-major, so the heads that
// share a KV head share its tiles.  A CTA works on two row tiles, A and B:
// while the softmax of one runs on its warpgroup, the tensor core works for
// the other.  S of a tile and its P share 128 TMEM columns (P replaces the
// S it came from), and PV(t) is issued before S(t + 1), so the tensor core's
// program order protects both: 2 x 128 columns of S / P and 2 x d of O fill
// the 512 TMEM columns at d = 128.
//
// Warp-collective instructions (.sync.aligned: TMEM loads and stores, the
// register split, TMEM's release) and named barriers want all 32 lanes at
// the same instruction.  What only some lanes do before one of them (an
// arrival, the stores of a partly filled tile, a box's store) is therefore
// one predicated instruction, or comes ahead of a vote or a __syncwarp(), so
// that the lanes' meeting does not hang on where the compiler joins a branch.
// (__syncwarp() at each of these places: few-shot prefill 452.6 us, 8192
// tokens 340.9 us; so 449.0 and 339.4 us.)
//
// A softmax thread owns one row: no exchange between threads.  The running
// maximum is stale: it is raised, and O and the sum rescaled, only when a
// logit exceeds it by 2^8 (base 2), decided per warp; the sum is fp32 over
// the unrounded probabilities.  P is rounded to bf16, the type of V (one MMA
// has one operand type): half a step of 2^-8 on each probability, of the
// size of the bf16 output's own rounding.
//
// Masks.  Only the pages that are partial, past the range or hold own tokens
// past a row's position are masked (at d 64: the tiles that hold such a page);
// a tile's description (page counts and positions, a bit a page for each
// tile's mask) travels with its K and V.  V rows of slots past a node's last
// token are zeroed in shared memory before the product (their P is 0, which
// must not meet a NaN), K's need not be: their logits are replaced.
//
// Bound: at 256 rows a KV tile costs 2 x 2 x 256 x 128 x d flop, 2048 clocks
// of the tensor core at d = 128, against 256 x 128 exponentials (1024 clocks
// of the special-function units) and, as shared-memory reads (Q and K for S,
// V for PV) and TMA writes, about 2048 clocks of shared-memory bandwidth.
// Measured: a tile step of about 2600 clocks, the tensor pipe 70% active; an
// 8192-token prompt of 32/8 heads, d 128, 339 us (1.62 PFLOP/s), 32768
// tokens 5.0 ms (1.75 PFLOP/s) until the power cap sets in (5.2-5.5 ms back
// to back); d 64, where the softmax bounds it, 267 us (1.0 PFLOP/s).  Short
// prompts pay about 4 us a unit for its end and the next one's start.
//
// What the shape of the code is worth (one change each, same box, each
// measured on the kernel of its time):
//   - One elected thread issues all MMAs, for both tiles.  With the warp
//     voting and re-converging around its waits the 32768-token prompt took
//     7.9 ms instead of 5.9; with warp-uniform code and an election around
//     each group 6.6.
//   - A thread that has committed MMAs gets past its next barrier only when
//     they have ended.  So a step has one barrier for K and V together, the
//     stage is freed by the softmax thread that sees the step's last S, and
//     the issuer commits twice a step: 5.9 -> 5.2 ms.
//   - The CTA's tiles are one sequence across its units, walked by one copy
//     of the issuing code, and the units' records are read a unit ahead:
//     what runs once a unit comes from a cold instruction cache (reasoning
//     tree's prefill, 22 units a CTA: 389 -> 286 us).
//   - V's empty rows are zeroed by a warp of its own: done by the producer,
//     no copy went out until V had landed (reasoning tree 266 -> 261 us).
//   - Slower or equal: P handed over when three quarters of it are written
//     (5.7 -> 6.1 ms), exponentials begun before the tile's maximum is known
//     (5.9 ms, registers), an issuer a tile (equal; in turns 5.7 ms), an
//     output warpgroup of its own (5.2-5.4 ms: 512 threads leave the softmax
//     192 registers), output held back until the next unit's first P (5.3
//     ms), three S buffers at d 64 (270 -> 287 us for 8192 tokens); masks
//     written into S in TMEM by a short loop, or a branch a page (few-shot
//     438 -> 472 us, registers), or their bits made while S is on its way
//     (equal).
//
// Roles (12 warps): warps 0-3 and 4-7 softmax and output of tiles A and B
// (216 registers a thread), warp 8 the TMA producer (a lane a page), warp 9
// the MMA issuer, warp 10 zeroes the empty rows of V; these and warp 11 run
// with 72 registers.  Every hand-off is an mbarrier, every wait is bounded; a
// CTA whose wait runs out fills its rows with NaN, records the code, waits
// for its copies and MMAs, frees TMEM and returns.
#include <atomic>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "common.cuh"
#include "prompt_internal.h"
#include "tcgen05.cuh"

namespace deft {
namespace {

constexpr int kThreads = 384;
constexpr uint32_t kRegsSoftmax = 216, kRegsOther = 72;
static_assert(2 * 128 * kRegsSoftmax + 128 * kRegsOther == kThreads * 168, "register split");
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kHalf = 128 * 128;   // 128 rows x 64 dims, bf16, 128-byte swizzled
constexpr int kMetaSlots = 8;
constexpr int kMetaInts = 12;           // 8 pages, flags
constexpr float kRescale = 8.f;         // base-2 logits a row may exceed its running maximum by

// flags of a tile's description, a bit a page: tile A's mask, tile B's, V rows
// past the count to be zeroed
constexpr int kMaskShift = 8, kFixShift = 16;

template <int D>
struct Smem {
    static constexpr uint32_t tile = (D / 64) * kHalf;       // one 128 x D operand
    static constexpr int stages = D == 128 ? 2 : 4;          // pairs: K of a tile and V of the tile before
    static constexpr uint32_t group = D * 16;                // 8 tokens x D dims
    static constexpr uint32_t q_off = 0;                     // [2]: [d half][128 rows][128 B]
    static constexpr uint32_t kv_off = 2 * tile;             // [stages][K, V]: [16 groups of 8 tokens][d half][8 tokens][128 B]
    static constexpr uint32_t out_off = kv_off + stages * 2 * tile;   // [2]: [128 rows][128 B] of output, swizzled
    static constexpr uint32_t meta_off = out_off + 2 * kHalf;
    static constexpr int fixes = stages + 1;                 // requests to zero rows of V
    static constexpr uint32_t fix_off = meta_off + kMetaSlots * kMetaInts * 4;
    static constexpr uint32_t bar_off = fix_off + ((fixes * kMetaInts * 4 + 7) & ~7);
    static constexpr int num_bars = 3 * stages + 11 + fixes;
    static constexpr uint32_t misc_off = bar_off + num_bars * 8;   // TMEM base, error
    static constexpr uint32_t total = misc_off + 16;
    static_assert(total <= 227 * 1024, "shared memory of one CTA");
};

struct PromptMaps {
    CUtensorMap q, k1, v1, k8, v8, out;
};

// D[tmem] (+)= A[tmem] . B[smem]
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate)
{
    asm volatile(
        "{\n.reg .pred p;\n"
        "setp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 32 columns of this thread's lane, not yet waited for.
__device__ __forceinline__ void tmem_ld32_issue(uint32_t taddr, uint32_t *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
// Waits for this thread's TMEM loads; the operands tie the loaded registers
// to the wait.
__device__ __forceinline__ void tmem_ld_wait(uint32_t *r)
{
    asm volatile("tcgen05.wait::ld.sync.aligned;\n"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                   "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}
// 16 columns of this thread's lane, not waited for.
__device__ __forceinline__ void tmem_st16_issue(uint32_t taddr, const uint32_t *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait()
{
    asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void *tmap, int c0, int c1, int c2, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void st_shared16(uint32_t dst, const uint32_t *r)
{
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(dst), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}
// 3-D box shared -> global by the thread with `on` (predicated, no branch),
// and the waits for its source to have been read / for everything to be
// written.
__device__ __forceinline__ void tma_store_3d(bool on, const void *tmap, uint32_t src, int c0, int c1, int c2)
{
    asm volatile(
        "{\n.reg .pred p;\n"
        "setp.ne.u32 p, %5, 0;\n"
        "@p cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];\n"
        "@p cp.async.bulk.commit_group;\n}\n" ::"l"(reinterpret_cast<uint64_t>(tmap)),
        "r"(src), "r"(c0), "r"(c1), "r"(c2), "r"((uint32_t)on)
        : "memory");
}
__device__ __forceinline__ void bulk_wait_read()
{
    asm volatile("cp.async.bulk.wait_group.read 0;\n" ::: "memory");
}
__device__ __forceinline__ void bulk_wait_all()
{
    asm volatile("cp.async.bulk.wait_group 0;\n" ::: "memory");
}

// 32 bytes to global memory, a whole sector a lane, by the lanes with `on`:
// one predicated instruction, no branch.
__device__ __forceinline__ void store32(bool on, void *dst, const uint32_t *r)
{
    asm volatile(
        "{\n.reg .pred p;\n"
        "setp.ne.u32 p, %9, 0;\n"
        "@p st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n}\n" ::"l"(dst),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"((uint32_t)on)
        : "memory");
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile(
        "{\n.reg .pred p;\n"
        "elect.sync _|p, 0xffffffff;\n"
        "selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ PromptItem load_item(const PromptItem *p)
{
    union {
        int4 v[3];
        PromptItem it;
    } u;
    const int4 *s = reinterpret_cast<const int4 *>(p);
    u.v[0] = __ldg(s);
    u.v[1] = __ldg(s + 1);
    u.v[2] = __ldg(s + 2);
    return u.it;
}

// Tokens of page entry `e` (count, own flag, page of the node) that a row at
// position `pos` of its node attends: 0..16.
__device__ __forceinline__ int attended(int32_t e, int pos)
{
    const int cnt = e & 31;
    return (e & 32) ? min(cnt, max(0, pos + 1 - (e >> 6) * kPageSize)) : cnt;
}

// Rows of the query tiles that no box fills (a group that does not divide
// 128): zeros, so that what lay there cannot ask for rescales.  One warp.
template <int D>
__device__ __noinline__ void zero_rows(uint8_t *q, int first)
{
    constexpr int kPieces = 2 * (D / 64) * 8;   // of one row: both tiles' halves, 16 bytes each
    for (int x = threadIdx.x & 31; x < (kPromptRows - first) * kPieces; x += 32) {
        const int row = first + x / kPieces, rest = x % kPieces;
        *reinterpret_cast<uint4 *>(q + (rest >> 3) * kHalf + row * 128 + (rest & 7) * 16) = make_uint4(0, 0, 0, 0);
    }
    tc::fence_proxy_async();
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) prompt_kernel(PromptArgs a, const __grid_constant__ PromptMaps maps)
{
    using L = Smem<D>;
    constexpr int NST = L::stages;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    volatile int32_t *meta = reinterpret_cast<volatile int32_t *>(smem + L::meta_off);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::misc_off);
    volatile int *err = reinterpret_cast<volatile int *>(smem + L::misc_off + 4);
    auto bar = [&](int i) { return base + L::bar_off + 8u * (uint32_t)i; };
    constexpr int kFull = 0, kEmpty = NST, kQFull = 2 * NST, kQEmpty = kQFull + 2, kSFull = kQFull + 4,
                  kPFull = kQFull + 6, kOFull = kQFull + 8, kDrain = kQFull + 10, kVLand = kQFull + 11, kFix = kVLand + NST;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = a.gqa_group, Hkv = a.num_kv_heads;
    const int tile_tok = kPromptRows / G;

    // ---------------- set-up ----------------
    // The launch may start while the stream's earlier work ends: nothing in
    // global memory is read or written before the grid-dependency wait (the
    // plan's copy may be among that work).
    if (tid == 0) {
        grid_dep_launch();
        for (int i = 0; i < NST; ++i) {
            tc::mbar_init(bar(kFull + i), 2);   // the copies' bytes, and V's empty rows are zeros
            tc::mbar_init(bar(kEmpty + i), 1);
        }
        for (int w = 0; w < 2; ++w) {
            tc::mbar_init(bar(kQFull + w), 1);
            tc::mbar_init(bar(kQEmpty + w), 1);
            tc::mbar_init(bar(kSFull + w), 1);
            tc::mbar_init(bar(kPFull + w), 4);   // one arrival a softmax warp
            tc::mbar_init(bar(kOFull + w), 1);
        }
        tc::mbar_init(bar(kDrain), 1);
        for (int i = 0; i < NST; ++i)
            tc::mbar_init(bar(kVLand + i), 1);
        for (int i = 0; i < L::fixes; ++i)
            tc::mbar_init(bar(kFix + i), 1);
        *err = 0;
        tc::fence_mbar_init();
    }
    if (warp == 8) {
        if (lane == 0) {
            tc::prefetch_tmap(&maps.q);
            tc::prefetch_tmap(&maps.k1);
            tc::prefetch_tmap(&maps.v1);
            tc::prefetch_tmap(&maps.k8);
            tc::prefetch_tmap(&maps.v8);
        }
    }
    if (warp == 10)
        zero_rows<D>(smem + L::q_off, tile_tok * G);
    if (warp == 9) {
        tc::tmem_alloc(smem_u32(tmem_slot), kTmemCols);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    if (tid == 0 && (base & 1023u) != 0)
        *err = 300;   // the swizzled operands need their atoms aligned
    grid_dep_wait();
    const int u0 = a.plan.cta_off[blockIdx.x], u1 = a.plan.cta_off[blockIdx.x + 1];
    // A bounded wait of a whole warp; the first one that runs out leaves its
    // code.  A warpgroup may sit out many units (tile B of units that have
    // none): its first wait of a unit goes on for 64 limits, unless another
    // role has failed; the warp that zeroes rows of V may have nothing to do
    // in the whole launch.
    // A lane given a barrier `then` arrives there as soon as its own wait has
    // ended, ahead of the vote in which the lanes meet again.
    auto wait = [&](int b, uint32_t parity, int code, int limits = 1, int then = -1) -> bool {
        for (int i = 0; i < limits; ++i) {
            const bool seen = tc::mbar_wait(bar(b), parity);
            if (seen && then >= 0) {
                tc::mbar_arrive(bar(then));
                then = -1;
            }
            if (__all_sync(0xffffffffu, seen))
                return true;
            if (__any_sync(0xffffffffu, *err != 0))
                return false;
        }
        *err = code;
        return false;
    };

    if (warp >= 8) {
        __syncwarp();
        tc::setmaxnreg_dec<kRegsOther>();
        if (warp == 8) {
            // ---------------- TMA producer ----------------
            const uint64_t pol = tc::l2_kv_policy(false);
            uint32_t nq[2] = {0, 0};      // Q tiles so far
            bool ok = true;
            // The unit ahead: lane i < 8 follows page i of every tile: its
            // node, that node's record and first page, the page of the node.
            int unit = u0 < u1 ? a.plan.cta_unit[u0] : 0, after = 0, h = 0, node = 0, pg = 0, first = 0, n = 0, tn = 0;
            int2 rec = make_int2(-1, 0);
            PromptItem it{};
            auto enter = [&]() {
                while (node != it.node) {
                    const int pages = (rec.y + kPageSize - 1) / kPageSize;
                    if (pg < pages)
                        break;
                    pg -= pages;
                    node = rec.x < 0 ? it.node : rec.x;
                    rec = __ldg(a.plan.nodes + node);
                    first = a.node_page_off[node];
                }
            };
            // This tile's pages, resolved one tile ahead (across units too),
            // so that the page table's latency is off the ring's path.
            int cnt = 0, page = 0;
            int32_t entry = 0, flags = 0;
            bool run8 = false;
            auto resolve = [&]() {
                const bool held = tn * kPromptTilePages + (lane & 7) < it.pages;
                bool mask_a = true, mask_b = true;
                cnt = 0;
                entry = 0;
                page = a.num_pages;   // past the range: a box out of the pool reads zeros
                if (held) {
                    const bool own = node == it.node;
                    page = __ldg(a.page_id + first + pg);
                    cnt = min(kPageSize, rec.y - pg * kPageSize);
                    entry = cnt | (own ? 32 : 0) | (pg << 6);
                    const int last = pg * kPageSize + kPageSize - 1;
                    mask_a = cnt < kPageSize || (own && last > it.pos0);
                    mask_b = cnt < kPageSize || (own && last > it.pos0 + it.tok_a);
                }
                flags = (int32_t)((__ballot_sync(0xffffffffu, mask_a) & 255u) |
                                  (__ballot_sync(0xffffffffu, mask_b) & 255u) << kMaskShift |
                                  (__ballot_sync(0xffffffffu, cnt > 0 && cnt < kPageSize) & 255u) << kFixShift);
                const int page0 = __shfl_sync(0xffffffffu, page, 0);
                run8 = __all_sync(0xffffffffu, held && page == page0 + (lane & 7));
                pg += kPromptTilePages;
                enter();
                ++tn;
            };
            auto open_unit = [&](int u) {
                it = load_item(a.plan.items + unit / Hkv);
                h = unit % Hkv;
                after = u + 1 < u1 ? __ldg(a.plan.cta_unit + u + 1) : 0;
                n = max(it.tiles_a, it.tiles_b);
                tn = 0;
                node = it.start_node;
                pg = it.start_page + (lane & 7);
                rec = __ldg(a.plan.nodes + node);
                first = a.node_page_off[node];
                enter();
                resolve();
            };
            if (u0 < u1)
                open_unit(u0);
            // A step loads K of the next tile and, beside it, V of the tile
            // before: what the MMA issuer needs of one step.
            bool v_run8 = false;
            int v_page = 0, v_cnt = 0, v_h = 0;
            uint32_t v_fix = 0, step = 0, fixed = 0;   // fixed: requests to warp 10 so far
            volatile int32_t *fix = reinterpret_cast<volatile int32_t *>(smem + L::fix_off);
            auto ask = [&](int32_t what) {
                const int x = (int)(fixed % L::fixes);
                if (lane < 8)
                    fix[x * kMetaInts + lane] = v_cnt;
                if (lane == 0)
                    fix[x * kMetaInts + 8] = what;
                __syncwarp();
                if (lane == 0)
                    tc::mbar_arrive(bar(kFix + x));
                ++fixed;
            };
            auto copy = [&](uint32_t dst, const CUtensorMap *one, const CUtensorMap *eight, bool whole, int pg0, int head, int b) {
                if (whole) {
                    if (lane == 0)
                        tc::tma_load_5d(dst, eight, 0, 0, 0, 2 * head, pg0, bar(b), pol);
                } else if (lane < 8) {
                    tc::tma_load_5d(dst + (uint32_t)lane * 2 * L::group, one, 0, 0, 0, 2 * head, pg0, bar(b), pol);
                }
            };
            for (int u = u0; ok; ++step) {
                const bool more = u < u1;
                const int t = tn - 1;
                const int s = (int)(step % NST);
                if (step >= NST && !(ok = wait(kEmpty + s, (step / NST - 1) & 1, 301)))
                    break;
                const uint32_t dst = base + L::kv_off + (uint32_t)s * 2 * L::tile;
                if (more) {
                    // The slot's last reader is done: its tile's P, which
                    // the stage just freed came after.
                    const int ms = (int)(step % kMetaSlots) * kMetaInts;
                    if (lane < 8)
                        meta[ms + lane] = entry;
                    if (lane == 0)
                        meta[ms + 8] = flags;
                    __syncwarp();
                }
                // V with partial pages lands on a barrier of its own: warp 10
                // zeroes its empty rows before the step is handed over, and
                // the copies of the steps behind go out meanwhile.
                if (lane == 0) {
                    tc::mbar_arrive_expect_tx(bar(kFull + s), (more ? L::tile : 0) + (step > 0 && !v_fix ? L::tile : 0));
                    if (v_fix)
                        tc::mbar_arrive_expect_tx(bar(kVLand + s), L::tile);
                    else
                        tc::mbar_arrive(bar(kFull + s));
                }
                __syncwarp();
                if (more)
                    copy(dst, &maps.k1, &maps.k8, run8, page, h, kFull + s);
                if (step > 0)
                    copy(dst + L::tile, &maps.v1, &maps.v8, v_run8, v_page, v_h, (v_fix ? kVLand : kFull) + s);
                if (v_fix)
                    ask((int32_t)v_fix | s << 8);
                if (more && t == 0) {
                    // The unit's rows, once the unit before has made its last
                    // S from the buffer.
                    for (int w = 0; w < 2 && ok; ++w) {
                        if ((w ? it.tiles_b : it.tiles_a) == 0)
                            continue;
                        if (nq[w] && !(ok = wait(kQEmpty + w, (nq[w] - 1) & 1, 302)))
                            break;
                        ++nq[w];
                        if (lane == 0) {
                            tc::mbar_arrive_expect_tx(bar(kQFull + w), (uint32_t)(tile_tok * G) * D * 2);
                            for (int x = 0; x < D / 64; ++x)
                                tma_load_3d(base + L::q_off + (uint32_t)w * L::tile + x * kHalf, &maps.q, 64 * x, h * G,
                                            it.row0 + (w ? it.tok_a : 0), bar(kQFull + w));
                        }
                    }
                    if (!ok) {
                        ++step;
                        break;
                    }
                }
                if (!more) {
                    ++step;
                    break;
                }
                // The next tile, while this one's copies are in flight.
                v_run8 = run8;
                v_page = page;
                v_cnt = cnt;
                v_h = h;
                v_fix = ((uint32_t)flags >> kFixShift) & 255u;
                if (tn < n) {
                    resolve();
                } else if (++u < u1) {
                    unit = after;
                    open_unit(u);
                }
            }
            if (!ok) {
                // Every copy that went out lands before the CTA ends.
                for (uint32_t i = step > (uint32_t)NST ? step - NST : 0; i < step; ++i)
                    tc::mbar_wait(bar(kFull + (int)(i % NST)), (i / NST) & 1);
                for (int w = 0; w < 2; ++w)
                    if (nq[w])
                        tc::mbar_wait(bar(kQFull + w), (nq[w] - 1) & 1);
            }
            ask(-1);
        } else if (warp == 10) {
            // ---------------- empty rows of V ----------------
            // V rows past a node's last token: the page holds anything there,
            // and their P of 0 must not meet a NaN.  A request's slot is free
            // again when its step's stage is, and there is one slot more than
            // stages for the last request, which ends the loop.
            volatile int32_t *fix = reinterpret_cast<volatile int32_t *>(smem + L::fix_off);
            uint32_t land = 0;   // parity of V's own barriers, by stage
            for (uint32_t i = 0;; ++i) {
                const int x = (int)(i % L::fixes);
                if (!wait(kFix + x, (i / L::fixes) & 1, 304, 4096))
                    break;
                const int32_t what = fix[x * kMetaInts + 8];
                if (what < 0)
                    break;
                const int s = what >> 8, cnt = fix[x * kMetaInts + (lane & 7)];
                if (!wait(kVLand + s, (land >> s) & 1, 303))
                    break;
                land ^= 1u << s;
                for (uint32_t pages = (uint32_t)what & 255u; pages; pages &= pages - 1) {
                    const int j = __ffs((int)pages) - 1, used = __shfl_sync(0xffffffffu, cnt, j);
                    uint8_t *at = smem + L::kv_off + (uint32_t)s * 2 * L::tile + L::tile + (uint32_t)j * 2 * L::group;
                    // 16 rows of D / 64 x 128 B, in 16-byte pieces
                    for (int y = lane; y < (kPageSize - used) * (D / 64) * 8; y += 32) {
                        const int row = used + y / ((D / 64) * 8), rest = y % ((D / 64) * 8);
                        *reinterpret_cast<uint4 *>(at + (row >> 3) * L::group + (rest >> 3) * 1024 + (row & 7) * 128 +
                                                   (rest & 7) * 16) = make_uint4(0, 0, 0, 0);
                    }
                }
                tc::fence_proxy_async();
                __syncwarp();
                if (lane == 0)
                    tc::mbar_arrive(bar(kFull + s));
            }
        } else if (warp == 9) {
            // ---------------- MMA issue ----------------
            // One thread runs the whole loop: the tensor core idles while
            // its issuer does anything else, so there is no vote, no
            // reconvergence and no shared work in it.
            if (elect_one()) {
                constexpr uint32_t idesc_s = tc::idesc_bf16(128, 128, 0, 0);
                constexpr uint32_t idesc_o = tc::idesc_bf16(128, D, 0, 1);
                const uint64_t dq0 = tc::smem_desc(base + L::q_off, 16, 1024);
                // K: K-major, 8-token groups L::group apart; V: MN-major, its
                // d halves 1 KB apart and its 8-token groups L::group apart.
                const uint64_t dk0 = tc::smem_desc(base + L::kv_off, 16, L::group);
                const uint64_t dv0 = tc::smem_desc(base + L::kv_off + L::tile, 1024, L::group);
                bool ok = true;
                auto wait1 = [&](int b, uint32_t parity, int code) {
                    if (!tc::mbar_wait(bar(b), parity)) {
                        if (!*err)
                            *err = code;
                        ok = false;
                    }
                    return ok;
                };
                // The CTA's KV tiles are one sequence, across units: a step
                // makes PV of the tile in hand and S of the one after, for A,
                // then for B.  One copy of the code serves both and the units'
                // ends, which would otherwise run from a cold instruction cache.
                uint32_t qp = 0, pp = 0;           // parities of Q full and P full, bit w
                uint32_t st = 0, ph = 0;           // the step's stage and its parity
                int u = u0, t = 0, n = 0, na = 0, nb = 0;   // tile t of n; A has na of them, B nb
                // The next unit is read in two steps a tile apart: nothing
                // here waits for a load just issued.
                int next_unit = u0 < u1 ? __ldg(a.plan.cta_unit + u0) : 0, next_a = 0, next_b = 0;
                auto look = [&]() {
                    const PromptItem *it = a.plan.items + next_unit / Hkv;
                    next_a = __ldg(&it->tiles_a);
                    next_b = __ldg(&it->tiles_b);
                };
                look();
                while (ok) {
                    // the tile after
                    int tx = t + 1, xa = na, xb = nb;
                    const bool same = tx < n;
                    if (!same) {
                        tx = 0;
                        xa = u < u1 ? next_a : 0;
                        xb = u < u1 ? next_b : 0;
                    }
                    if (!wait1(kFull + st, ph, 313))
                        break;
                    const uint32_t at = (st * 2 * L::tile) >> 4;
#pragma unroll 1
                    for (int w = 0; w < 2; ++w) {
                        const uint32_t ts = tmem + w * 128;
                        const int now = w ? nb : na, nxt = w ? xb : xa;
                        if (t < now) {
                            if (!wait1(kPFull + w, (pp >> w) & 1, 314))
                                break;
                            pp ^= 1u << w;
                            tc::fence_after_sync();
#pragma unroll
                            for (int s = 0; s < 8; ++s)
                                mma_ts(ts + 256, ts + s * 8, dv0 + (uint64_t)(at + ((s * 2 * L::group) >> 4)), idesc_o,
                                       (t > 0 || s > 0) ? 1u : 0u);
                            if (t + 1 == now)
                                tc::mma_commit(bar(kOFull + w));
                        }
                        if (tx < nxt) {
                            if (tx == 0) {
                                if (!wait1(kQFull + w, (qp >> w) & 1, 312))
                                    break;
                                qp ^= 1u << w;
                            }
                            tc::fence_after_sync();
                            const uint64_t dq = dq0 + (uint64_t)((w * L::tile) >> 4);
#pragma unroll
                            for (int s = 0; s < D / 16; ++s)
                                tc::mma_bf16(ts, dq + (uint64_t)(((s >> 2) * kHalf + (s & 3) * 32) >> 4),
                                             dk0 + (uint64_t)(at + (((s >> 2) * 1024 + (s & 3) * 32) >> 4)), idesc_s,
                                             s > 0 ? 1u : 0u);
                            tc::mma_commit(bar(kSFull + w));
                            if (tx + 1 == nxt)
                                tc::mma_commit(bar(kQEmpty + w));
                        }
                    }
                    if (!ok)
                        break;
                    // A unit's first step frees its stage here; the others'
                    // are freed by the softmax of the step's last S.
                    if (!same) {
                        tc::mma_commit(bar(kEmpty + st));
                        if (u == u1)
                            break;
                        na = xa;
                        nb = xb;
                        n = max(na, nb);
                        ++u;
                        if (u < u1)
                            next_unit = __ldg(a.plan.cta_unit + u);
                    }
                    // (a unit of one tile has no later step to do it in)
                    if (tx == 1 || (tx == 0 && n == 1))
                        look();
                    t = tx;
                    st = st + 1 == NST ? 0 : st + 1;
                    ph ^= st == 0;
                }
                // Every MMA and its arrivals end before the CTA does.
                tc::mma_commit(bar(kDrain));
                wait1(kDrain, 0, 316);
            }
            __syncwarp();
        }
    } else {
        __syncwarp();
        tc::setmaxnreg_inc<kRegsSoftmax>();
        // ---------------- softmax and output: one row a thread ----------------
        const int w = warp >> 2, r = tid & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;   // this warp's TMEM lanes
        const uint32_t ts = tmem + lanes + w * 128, to = tmem + lanes + 256 + w * 128;
        const int tok = r / G, head = r - tok * G;
        const float scale = a.scale_log2;
        const f32x2 scale2 = f2_pack(scale, scale);
        uint32_t gt = 0, ns = 0, no = 0;
        bool ok = true;
        // The next unit's record is loaded a unit ahead, its number two.
        int unit = u0 < u1 ? __ldg(a.plan.cta_unit + u0) : 0;
        int next_unit = u0 + 1 < u1 ? __ldg(a.plan.cta_unit + u0 + 1) : unit;
        PromptItem next = load_item(a.plan.items + unit / Hkv);
        for (int u = u0; u < u1 && ok; ++u) {
            const PromptItem it = next;
            const int h = unit % Hkv;
            next = load_item(a.plan.items + next_unit / Hkv);
            unit = next_unit;
            if (u + 2 < u1)
                next_unit = __ldg(a.plan.cta_unit + u + 2);
            const int nt = w ? it.tiles_b : it.tiles_a, before = w ? it.tok_a : 0;
            const int toks = w ? it.tok_b : it.tok_a;
            const bool held = tok < toks;
            const int pos = it.pos0 + before + tok;
            const bool frees = w == (it.tiles_b > 0);
            float m = -INFINITY, l = 0.f;
            for (int t = 0; t < nt; ++t) {
                // S of this tile is made, and what came before it: both
                // operands of the step are free (of its last S, B's if the
                // unit has a B; a unit's first step is freed by the issuer).
                const int free_bar = frees && t > 0 && r == 0 ? kEmpty + (int)((gt + t) % NST) : -1;
                if (!wait(kSFull + w, ns & 1, 321 + w, t == 0 ? 64 : 1, free_bar)) {
                    ok = false;
                    break;
                }
                ++ns;
                tc::fence_after_sync();
                uint32_t sr[128];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    tmem_ld32_issue(ts + 32 * c, sr + 32 * c);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    tmem_ld_wait(sr + 32 * c);
                const int ms = (int)((gt + t) % kMetaSlots) * kMetaInts;
                const int masked = meta[ms + 8] >> (w * kMaskShift) & 255;
                if (masked) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        // Two pages without a mask are passed over at d 128
                        // (reasoning tree 261 -> 254 us); at d 64 the vote
                        // costs more than it saves (trees 112.5 -> 114.5 us).
                        if (D == 128 && !__any_sync(0xffffffffu, masked >> (2 * c) & 3))
                            continue;
                        const uint32_t bits = ((1u << attended(meta[ms + 2 * c], pos)) - 1) |
                                              (((1u << attended(meta[ms + 2 * c + 1], pos)) - 1) << 16);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            sr[32 * c + i] = (bits >> i) & 1 ? sr[32 * c + i] : 0xff800000u;   // -inf
                    }
                }
                float mx0 = -INFINITY, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
                for (int i = 0; i < 128; i += 8) {
                    mx0 = fmaxf(mx0, fmaxf(__uint_as_float(sr[i]), __uint_as_float(sr[i + 1])));
                    mx1 = fmaxf(mx1, fmaxf(__uint_as_float(sr[i + 2]), __uint_as_float(sr[i + 3])));
                    mx2 = fmaxf(mx2, fmaxf(__uint_as_float(sr[i + 4]), __uint_as_float(sr[i + 5])));
                    mx3 = fmaxf(mx3, fmaxf(__uint_as_float(sr[i + 6]), __uint_as_float(sr[i + 7])));
                }
                const float mx = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3)) * scale;
                if (t == 0) {
                    m = mx;
                } else if (__any_sync(0xffffffffu, mx > m + kRescale)) {
                    // PV(t - 1) has ended (S(t) came after it): O may be rescaled here.
                    const float mn = fmaxf(m, mx);
                    const float f = mn == -INFINITY ? 1.f : tc::ex2(m - mn);
                    m = mn;
                    l *= f;
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        tmem_ld32_issue(to + 32 * c, o);
                        tmem_ld_wait(o);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                        tmem_st16_issue(to + 32 * c, o);
                        tmem_st16_issue(to + 32 * c + 16, o + 16);
                    }
                }
                const float neg = m == -INFINITY ? 0.f : -m;
                const f32x2 neg2 = f2_pack(neg, neg);
                f32x2 sum0 = f2_pack(0.f, 0.f), sum1 = sum0;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t pk[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const f32x2 x = f2_fma(f2_pack(__uint_as_float(sr[32 * c + 2 * i]), __uint_as_float(sr[32 * c + 2 * i + 1])),
                                               scale2, neg2);
                        float2 y = f2_unpack(x);
                        y.x = tc::ex2(y.x);
                        y.y = tc::ex2(y.y);
                        if (i & 1)
                            sum1 = f2_add(sum1, f2_pack(y.x, y.y));
                        else
                            sum0 = f2_add(sum0, f2_pack(y.x, y.y));
                        pk[i] = tc::pack_bf16x2(y.x, y.y);
                    }
                    tmem_st16_issue(ts + 16 * c, pk);
                }
                const float2 s2 = f2_unpack(f2_add(sum0, sum1));
                l += s2.x + s2.y;
                tmem_st_wait();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    tc::mbar_arrive(bar(kPFull + w));
            }
            gt += (uint32_t)max(it.tiles_a, it.tiles_b);
            const int rows = (it.tok_a + it.tok_b) * G;
            const size_t orow = (size_t)(it.row0 + before + tok) * a.num_q_heads + h * G + head;
            const size_t slot = (size_t)it.part0 + (size_t)h * rows + before * G + r;
            if (nt > 0) {
                ok = ok && wait(kOFull + w, no & 1, 323 + w);
                // The four warps go on, or end, together; the staging rows
                // are free behind this barrier.
                if ((warp & 3) == 0)
                    bulk_wait_read();
                if (tc::named_sync_or(1 + w, 128, !ok)) {
                    ok = false;
                    break;
                }
                ++no;
                tc::fence_after_sync();
                // l is NaN where a logit is NaN or +inf, 0 where all are -inf
                // (or, in a piece, none is seen: the merge passes over such
                // rows): both reach the output (NaN, 0 x inf) unguarded.
                const float inv = __fdividef(1.f, l);
                const bool f32 = it.part0 >= 0 || a.out_dtype == DEFT_OUT_F32;
                if (!f32 && toks == tile_tok) {
                    // A whole tile in bf16: 64 dims of its rows to shared
                    // memory, and out as one box.  (Written from here, 32
                    // bytes of 32 rows a store, the rows cost the load/store
                    // unit eight times as much: the reasoning tree's prefill
                    // took 276 us instead of 267.)
                    const uint32_t row_s = base + L::out_off + w * kHalf + (uint32_t)r * 128;
#pragma unroll 1
                    for (int c = 0; c < D / 64; ++c) {
                        uint32_t o[64];
                        tmem_ld32_issue(to + 64 * c, o);
                        tmem_ld32_issue(to + 64 * c + 32, o + 32);
                        tmem_ld_wait(o);
                        tmem_ld_wait(o + 32);
                        if (c > 0) {
                            if ((warp & 3) == 0)
                                bulk_wait_read();   // the box before has been read
                            tc::named_sync(1 + w, 128);
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            uint32_t x[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                x[k] = tc::pack_bf16x2(__uint_as_float(o[8 * i + 2 * k]) * inv,
                                                       __uint_as_float(o[8 * i + 2 * k + 1]) * inv);
                            st_shared16(row_s + ((uint32_t)(i ^ (r & 7)) << 4), x);
                        }
                        tc::fence_proxy_async();
                        tc::named_sync(1 + w, 128);
                        tma_store_3d(r == 0, &maps.out, base + L::out_off + w * kHalf, 64 * c, h * G, it.row0 + before);
                    }
                } else {
                    uint8_t *dst = it.part0 >= 0 ? reinterpret_cast<uint8_t *>(a.o_part + slot * D)
                                                 : static_cast<uint8_t *>(a.out) + orow * D * (f32 ? 4 : 2);
                    // One copy of the code for the parts of a row: it runs
                    // once a unit, from a cold instruction cache.
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        tmem_ld32_issue(to + 32 * c, o);
                        tmem_ld_wait(o);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            o[i] = __float_as_uint(__uint_as_float(o[i]) * inv);
                        if (f32) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                store32(held, dst + 128 * c + 32 * i, o + 8 * i);
                        } else {
                            uint32_t x[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                x[i] = tc::pack_bf16x2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]));
                            store32(held, dst + 64 * c, x);
                            store32(held, dst + 64 * c + 32, x + 8);
                        }
                    }
                }
            }
            if (held) {
                // -inf where nothing was seen (m = -inf, l = 0), NaN with l
                const float lse2 = m + __log2f(l);
                if (it.part0 >= 0)
                    a.lse_part[slot] = lse2;
                else
                    a.lse[orow] = lse2 * kLn2;
            }
        }
    }
    if (tid == 0 || tid == 128)
        bulk_wait_all();
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (*err) {
        // A wait ran out: every row of the CTA's units is marked.
        if (tid == 0)
            atomicCAS(a.plan.status, 0u, (uint32_t)*err);
        const float nan = __int_as_float(0x7fc00000);
        for (int u = u0; u < u1; ++u) {
            const int unit = a.plan.cta_unit[u], h = unit % Hkv;
            const PromptItem it = load_item(a.plan.items + unit / Hkv);
            const int rows = (it.tok_a + it.tok_b) * G;
            for (int x = tid; x < rows; x += kThreads) {
                if (it.part0 >= 0) {
                    a.lse_part[(size_t)it.part0 + (size_t)h * rows + x] = nan;
                    continue;
                }
                const size_t orow = (size_t)(it.row0 + x / G) * a.num_q_heads + h * G + x % G;
                a.lse[orow] = nan;
                for (int e = 0; e < D; ++e) {
                    if (a.out_dtype == DEFT_OUT_F32)
                        static_cast<float *>(a.out)[orow * D + e] = nan;
                    else
                        static_cast<__nv_bfloat16 *>(a.out)[orow * D + e] = __float2bfloat16_rn(nan);
                }
            }
        }
    }
    if (warp == 9) {
        __syncwarp();
        tc::tmem_dealloc(tmem, kTmemCols);
    }
}

// ---- host ----
PFN_cuTensorMapEncodeTiled_v12000 encoder()
{
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            ptr = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    }();
    return fn;
}

// A view of the pool [pages][Hkv][16][D], innermost first: 64 dims (one
// 128-byte swizzle row), 8 tokens, the D / 64 parts of a row, 2 Hkv groups of
// 8 tokens and pages; a box holds one page (or eight) of one head and lands
// as [8-token group][part][8 tokens][128 B].
bool pool_map(const void *ptr, const PromptArgs &a, bool run8, CUtensorMap *m)
{
    const cuuint64_t row = (cuuint64_t)a.head_dim * 2;
    const cuuint32_t parts = (cuuint32_t)a.head_dim / 64;
    const cuuint64_t dims[5] = {64, 8, parts, 2 * (cuuint64_t)a.num_kv_heads, (cuuint64_t)a.num_pages};
    const cuuint64_t strides[4] = {row, 128, 8 * row, row * kPageSize * a.num_kv_heads};
    const cuuint32_t box[5] = {64, 8, parts, 2, run8 ? 8u : 1u};
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return encoder()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void *>(ptr), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// q (or out) as [tokens][Hq][D]; a box is a tile's tokens of one group, 64 dims.
bool rows_map(const PromptArgs &a, const void *ptr, int64_t stride, CUtensorMap *m)
{
    const cuuint64_t dims[3] = {(cuuint64_t)a.head_dim, (cuuint64_t)a.num_q_heads, (cuuint64_t)a.num_rows};
    const cuuint64_t strides[2] = {(cuuint64_t)a.head_dim * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)a.gqa_group, (cuuint32_t)(kPromptRows / a.gqa_group)};
    const cuuint32_t estr[3] = {1, 1, 1};
    return encoder()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
int launch_dim(const PromptArgs &a, const PromptMaps &maps, int32_t ctas, cudaStream_t st)
{
    // The shared-memory size is set once a device.
    static std::atomic<uint64_t> set{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return (int)e;
    if (dev >= 64 || !(set.load(std::memory_order_acquire) >> dev & 1)) {
        e = cudaFuncSetAttribute(prompt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Smem<D>::total);
        if (e != cudaSuccess)
            return (int)e;
        if (dev < 64)
            set.fetch_or(1ull << dev, std::memory_order_release);
    }
    return (int)launch_dependent(prompt_kernel<D>, dim3(ctas), dim3(kThreads), Smem<D>::total, st, a, maps);
}

}  // namespace

int launch_prompt(const PromptArgs &a, int32_t ctas, void *stream)
{
    PromptMaps maps;
    if (!encoder() || !rows_map(a, a.q, a.q_stride, &maps.q) ||
        !rows_map(a, a.out, (int64_t)a.num_q_heads * a.head_dim, &maps.out) || !pool_map(a.k_pages, a, false, &maps.k1) ||
        !pool_map(a.v_pages, a, false, &maps.v1) || !pool_map(a.k_pages, a, true, &maps.k8) ||
        !pool_map(a.v_pages, a, true, &maps.v8))
        return (int)cudaErrorInvalidValue;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return a.head_dim == 128 ? launch_dim<128>(a, maps, ctas, st) : launch_dim<64>(a, maps, ctas, st);
}

}  // namespace deft
