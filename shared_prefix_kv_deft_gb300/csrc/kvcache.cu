// kvcache.cu -- filling the paged KV cache: page tables and slot maps built
// on the GPU from node lengths (deft_page_table), and K / V rows written into
// the pages by slot (deft_kv_write).
//
// Page tables.  With P = 16 tokens a page, node n of `len` tokens, `prev` of
// them in the cache already, needs ceil(len / P) pages, keeps the first
// min(ceil(prev / P), pages) of its earlier ones and brings max(0, len -
// prev) new tokens.  Three exclusive sums over the nodes (pages, new tokens,
// pages taken) give node_page_off, tok_off and each node's place in the free
// list; the rest is a copy.  Sums saturate at 2^31 - 1 (saturating addition
// of non-negative numbers is associative, so the scan may), which no
// capacity reaches, so an overflow shows as a capacity exceeded.
//
// The work is a few bytes a page and a token, so a call costs its launch and
// a chain of dependent loads, not bandwidth.  Up to kBlockNodes nodes it is
// one launch: every CTA scans all lengths into shared memory itself (8 KB
// from L2) and fills its share of the pages and their slots, found by binary
// search in the scanned offsets, so a single long node is spread over all
// CTAs as well.  Above that a first launch writes the sums of every block of
// kBlockNodes nodes to the workspace, and each CTA of the second scans the
// block sums and then only the blocks its share touches.  The share is one
// of pages: a thread finds its page's node and number, and half a warp then
// writes that page's new slots, 64 bytes at a time.  (A thread a slot, with
// a search and a table lookup each, took 20.2 us instead of 13.6 for 20000
// nodes with 1.3M tokens.)  256 growing nodes over 27000 pages: 4.5 us.
//
// KV write.  One thread moves 16 bytes of a page row (8 elements of one head
// of one token), several in flight; reads are coalesced over a token's row
// (all heads), writes over one head's row of 128 or 256 bytes.  Bound by
// DRAM bandwidth for prompts (32768 tokens of 8 heads of 128: 38.5 us on the
// device, the 268 MB at the measured copy rate take 39.5), by latency for a
// decode step (256 tokens: 2.6 us).
#include <cstdint>

#include "common.cuh"
#include "deft_internal.h"

namespace deft {
namespace {

// An ordinary launch, with its own status: the thread's last error, which a
// launch by <<<>>> is asked for, may be that of a call before.
template <typename Args, typename... More>
int launch(void (*kernel)(Args, More...), unsigned grid, int threads, cudaStream_t st, const Args &a, More... more)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.stream = st;
    return cudaLaunchKernelEx(&cfg, kernel, a, more...) == cudaSuccess ? DEFT_OK : DEFT_ECUDA;
}

constexpr int kTableThreads = 512;
constexpr int kPerThread = 4;
constexpr int kBlockNodes = kTableThreads * kPerThread;   // nodes scanned at once
constexpr int kMaxBlocks = 512;                           // blocks of one call
constexpr uint32_t kSat = 0x7fffffffu;

// counts[3]
constexpr int32_t kBadLength = DEFT_TABLE_BAD_LENGTH, kBadPrev = DEFT_TABLE_BAD_PREV, kNoPages = DEFT_TABLE_NO_FREE_PAGE,
                  kPageCap = DEFT_TABLE_PAGE_CAP, kTokenCap = DEFT_TABLE_TOKEN_CAP;

struct TableArgs {
    const int32_t *node_len, *prev_len, *prev_off, *prev_id, *free_pages;
    int32_t num_nodes, num_prev, num_free;
    int64_t num_prev_ids;
    int32_t *page_off, *page_id, *tok_off, *slot, *counts;
    int32_t max_pages, max_tokens;
    uint32_t *block_sums;   // [4][kMaxBlocks]: pages, tokens, taken, flags (null: one block)
};

struct Sum3 {
    uint32_t pages, toks, taken;
};

__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b)
{
    return min(a + b, kSat);
}
__device__ __forceinline__ Sum3 add(const Sum3 &a, const Sum3 &b)
{
    return Sum3{sat_add(a.pages, b.pages), sat_add(a.toks, b.toks), sat_add(a.taken, b.taken)};
}

// One node's pages, new tokens and pages taken from the free list; `prev`
// and `first` are its earlier length and first page.
__device__ __forceinline__ Sum3 node_sum(const TableArgs &a, int n, int32_t &bad, int32_t &prev, int32_t &first)
{
    int32_t len = a.node_len[n];
    prev = n < a.num_prev ? a.prev_len[n] : 0;
    first = n < a.num_prev ? a.prev_off[n] : 0;
    if (len < 0 || prev < 0) {
        bad |= kBadLength;
        len = max(len, 0);
        prev = max(prev, 0);
    }
    const uint32_t pages = ((uint32_t)len + kPageSize - 1) / kPageSize;
    const uint32_t had = ((uint32_t)prev + kPageSize - 1) / kPageSize;
    const uint32_t kept = min(had, pages);
    if (kept > 0) {
        if (first < 0 || first + (int64_t)kept > a.num_prev_ids)
            bad |= kBadPrev;
    }
    return Sum3{pages, (uint32_t)max(len - prev, 0), pages - kept};
}

__device__ __forceinline__ Sum3 shfl_up(const Sum3 &v, int o)
{
    return Sum3{__shfl_up_sync(0xffffffffu, v.pages, o), __shfl_up_sync(0xffffffffu, v.toks, o),
                __shfl_up_sync(0xffffffffu, v.taken, o)};
}
__device__ __forceinline__ Sum3 shfl(const Sum3 &v, int l)
{
    return Sum3{__shfl_sync(0xffffffffu, v.pages, l), __shfl_sync(0xffffffffu, v.toks, l),
                __shfl_sync(0xffffffffu, v.taken, l)};
}
// Inclusive scan over the first N lanes of a warp.
template <int N>
__device__ __forceinline__ Sum3 warp_scan(Sum3 v)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < N; o <<= 1) {
        const Sum3 u = shfl_up(v, o);
        if (lane >= o)
            v = add(v, u);
    }
    return v;
}

// Exclusive scan over the CTA's threads; `total` is every thread's.
__device__ __forceinline__ Sum3 cta_scan(Sum3 v, Sum3 *warp_sum, Sum3 &total)
{
    constexpr int kWarps = kTableThreads / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Sum3 inc = warp_scan<32>(v);
    __syncthreads();   // an earlier scan's readers are done
    if (lane == 31)
        warp_sum[warp] = inc;
    __syncthreads();
    // Every warp scans the warps' sums itself.
    const Sum3 sums = warp_scan<kWarps>(lane < kWarps ? warp_sum[lane] : Sum3{0, 0, 0});
    total = shfl(sums, kWarps - 1);
    const Sum3 before = shfl(sums, warp > 0 ? warp - 1 : 0), prior = shfl_up(inc, 1);
    Sum3 exc{0, 0, 0};
    if (warp > 0)
        exc = before;
    if (lane > 0)
        exc = add(exc, prior);
    return exc;
}

// Sums of every block of nodes (more than one block only).
__global__ void __launch_bounds__(kTableThreads) table_sums_kernel(TableArgs a)
{
    __shared__ Sum3 warp_sum[kTableThreads / 32];
    grid_dep_launch();
    int32_t bad = 0, prev, off;
    Sum3 v{0, 0, 0}, total;
    const int first = blockIdx.x * kBlockNodes + threadIdx.x * kPerThread;
    for (int i = 0; i < kPerThread; ++i)
        if (first + i < a.num_nodes)
            v = add(v, node_sum(a, first + i, bad, prev, off));
    cta_scan(v, warp_sum, total);
    const int neg = __syncthreads_or(bad & kBadLength), outside = __syncthreads_or(bad & kBadPrev);
    if (threadIdx.x == 0) {
        a.block_sums[blockIdx.x] = total.pages;
        a.block_sums[kMaxBlocks + blockIdx.x] = total.toks;
        a.block_sums[2 * kMaxBlocks + blockIdx.x] = total.taken;
        a.block_sums[3 * kMaxBlocks + blockIdx.x] = (neg ? kBadLength : 0) | (outside ? kBadPrev : 0);
    }
}

struct TableSmem {
    uint32_t blk[3][kMaxBlocks + 1];    // exclusive sums before each block
    uint32_t off[3][kBlockNodes + 1];   // ... before each node of the block in hand
    int32_t prev[kBlockNodes], first[kBlockNodes];   // those nodes' earlier lengths and first pages
    Sum3 warp_sum[kTableThreads / 32];
};

// Largest i in [lo, hi) with off[i] <= x (off[lo] <= x < off[hi]).
__device__ __forceinline__ int find(const uint32_t *off, int lo, int hi, uint32_t x)
{
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kTableThreads) table_fill_kernel(TableArgs a, int32_t num_blocks)
{
    __shared__ TableSmem s;
    const int tid = threadIdx.x;
    int32_t bad = 0;
    int in_hand = -1;
    Sum3 total;
    if (num_blocks > 1) {
        grid_dep_wait();
        Sum3 v{0, 0, 0};
        if (tid < num_blocks) {
            v = Sum3{a.block_sums[tid], a.block_sums[kMaxBlocks + tid], a.block_sums[2 * kMaxBlocks + tid]};
            bad = (int32_t)a.block_sums[3 * kMaxBlocks + tid];
        }
        const Sum3 e = cta_scan(v, s.warp_sum, total);
        if (tid <= num_blocks) {
            s.blk[0][tid] = e.pages;
            s.blk[1][tid] = e.toks;
            s.blk[2][tid] = e.taken;
        }
        // num_blocks can equal the thread count: the end by thread 0.
        if (tid == 0) {
            s.blk[0][num_blocks] = total.pages;
            s.blk[1][num_blocks] = total.toks;
            s.blk[2][num_blocks] = total.taken;
        }
        __syncthreads();
    }
    // Scans block b's nodes into s.off (absolute offsets).
    auto take_block = [&](int b) {
        if (b == in_hand)
            return;
        __syncthreads();
        in_hand = b;
        const int first = b * kBlockNodes + tid * kPerThread;
        Sum3 node[kPerThread], sum{0, 0, 0}, all;
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) {
            const int x = tid * kPerThread + i;
            node[i] = first + i < a.num_nodes ? node_sum(a, first + i, bad, s.prev[x], s.first[x]) : Sum3{0, 0, 0};
            sum = add(sum, node[i]);
        }
        Sum3 e = cta_scan(sum, s.warp_sum, all);
        if (num_blocks > 1)
            e = add(e, Sum3{s.blk[0][b], s.blk[1][b], s.blk[2][b]});
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) {
            s.off[0][tid * kPerThread + i] = e.pages;
            s.off[1][tid * kPerThread + i] = e.toks;
            s.off[2][tid * kPerThread + i] = e.taken;
            e = add(e, node[i]);
        }
        if (tid == kTableThreads - 1) {
            s.off[0][kBlockNodes] = e.pages;
            s.off[1][kBlockNodes] = e.toks;
            s.off[2][kBlockNodes] = e.taken;
        }
        __syncthreads();
        if (num_blocks == 1)
            total = all;
    };
    if (num_blocks == 1)
        take_block(0);
    const int grid = gridDim.x, cta = blockIdx.x;

    // Where page j of the node at index i of the block in hand is listed
    // (null: nowhere).
    auto page_at = [&](int i, uint32_t j) -> const int32_t * {
        const uint32_t first_taken = s.off[2][i];
        const uint32_t pages = s.off[0][i + 1] - s.off[0][i], kept = pages - (s.off[2][i + 1] - first_taken);
        if (j < kept) {
            const int64_t at = (int64_t)s.first[i] + j;
            return at >= 0 && at < a.num_prev_ids ? a.prev_id + at : nullptr;
        }
        const uint32_t at = first_taken + (j - kept);
        return at < (uint32_t)a.num_free ? a.free_pages + at : nullptr;
    };
    // Offsets: block b by CTA b (and b + grid ...).
    for (int b = cta; b < num_blocks; b += grid) {
        take_block(b);
        for (int i = tid; i < kBlockNodes && b * kBlockNodes + i < a.num_nodes; i += kTableThreads) {
            a.page_off[b * kBlockNodes + i] = (int32_t)s.off[0][i];
            a.tok_off[b * kBlockNodes + i] = (int32_t)s.off[1][i];
        }
    }
    // Page ids and slots together: a thread a page (its node by binary
    // search), then the warp's pages' slots, half a warp a page.
    {
        const int64_t share = ((int64_t)total.pages + grid - 1) / grid;
        const uint32_t lo = (uint32_t)min(share * cta, (int64_t)total.pages);
        const uint32_t hi = (uint32_t)min(share * (cta + 1), (int64_t)total.pages);
        const int lane = tid & 31;
        uint32_t at = lo;
        while (at < hi) {
            const int b = num_blocks > 1 ? find(s.blk[0], 0, num_blocks, at) : 0;
            take_block(b);
            const uint32_t end = min(hi, s.off[0][kBlockNodes]);
            for (uint32_t x0 = at + (tid - lane); x0 < end; x0 += kTableThreads) {
                const uint32_t x = min(x0 + lane, end - 1);
                const int i = find(s.off[0], 0, kBlockNodes, x);
                const uint32_t j = x - s.off[0][i], first = s.off[1][i], fresh = s.off[1][i + 1] - first;
                const uint32_t prev = (uint32_t)max(s.prev[i], 0);
                // The new tokens of this page: t0 .. t0 + count - 1 of the
                // node, slots from q on.
                const uint32_t t0 = max(prev, j * kPageSize);
                const uint32_t t1 = min(prev + fresh, (j + 1) * kPageSize);
                const uint32_t count = x0 + lane < end && fresh > 0 && t1 > t0 ? t1 - t0 : 0;
                const uint32_t q = sat_add(first, t0 - min(t0, prev));
                // Pages and slots only grow from here on: past both
                // capacities there is nothing left to write.
                if (__all_sync(0xffffffffu, x >= (uint32_t)a.max_pages && q >= (uint32_t)a.max_tokens))
                    break;
                const int32_t *from = page_at(i, j);
                const int32_t page = from ? *from : -1;
                if (x0 + lane < end && x < (uint32_t)a.max_pages)
                    a.page_id[x] = page;
                const int32_t value = page < 0 || page > INT32_MAX / kPageSize ? -1 : page * kPageSize + (int32_t)(t0 % kPageSize);
                uint32_t left = __ballot_sync(0xffffffffu, count > 0 && q < (uint32_t)a.max_tokens);
                while (left) {
                    const int b0 = __ffs((int)left) - 1;
                    left &= left - 1;
                    const int b1 = left ? __ffs((int)left) - 1 : -1;
                    left &= left - 1;
                    const int src = lane < 16 ? b0 : b1 < 0 ? b0 : b1;
                    const uint32_t l = lane & 15;
                    const uint32_t sq = __shfl_sync(0xffffffffu, q, src) + l;
                    const uint32_t sn = __shfl_sync(0xffffffffu, count, src);
                    const int32_t sv = __shfl_sync(0xffffffffu, value, src);
                    if (l < sn && sq < (uint32_t)a.max_tokens && (lane < 16 || b1 >= 0))
                        a.slot[sq] = sv < 0 ? -1 : sv + (int32_t)l;
                }
            }
            at = end;
        }
    }
    // Past the last token, -1.
    for (int64_t x = (int64_t)total.toks + (int64_t)cta * kTableThreads + tid; x < a.max_tokens; x += (int64_t)grid * kTableThreads)
        a.slot[x] = -1;
    // The ends of both offset arrays and the counts, by CTA 0: every CTA has
    // the totals, and the flags of all nodes (scanned, or of the sums).
    if (cta == 0) {
        const int neg = __syncthreads_or(bad & kBadLength), prev = __syncthreads_or(bad & kBadPrev);
        if (tid == 0) {
            a.page_off[a.num_nodes] = (int32_t)total.pages;
            a.tok_off[a.num_nodes] = (int32_t)total.toks;
            a.counts[0] = (int32_t)total.pages;
            a.counts[1] = (int32_t)total.taken;
            a.counts[2] = (int32_t)total.toks;
            int32_t st = (neg ? kBadLength : 0) | (prev ? kBadPrev : 0);
            st |= total.taken > (uint32_t)a.num_free ? kNoPages : 0;
            st |= total.pages > (uint32_t)a.max_pages ? kPageCap : 0;
            st |= total.toks > (uint32_t)a.max_tokens ? kTokenCap : 0;
            a.counts[3] = st;
        }
    }
}

// 8 elements from `src` as bf16.
template <bool kF32>
struct Row8 {
    uint4 v[kF32 ? 2 : 1];
    __device__ __forceinline__ void load(const void *src, int64_t elem)
    {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const char *>(src) + elem * (kF32 ? 4 : 2));
        v[0] = __ldcs(p);
        if constexpr (kF32)
            v[1] = __ldcs(p + 1);
    }
    __device__ __forceinline__ uint4 bf16() const
    {
        if constexpr (!kF32) {
            return v[0];
        } else {
            auto two = [](uint32_t x, uint32_t y) {
                const __nv_bfloat162 r = __floats2bfloat162_rn(__uint_as_float(x), __uint_as_float(y));
                return *reinterpret_cast<const uint32_t *>(&r);
            };
            return make_uint4(two(v[0].x, v[0].y), two(v[0].z, v[0].w), two(v[1].x, v[1].y), two(v[1].z, v[1].w));
        }
    }
};

struct WriteArgs {
    const void *k, *v;
    int64_t k_stride, v_stride;   // elements between tokens
    const int32_t *slot;
    uint4 *k_pages, *v_pages;
    int32_t num_tokens, num_pages, num_kv_heads, head_dim;
};

constexpr int kWriteThreads = 256;

// U 16-byte pieces a thread, kWriteThreads apart; a token's pieces are its K
// row's, then its V row's (c8 = heads * head_dim / 8 each).  All loads go
// out before the first store.
template <bool kF32, int U>
__global__ void __launch_bounds__(kWriteThreads) kv_write_kernel(WriteArgs a, uint32_t c8, int64_t pieces)
{
    const uint32_t per_tok = 2 * c8;
    const int d8_log2 = a.head_dim == 128 ? 4 : 3;   // pieces of a head's row
    const int64_t x0 = (int64_t)blockIdx.x * (kWriteThreads * U) + threadIdx.x;
    const int64_t num_slots = (int64_t)a.num_pages * kPageSize;
    int64_t tok = x0 / per_tok;
    uint32_t j = (uint32_t)(x0 - tok * per_tok);
    Row8<kF32> row[U];
    uint4 *dst[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        dst[u] = nullptr;
        if (x0 + u * kWriteThreads < pieces) {
            const bool is_v = j >= c8;
            const uint32_t e = is_v ? j - c8 : j;
            const int32_t slot = a.slot[tok];
            if (slot >= 0 && slot < num_slots) {
                const uint32_t h = e >> d8_log2, part = e & ((1u << d8_log2) - 1);
                const int64_t line = ((int64_t)(slot / kPageSize) * a.num_kv_heads + h) * kPageSize + slot % kPageSize;
                dst[u] = (is_v ? a.v_pages : a.k_pages) + (line << d8_log2) + part;
                row[u].load(is_v ? a.v : a.k, tok * (is_v ? a.v_stride : a.k_stride) + (int64_t)e * 8);
            }
            for (j += kWriteThreads; j >= per_tok; j -= per_tok)
                ++tok;
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (dst[u])
            *dst[u] = row[u].bf16();
}

template <bool kF32>
int launch_write(const WriteArgs &a, cudaStream_t st)
{
    constexpr int U = 4;   // (2 or 8: 2% slower over 32768 tokens)
    const uint32_t c8 = (uint32_t)a.num_kv_heads * a.head_dim / 8;
    const int64_t pieces = (int64_t)a.num_tokens * 2 * c8;
    const int64_t blocks = (pieces + kWriteThreads * U - 1) / (kWriteThreads * U);
    if (blocks > INT32_MAX)
        return DEFT_EUNSUPPORTED;
    return launch(kv_write_kernel<kF32, U>, (unsigned)blocks, kWriteThreads, st, a, c8, pieces);
}

}  // namespace
}  // namespace deft

extern "C" {

size_t deft_page_table_workspace_bytes(int32_t num_nodes)
{
    if (num_nodes < 1)
        return 0;
    return num_nodes <= deft::kBlockNodes ? 0 : (size_t)4 * deft::kMaxBlocks * sizeof(uint32_t);
}

int deft_page_table(const int32_t *node_len, int32_t num_nodes, const int32_t *prev_len, const int32_t *prev_page_off,
                    const int32_t *prev_page_id, int32_t num_prev_nodes, int64_t num_prev_ids,
                    const int32_t *free_pages, int32_t num_free, int32_t page_size, int32_t *node_page_off,
                    int32_t *page_id, int32_t max_pages, int32_t *tok_off, int32_t *slot, int32_t max_tokens,
                    int32_t *counts, void *workspace, size_t workspace_bytes, void *stream)
{
    using namespace deft;
    if (!node_len || num_nodes < 1 || !node_page_off || !tok_off || !counts || num_free < 0 || max_pages < 0 ||
        max_tokens < 0 || num_prev_nodes < 0 || num_prev_ids < 0 || num_prev_nodes > num_nodes)
        return DEFT_EINVAL;
    if ((num_free > 0 && !free_pages) || (max_pages > 0 && !page_id) || (max_tokens > 0 && !slot) ||
        (num_prev_nodes > 0 && (!prev_len || !prev_page_off)) || (num_prev_ids > 0 && !prev_page_id))
        return DEFT_EINVAL;
    // The earlier table is read while the new one is written.
    if (num_prev_nodes > 0 && (prev_page_off == node_page_off || prev_len == node_page_off || prev_len == tok_off ||
                               (num_prev_ids > 0 && prev_page_id == page_id)))
        return DEFT_EINVAL;
    if (page_size != kPageSize || num_nodes > kMaxBlocks * kBlockNodes)
        return DEFT_EUNSUPPORTED;
    const size_t need = deft_page_table_workspace_bytes(num_nodes);
    if (need && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) || workspace_bytes < need))
        return DEFT_EWORKSPACE;
    TableArgs a{node_len, prev_len, prev_page_off, prev_page_id, free_pages, num_nodes, num_prev_nodes, num_free,
                num_prev_ids, node_page_off, page_id, tok_off, slot, counts, max_pages, max_tokens,
                need ? static_cast<uint32_t *>(workspace) : nullptr};
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int blocks = (num_nodes + kBlockNodes - 1) / kBlockNodes;
    // One CTA for every 1024 outputs, at most one an SM: each repeats the
    // scan of its nodes' block.
    const int64_t outputs = (int64_t)max_pages + max_tokens;
    const int64_t want = (outputs + 1023) / 1024;
    const int grid = (int)(want < 1 ? 1 : want > num_sms() ? num_sms() : want);
    if (blocks > 1) {
        if (launch(table_sums_kernel, (unsigned)blocks, kTableThreads, st, a) != DEFT_OK)
            return DEFT_ECUDA;
        return launch_dependent(table_fill_kernel, dim3(grid), dim3(kTableThreads), 0, st, a, blocks) == cudaSuccess
                   ? DEFT_OK
                   : DEFT_ECUDA;
    }
    return launch(table_fill_kernel, (unsigned)grid, kTableThreads, st, a, (int32_t)1);
}

int deft_kv_write(const void *k, const void *v, int32_t in_dtype, int64_t k_stride, int64_t v_stride,
                  const int32_t *slot, int32_t num_tokens, void *k_pages, void *v_pages, int32_t num_pages,
                  int32_t num_kv_heads, int32_t head_dim, int32_t page_size, void *stream)
{
    using namespace deft;
    if (num_tokens < 0 || num_pages < 1 || num_kv_heads < 1 || !k_pages || !v_pages || k_pages == v_pages ||
        (in_dtype != DEFT_OUT_BF16 && in_dtype != DEFT_OUT_F32))
        return DEFT_EINVAL;
    if ((head_dim != 64 && head_dim != 128) || page_size != kPageSize || num_pages > INT32_MAX / kPageSize)
        return DEFT_EUNSUPPORTED;
    if (num_tokens == 0)
        return DEFT_OK;
    const int64_t row = (int64_t)num_kv_heads * head_dim;
    const int64_t es = in_dtype == DEFT_OUT_F32 ? 4 : 2;
    if (!k || !v || !slot || row > (1 << 24))
        return DEFT_EINVAL;
    // Rows are read in 16-byte pieces and do not overlap.
    if (((uintptr_t)k | (uintptr_t)v | (uintptr_t)k_pages | (uintptr_t)v_pages) & 15u)
        return DEFT_EINVAL;
    if ((num_tokens > 1) && (k_stride < row || v_stride < row || (k_stride * es) % 16 || (v_stride * es) % 16))
        return DEFT_EINVAL;
    WriteArgs a{k, v, k_stride, v_stride, slot, static_cast<uint4 *>(k_pages), static_cast<uint4 *>(v_pages),
                num_tokens, num_pages, num_kv_heads, head_dim};
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return in_dtype == DEFT_OUT_F32 ? launch_write<true>(a, st) : launch_write<false>(a, st);
}

}  // extern "C"
