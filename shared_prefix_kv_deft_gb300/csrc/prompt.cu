// prompt.cu -- entry points of the prompt step (deft_prompt_*) and the merge
// of its split ranges.
//
// The step: row t of a prompt (position t in its node) and query head h
// attend, with one softmax, to every token of the ancestors and to tokens
// 0..t of the node:
//     s_j = scale * q.k_j,  M = max s_j,  l = sum 2^((s_j - M) log2 e),
//     out = sum_j 2^((s_j - M) log2 e) v_j / l,  lse = M + ln l.
// A range-split item's pieces hold (o, base-2 lse) of their own pages; the
// merge weighs them by 2^(lse - max), as phase2.cu does for tree steps.
// A NaN or +inf among a row's logits makes l, out and lse NaN, and so does a
// NaN lse of one piece; logits that are all -inf give out NaN (0 / 0) and
// lse -inf, whether the range is cut or not.
#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>
#include <type_traits>
#include <utility>

#include <cuda_runtime.h>

#include "common.cuh"
#include "prompt_internal.h"

namespace deft {
namespace {

constexpr int kMergeThreads = 256;

// One warp per (split item, KV head, row): lane i owns D / 32 consecutive
// elements.  The lse of all pieces first (one a lane), then the pieces' rows
// four at a time, so that a row costs about two L2 latencies; pieces none of
// whose tokens the row sees (lse -inf, their rows never written) are not
// read.  The sum runs over the pieces in order.
template <int D>
__global__ void __launch_bounds__(kMergeThreads) prompt_merge_kernel(PromptArgs a)
{
    constexpr int E = D / 32;
    using Vec = typename std::conditional<E == 4, float4, float2>::type;
    grid_dep_launch();
    // The plan too is read behind the wait: the attention launch lets this
    // one start before it has waited for the plan's copy itself.
    grid_dep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int G = a.gqa_group, Hkv = a.num_kv_heads;
    const PromptMerge m = a.plan.merges[blockIdx.x / Hkv];
    const int h = blockIdx.x % Hkv, rows = m.tokens * G;
    const int r = blockIdx.y * (kMergeThreads / 32) + warp;
    if (r >= rows)
        return;
    const size_t first = (size_t)m.part0 + (size_t)h * rows + r, step = (size_t)Hkv * rows;
    float M = -INFINITY;
    for (int j = lane; j < m.pieces; j += 32)
        M = fmaxf(M, a.lse_part[first + j * step]);
    M = warp_max(M);   // (passes over NaN: the weights below bring it in)
    const float base = M == -INFINITY ? 0.f : M;
    float acc[E] = {}, sum = 0.f;
    for (int j0 = 0; j0 < m.pieces; j0 += 32) {
        const float w = j0 + lane < m.pieces ? exp2f(a.lse_part[first + (j0 + lane) * step] - base) : 0.f;
        sum += w;
        const int n = min(32, m.pieces - j0);
        for (int j = 0; j < n; j += 4) {
            Vec v[4];
            float wj[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                wj[i] = __shfl_sync(0xffffffffu, w, (j + i) & 31);
                if (j + i >= n)
                    wj[i] = 0.f;
                if (wj[i] != 0.f)
                    v[i] = *reinterpret_cast<const Vec *>(a.o_part + (first + (j0 + j + i) * step) * D + lane * E);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (wj[i] == 0.f)
                    continue;
                const float *o = reinterpret_cast<const float *>(&v[i]);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    acc[e] = fmaf(wj[i], o[e], acc[e]);
            }
        }
    }
    sum = warp_sum(sum);
    const float inv = 1.f / sum;
    const size_t row = (size_t)(m.row0 + r / G) * a.num_q_heads + h * G + r % G;
    if (a.out_dtype == DEFT_OUT_F32) {
        Vec v;
        float *o = reinterpret_cast<float *>(&v);
#pragma unroll
        for (int e = 0; e < E; ++e)
            o[e] = acc[e] * inv;
        *reinterpret_cast<Vec *>(static_cast<float *>(a.out) + row * D + lane * E) = v;
    } else {
        __nv_bfloat162 *o = reinterpret_cast<__nv_bfloat162 *>(static_cast<__nv_bfloat16 *>(a.out) + row * D + lane * E);
#pragma unroll
        for (int e = 0; e < E; e += 2)
            o[e / 2] = __floats2bfloat162_rn(acc[e] * inv, acc[e + 1] * inv);
    }
    if (lane == 0)
        a.lse[row] = (M + log2f(sum)) * kLn2;
}

}  // namespace

int launch_prompt_merge(const PromptArgs &a, int32_t num_merges, void *stream)
{
    const dim3 grid((unsigned)(num_merges * a.num_kv_heads), 2 * kPromptRows / (kMergeThreads / 32));
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (a.head_dim == 128)
        return (int)launch_dependent(prompt_merge_kernel<128>, grid, dim3(kMergeThreads), 0, st, a);
    return (int)launch_dependent(prompt_merge_kernel<64>, grid, dim3(kMergeThreads), 0, st, a);
}

}  // namespace deft

namespace {

constexpr size_t kAlign = deft::kWorkAlign;

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

// The arrays of the device copy, in order, then the status word.
constexpr int kPromptArrays = 5;
struct PromptLayout {
    deft::ArrayRef src[kPromptArrays];
    size_t off[kPromptArrays + 1];
    size_t end;
};

PromptLayout prompt_layout(const deft_prompt_plan_t &p)
{
    PromptLayout L{{deft::aref(p.nodes), deft::aref(p.items), deft::aref(p.cta_off), deft::aref(p.cta_unit),
                    deft::aref(p.merges)},
                   {},
                   0};
    for (int i = 0; i < kPromptArrays; ++i) {
        L.off[i] = L.end;
        L.end = align_up(L.end + (L.src[i].bytes ? L.src[i].bytes : 4));
    }
    L.off[kPromptArrays] = L.end;
    L.end += kAlign;
    return L;
}

int build_prompt_host(const int32_t *parent, const int32_t *node_len, int32_t num_nodes, const int32_t *prompt_node,
                      const int32_t *prompt_len, int32_t num_prompts, int32_t num_kv_heads, int32_t gqa_group,
                      deft_prompt_plan_t *p)
{
    int rc;
    try {
        rc = deft::build_prompt_plan(parent, node_len, num_nodes, prompt_node, prompt_len, num_prompts, num_kv_heads,
                                     gqa_group, p);
    } catch (const std::bad_alloc &) {
        rc = DEFT_ENOMEM;
    }
    if (rc == DEFT_OK)
        p->stats.device_bytes = (int64_t)prompt_layout(*p).end;
    return rc;
}

}  // namespace

extern "C" {

int deft_prompt_plan(const int32_t *parent, const int32_t *node_len, int32_t num_nodes, const int32_t *prompt_node,
                     const int32_t *prompt_len, int32_t num_prompts, int32_t num_kv_heads, int32_t gqa_group,
                     deft_prompt_plan_t **out)
{
    if (!out)
        return DEFT_EINVAL;
    *out = nullptr;
    deft_prompt_plan_t *p = new (std::nothrow) deft_prompt_plan_t();
    if (!p)
        return DEFT_ENOMEM;
    const int rc = build_prompt_host(parent, node_len, num_nodes, prompt_node, prompt_len, num_prompts, num_kv_heads,
                                     gqa_group, p);
    if (rc != DEFT_OK) {
        delete p;
        return rc;
    }
    *out = p;
    return DEFT_OK;
}

int deft_prompt_plan_rebuild(deft_prompt_plan_t *plan, const int32_t *parent, const int32_t *node_len,
                             int32_t num_nodes, const int32_t *prompt_node, const int32_t *prompt_len,
                             int32_t num_prompts, int32_t num_kv_heads, int32_t gqa_group)
{
    if (!plan)
        return DEFT_EINVAL;
    // Built into this thread's spare and swapped in: the plan is as it was
    // on an error, and the replaced arrays' storage serves the next rebuild.
    thread_local deft_prompt_plan_t spare;
    const int rc = build_prompt_host(parent, node_len, num_nodes, prompt_node, prompt_len, num_prompts, num_kv_heads,
                                     gqa_group, &spare);
    if (rc != DEFT_OK)
        return rc;
    plan->num_nodes = spare.num_nodes;
    plan->num_prompts = spare.num_prompts;
    plan->num_kv_heads = spare.num_kv_heads;
    plan->gqa_group = spare.gqa_group;
    plan->num_rows = spare.num_rows;
    plan->part_slots = spare.part_slots;
    plan->stats = spare.stats;
    std::swap(plan->nodes, spare.nodes);
    std::swap(plan->items, spare.items);
    std::swap(plan->cta_off, spare.cta_off);
    std::swap(plan->cta_unit, spare.cta_unit);
    std::swap(plan->merges, spare.merges);
    plan->uploaded = false;
    return DEFT_OK;
}

int deft_prompt_plan_stats_get(const deft_prompt_plan_t *plan, deft_prompt_stats *out)
{
    if (!plan || !out)
        return DEFT_EINVAL;
    *out = plan->stats;
    return DEFT_OK;
}

int deft_prompt_plan_get(const deft_prompt_plan_t *plan, int32_t which, void *dst, size_t bytes)
{
    if (!plan || (!dst && bytes) || which < 0 || which >= kPromptArrays)
        return DEFT_EINVAL;
    const deft::ArrayRef src = prompt_layout(*plan).src[which];
    if (bytes < src.bytes)
        return DEFT_EINVAL;
    if (src.bytes)
        std::memcpy(dst, src.ptr, src.bytes);
    return DEFT_OK;
}

int deft_prompt_plan_upload(deft_prompt_plan_t *plan, void *stream)
{
    if (!plan)
        return DEFT_EINVAL;
    const PromptLayout L = prompt_layout(*plan);
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return DEFT_ECUDA;
    if (plan->dev_blob && (plan->dev_bytes < L.end || plan->dev_device != dev)) {
        cudaFree(plan->dev_blob);
        plan->dev_blob = nullptr;
        plan->uploaded = false;
    }
    if (!plan->dev_blob) {
        if (cudaMalloc(&plan->dev_blob, L.end) != cudaSuccess) {
            plan->dev_blob = nullptr;
            return DEFT_ENOMEM;
        }
        plan->dev_bytes = L.end;
        plan->dev_device = dev;
    }
    cudaEvent_t done = reinterpret_cast<cudaEvent_t>(plan->stage_done);
    if (done && cudaEventSynchronize(done) != cudaSuccess)
        return DEFT_ECUDA;
    if (done && plan->stage_device != dev) {
        cudaEventDestroy(done);
        done = nullptr;
        plan->stage_done = nullptr;
    }
    if (!done) {
        if (cudaEventCreateWithFlags(&done, cudaEventDisableTiming) != cudaSuccess)
            return DEFT_ECUDA;
        plan->stage_done = done;
        plan->stage_device = dev;
    }
    if (plan->host_stage_bytes < L.end) {
        if (plan->host_stage)
            cudaFreeHost(plan->host_stage);
        plan->host_stage = nullptr;
        plan->host_stage_bytes = 0;
        if (cudaHostAlloc(&plan->host_stage, L.end, cudaHostAllocPortable) != cudaSuccess) {
            plan->host_stage = nullptr;
            return DEFT_ENOMEM;
        }
        plan->host_stage_bytes = L.end;
    }
    uint8_t *host = static_cast<uint8_t *>(plan->host_stage);
    for (int i = 0; i < kPromptArrays; ++i)
        if (L.src[i].bytes)
            std::memcpy(host + L.off[i], L.src[i].ptr, L.src[i].bytes);
    std::memset(host + L.off[kPromptArrays], 0, kAlign);   // the status word
    uint8_t *dev_base = static_cast<uint8_t *>(plan->dev_blob);
    plan->dev.nodes = reinterpret_cast<const int2 *>(dev_base + L.off[0]);
    plan->dev.items = reinterpret_cast<const deft::PromptItem *>(dev_base + L.off[1]);
    plan->dev.cta_off = reinterpret_cast<const int32_t *>(dev_base + L.off[2]);
    plan->dev.cta_unit = reinterpret_cast<const int32_t *>(dev_base + L.off[3]);
    plan->dev.merges = reinterpret_cast<const deft::PromptMerge *>(dev_base + L.off[4]);
    plan->dev.status = reinterpret_cast<uint32_t *>(dev_base + L.off[5]);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (cudaMemcpyAsync(plan->dev_blob, host, L.end, cudaMemcpyHostToDevice, st) != cudaSuccess ||
        cudaEventRecord(done, st) != cudaSuccess)
        return DEFT_ECUDA;
    plan->uploaded = true;
    return DEFT_OK;
}

size_t deft_prompt_workspace_bytes(const deft_prompt_plan_t *plan, int32_t num_q_heads, int32_t head_dim)
{
    if (!plan || num_q_heads < 1 || head_dim < 1)
        return 0;
    // Slots count the rows of all query heads already (group x KV heads).
    return deft::work_layout(plan->part_slots > 0 ? plan->part_slots : 1, 1, head_dim).total;
}

int deft_prompt_attn(const void *q, int64_t q_stride, int32_t num_rows, const void *k_pages, const void *v_pages,
                     const int32_t *node_page_off, const int32_t *page_id, int32_t num_pages, int32_t num_q_heads,
                     int32_t num_kv_heads, int32_t head_dim, int32_t page_size, float scale,
                     const deft_prompt_plan_t *plan, void *out, int32_t out_dtype, float *lse, void *workspace,
                     size_t workspace_bytes, void *stream)
{
    using namespace deft;
    if (!plan || !q || !k_pages || !v_pages || !node_page_off || !page_id || !out || !lse)
        return DEFT_EINVAL;
    if (out_dtype != DEFT_OUT_BF16 && out_dtype != DEFT_OUT_F32)
        return DEFT_EINVAL;
    if (!(scale > 0.f) || !std::isfinite(scale) || num_pages < 1 || num_rows < 0)
        return DEFT_EINVAL;
    if (num_kv_heads < 1 || num_q_heads < 1 || num_q_heads % num_kv_heads != 0)
        return DEFT_EINVAL;
    if ((((uintptr_t)q | (uintptr_t)k_pages | (uintptr_t)v_pages) & 15u) || ((uintptr_t)out & 31u))
        return DEFT_EINVAL;
    if ((head_dim != 64 && head_dim != 128) || page_size != kPageSize)
        return DEFT_EUNSUPPORTED;
    if (q_stride < (int64_t)num_q_heads * head_dim || (q_stride * 2) % 16 != 0 || q_stride > ((int64_t)1 << 38))
        return DEFT_EINVAL;
    if (num_kv_heads != plan->num_kv_heads || num_q_heads / num_kv_heads != plan->gqa_group || !plan->uploaded)
        return DEFT_ESTATE;
    if (num_rows < plan->num_rows)
        return DEFT_EINVAL;   // fewer q rows than the plan's prompts have tokens
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return DEFT_ECUDA;
    if (dev != plan->dev_device)
        return DEFT_ESTATE;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) % kAlign) != 0 ||
        workspace_bytes < deft_prompt_workspace_bytes(plan, num_q_heads, head_dim))
        return DEFT_EWORKSPACE;
    if (plan->num_rows == 0)
        return DEFT_OK;
    const WorkLayout wl = work_layout(plan->part_slots > 0 ? plan->part_slots : 1, 1, head_dim);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    PromptArgs a{};
    a.q = q;
    a.q_stride = q_stride;
    a.k_pages = k_pages;
    a.v_pages = v_pages;
    a.node_page_off = node_page_off;
    a.page_id = page_id;
    a.num_pages = num_pages;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = num_kv_heads;
    a.head_dim = head_dim;
    a.gqa_group = plan->gqa_group;
    a.num_rows = num_rows;
    a.scale_log2 = scale * 1.44269504088896340736f;
    a.out = out;
    a.out_dtype = out_dtype;
    a.lse = lse;
    a.o_part = reinterpret_cast<float *>(ws + wl.o_off);
    a.lse_part = reinterpret_cast<float *>(ws + wl.lse_off);
    a.plan = plan->dev;
    if (launch_prompt(a, plan->stats.ctas, stream) != 0)
        return DEFT_ECUDA;
    if (!plan->merges.empty() && launch_prompt_merge(a, (int32_t)plan->merges.size(), stream) != 0)
        return DEFT_ECUDA;
    return DEFT_OK;
}

int deft_prompt_status(deft_prompt_plan_t *plan, void *stream, int32_t *code)
{
    if (!plan || !code)
        return DEFT_EINVAL;
    *code = 0;
    if (!plan->uploaded)
        return DEFT_ESTATE;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    uint32_t word = 0;
    if (cudaMemcpyAsync(&word, plan->dev.status, 4, cudaMemcpyDeviceToHost, st) != cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess)
        return DEFT_ECUDA;
    if (word && cudaMemsetAsync(plan->dev.status, 0, 4, st) != cudaSuccess)
        return DEFT_ECUDA;
    *code = (int32_t)word;
    return word ? DEFT_EDEVICE : DEFT_OK;
}

void deft_prompt_plan_free(deft_prompt_plan_t *plan)
{
    if (!plan)
        return;
    if (plan->stage_done) {
        cudaEventSynchronize(reinterpret_cast<cudaEvent_t>(plan->stage_done));
        cudaEventDestroy(reinterpret_cast<cudaEvent_t>(plan->stage_done));
    }
    if (plan->host_stage)
        cudaFreeHost(plan->host_stage);
    if (plan->dev_blob)
        cudaFree(plan->dev_blob);
    delete plan;
}

}  // extern "C"
