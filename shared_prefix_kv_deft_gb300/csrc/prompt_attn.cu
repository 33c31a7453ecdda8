// prompt_attn.cu -- attention of whole prompts over the paged cache: a
// simple form, one warp per row and head, tokens one after another.
#include "common.cuh"
#include "prompt_internal.h"

namespace deft {
namespace {

constexpr int kThreads = 512;

template <int D>
__global__ void __launch_bounds__(kThreads) prompt_kernel(PromptArgs a)
{
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int G = a.gqa_group, Hkv = a.num_kv_heads;
    const __nv_bfloat16 *K = static_cast<const __nv_bfloat16 *>(a.k_pages), *V = static_cast<const __nv_bfloat16 *>(a.v_pages);
    for (int u = a.plan.cta_off[blockIdx.x]; u < a.plan.cta_off[blockIdx.x + 1]; ++u) {
        const int unit = a.plan.cta_unit[u], h = unit % Hkv;
        const PromptItem it = a.plan.items[unit / Hkv];
        const int rows = (it.tok_a + it.tok_b) * G;
        for (int r = warp; r < rows; r += kThreads / 32) {
            const int tok = r / G, head = h * G + r % G, pos = it.pos0 + tok;
            const __nv_bfloat16 *qp = static_cast<const __nv_bfloat16 *>(a.q) + (it.row0 + tok) * a.q_stride + (size_t)head * D + lane * E;
            float q[E], o[E] = {}, m = -INFINITY, l = 0.f;
            for (int e = 0; e < E; ++e)
                q[e] = __bfloat162float(qp[e]) * a.scale_log2;
            int node = it.start_node, pg = it.start_page;
            for (int k = 0; k < it.pages; ++k) {
                const int2 rec = a.plan.nodes[node];
                const bool own = node == it.node;
                const int cnt = min(kPageSize, (own ? pos + 1 : rec.y) - pg * kPageSize);
                const size_t page = a.page_id[a.node_page_off[node] + pg];
                for (int i = 0; i < cnt; ++i) {
                    const size_t at = ((page * Hkv + h) * kPageSize + i) * D + lane * E;
                    float s = 0.f;
                    for (int e = 0; e < E; ++e)
                        s += q[e] * __bfloat162float(K[at + e]);
                    s = warp_sum(s);
                    const float mn = fmaxf(m, s), f = exp2f(m - mn), p = exp2f(s - mn);
                    m = mn;
                    l = l * f + p;
                    for (int e = 0; e < E; ++e)
                        o[e] = o[e] * f + p * __bfloat162float(V[at + e]);
                }
                if (++pg * kPageSize >= rec.y && !own) {
                    node = rec.x < 0 ? it.node : rec.x;
                    pg = 0;
                }
            }
            const float inv = l > 0.f ? 1.f / l : 0.f;
            if (it.part0 >= 0) {
                const size_t slot = (size_t)it.part0 + (size_t)h * rows + r;
                for (int e = 0; e < E; ++e)
                    a.o_part[slot * D + lane * E + e] = o[e] * inv;
                if (lane == 0)
                    a.lse_part[slot] = m + log2f(l);
            } else {
                const size_t row = (size_t)(it.row0 + tok) * a.num_q_heads + head;
                for (int e = 0; e < E; ++e) {
                    if (a.out_dtype == DEFT_OUT_F32)
                        static_cast<float *>(a.out)[row * D + lane * E + e] = o[e] * inv;
                    else
                        static_cast<__nv_bfloat16 *>(a.out)[row * D + lane * E + e] = __float2bfloat16_rn(o[e] * inv);
                }
                if (lane == 0)
                    a.lse[row] = (m + log2f(l)) * kLn2;
            }
        }
    }
}

}  // namespace

int launch_prompt(const PromptArgs &a, int32_t ctas, void *stream)
{
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (a.head_dim == 128)
        prompt_kernel<128><<<ctas, kThreads, 0, st>>>(a);
    else
        prompt_kernel<64><<<ctas, kThreads, 0, st>>>(a);
    return (int)cudaGetLastError();
}

}  // namespace deft
