// prompt_internal.h -- the prompt plan (deft_prompt_plan_t) and what its
// kernels read: host planning in prompt_plan.cpp, the attention kernel in
// prompt_attn.cu, entry points and the merge kernel in prompt.cu.
#pragma once

#include <cstdint>
#include <vector>

#include "deft_internal.h"

namespace deft {

constexpr int kPromptRows = 128;      // rows of a query tile (tokens x GQA group)
constexpr int kPromptTilePages = 8;   // pages of a KV tile (128 tokens)
// CTAs the plan deals its units to, one per SM of a whole GB300 and the same
// on any device: results do not depend on it, the balance does.
constexpr int kPromptCtas = 152;

// One work item: up to two neighbouring query tiles (A, then B) of a prompt
// against a range of the pages of its path.  A unit is an item and a KV
// head.  Pages are counted along the path: those of the ancestors from the
// node's parent up to its root, then the node's own.
struct PromptItem {
    int32_t row0;        // q / out row (token) of tile A's first token
    int32_t tok_a;       // tokens of tile A, 1 .. tokens a tile holds
    int32_t tok_b;       // tokens of tile B (they follow tile A's), 0: none
    int32_t pos0;        // position in the node of tile A's first token
    int32_t node;
    int32_t pages;       // pages of the range
    int32_t tiles_a;     // KV tiles tile A reads (0: its rows see none of the range)
    int32_t tiles_b;
    int32_t start_node;  // the range's first page: page start_page of start_node
    int32_t start_page;
    int32_t part0;       // first partial slot, -1: the rows are written to out / lse
    int32_t pad;
};
static_assert(sizeof(PromptItem) == 48, "read as three 16-byte pieces");

// The rows of a range-split item, merged after the pieces: piece j of KV
// head h holds row r (token x group) at part0 + (j * Hkv + h) * rows + r.
struct PromptMerge {
    int32_t row0, tokens, part0, pieces;
};

// Arrays of the device copy.
struct PromptDev {
    const int2 *nodes;          // per node: nearest ancestor with tokens (-1: none), tokens
    const PromptItem *items;
    const int32_t *cta_off;     // [kPromptCtas + 1]
    const int32_t *cta_unit;    // item * Hkv + KV head, in the order the CTA runs them
    const PromptMerge *merges;
    uint32_t *status;           // 0, or the code of the first wait that ran out
};

}  // namespace deft

struct deft_prompt_plan_t {
    int32_t num_nodes = 0, num_prompts = 0, num_kv_heads = 0, gqa_group = 1;
    int32_t num_rows = 0;                   // q rows (tokens)
    std::vector<int32_t> nodes;             // [2 * num_nodes]
    std::vector<deft::PromptItem> items;
    std::vector<int32_t> cta_off, cta_unit;
    std::vector<deft::PromptMerge> merges;
    int64_t part_slots = 0;                 // partial rows (per query head)
    deft_prompt_stats stats{};
    // Device copy and its pinned staging buffer, as deft_plan_t's.
    void *dev_blob = nullptr;
    size_t dev_bytes = 0;
    int dev_device = -1;
    bool uploaded = false;
    deft::PromptDev dev{};
    void *host_stage = nullptr;
    size_t host_stage_bytes = 0;
    void *stage_done = nullptr;
    int stage_device = -1;
};

namespace deft {

// Builds the host side of `p` (its device state untouched); a status code.
int build_prompt_plan(const int32_t *parent, const int32_t *node_len, int32_t num_nodes, const int32_t *prompt_node,
                      const int32_t *prompt_len, int32_t num_prompts, int32_t num_kv_heads, int32_t gqa_group,
                      deft_prompt_plan_t *p);

}  // namespace deft

namespace deft {

// What the prompt kernels get.
struct PromptArgs {
    const void *q;
    int64_t q_stride;        // elements between tokens
    const void *k_pages, *v_pages;
    const int32_t *node_page_off, *page_id;
    int32_t num_pages, num_q_heads, num_kv_heads, head_dim, gqa_group, num_rows;
    float scale_log2;        // base-2 logits
    void *out;
    int32_t out_dtype;
    float *lse;
    float *o_part, *lse_part;   // pieces: fp32 rows and base-2 lse per slot
    PromptDev plan;
};

int launch_prompt(const PromptArgs &a, int32_t ctas, void *stream);
int launch_prompt_merge(const PromptArgs &a, int32_t num_merges, void *stream);

}  // namespace deft
