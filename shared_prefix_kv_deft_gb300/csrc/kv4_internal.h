// kv4_internal.h -- launchers of the steps over a 4-bit cache (the plan and
// the arguments they share with the bf16 steps: deft_internal.h).
#pragma once

#include "deft_internal.h"

namespace deft {

// A phase-1 launch over a 4-bit cache: items [first, first + n) of one of
// the partition's two lists.
struct Kv4Args {
    AttnArgs a;                // k_pages, v_pages: the 4-bit pools
    float k_scale, v_scale;
    int32_t first, n;
    int32_t wide;              // 1: of the tensor-core list
    int32_t mma_narrow;        // tensor-core items below this have their row masks split at 16, not 32
    int32_t heads;             // KV heads a CTA takes (1, 2 or 4)
    int32_t head_groups;       // CTAs of an item
    int32_t last;              // 1: not the step's first phase-1 launch
};
// Tensor-core items of at most 32 or 64 rows at head_dim 128.
int launch_phase1_kv4_mma(const Kv4Args &ka, const DevPartition &p, int rows, void *stream);
// dispatch_step over a 4-bit cache: phase-1 launches by width, and the merge
// (phase1_kv4.cu).
// max_slots: the most partials a query has.
int dispatch_step4(const AttnArgs &a, const DevPartition &dp, const Partition &hp, float k_scale, float v_scale,
                   int32_t max_slots, void *stream, const LaunchTracer &trace);

}  // namespace deft
