// kv4_internal.h -- launchers of the steps over a 4-bit cache (the plan and
// the arguments they share with the bf16 steps: deft_internal.h).
#pragma once

#include "deft_internal.h"

#ifdef __CUDACC__
#define DEFT_HOST_DEVICE __host__ __device__
#else
#define DEFT_HOST_DEVICE
#endif

namespace deft {

// A ring of barriers, one copy a phase: copy j completes phase j / stages of
// barrier j % stages.
template <typename Wait>
DEFT_HOST_DEVICE inline bool ring_wait(int j, int stages, Wait &&wait)
{
    return wait(j % stages, (uint32_t)(j / stages) & 1u);
}

// The copies that may still be on their way when the wait for copy `first`
// has run out and `issued` copies went out in all: the ones from `first` on.
// (Earlier ones have been waited for.  A barrier answers for the parity of the
// phase before the one it is in: another parity than the copy's would be
// answered at once with the copy in flight, and a stage without a copy never.)
template <typename Wait>
DEFT_HOST_DEVICE inline void ring_drain(int first, int issued, int stages, Wait &&wait)
{
    for (int j = first; j < issued; ++j)
        ring_wait(j, stages, wait);
}

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
