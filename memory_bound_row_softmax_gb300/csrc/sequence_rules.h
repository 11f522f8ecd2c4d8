// sequence_rules.h -- the rules by which a sequence attention call chooses how it
// runs, from sizes alone: plain C++, for the host and the device alike.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define MBRS_RULE __host__ __device__ inline
#else
#define MBRS_RULE inline
#endif

namespace mbrs {
namespace seq {

// What k_tiles_plan has counted: row blocks (at one kv head), their key tiles in
// all, and those of the longest and the shortest.  In 64 bits: offsets that do not
// rise can name more row blocks than 32 bits hold (sequences may overlap), and a
// count that wrapped would pass for one that the plan has room for.
struct PlanCounts {
    uint64_t blocks, tiles;
    uint32_t most, least;
};

// Whether items are cut into equal stretches instead of taken whole: where one item
// is longer than an SM's share, or where the last wave of items would leave SMs idle
// for longer than cutting costs (items of one length leave waves rounded up less
// waves, in items' time; others at least that of the shortest, which come last), or
// where there are more row blocks than the plan has room for.
MBRS_RULE bool plan_cuts(const PlanCounts &c, uint32_t kv_heads, uint32_t sms, uint32_t capacity, uint32_t cut_cost) {
    if (c.blocks > capacity) return true;
    const uint64_t items = c.blocks * kv_heads;
    const uint64_t idle = ((items + sms - 1) / sms * sms - items) * c.least;
    return (uint64_t)c.most * sms > c.tiles * kv_heads || idle > (uint64_t)cut_cost * sms;
}

}  // namespace seq
}  // namespace mbrs
