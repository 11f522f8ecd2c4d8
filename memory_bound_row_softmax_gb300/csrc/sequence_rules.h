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

// Whether the keys stream by blocks of 16 or 32 query rows (k_seq_rows) or meet tiles
// of 256 (k_seq_tiles), for the whole batch: lengths are on the device, so the host
// goes by the rows of an average sequence at one kv head, and by how many there are
// beyond one token a sequence: a batch of single tokens with a long chunk (or a prompt
// beside empty sequences) has a low average too, and there each 32 rows of the chunk
// would read all of its keys again.  Measured in us, streaming against tiles, over 4000
// keys a sequence of head dim 128 where not said otherwise:
//   equal sequences, 4 tokens of 64/8 heads: 32 of them (768 rows beyond) 113 and 124,
//     64 (1536) 204 and 229; 6 tokens of 32/8 heads, 48 (960): 156 and 180; 4 tokens of
//     32/8 heads, 128 (1536, 16 rows each): 333 and 438
//   a chunk beside 64 single tokens, 32/8 heads: 128 tokens (508) over 2000 keys 212 and
//     246, over 16000 333 and 277; 256 (1020) 325 and 246, 535 and 308; 448 (1788) over
//     8000 keys 518 and 294; 900 over 16000 keys beside 128 (3596) 1574 and 682; 512
//     beside 200 (2044, 14 rows on average) over 2000 keys 606 and 728, over 16000 1101
//     and 870
//   packed prompts, 32/8 heads: one of 2000 tokens beside 255 empty ones (6976) 592 and
//     50, one of 1000 (2976, 16 rows on average: it looks like 250 of 4) 225 and 28; 64
//     of 7 (1400) 35 and 27; 48 of 30, 8/8 heads of 64 (1373) 20 and 20
MBRS_RULE bool few_rows(int64_t tokens, int64_t batch, int64_t group) {
    const int64_t rows = tokens * group;
    return rows <= 16 * batch || (rows <= 32 * batch && rows - group * batch <= 1024);
}

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
