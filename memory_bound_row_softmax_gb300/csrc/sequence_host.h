// sequence_host.h -- host-side helpers of the sequence attention launchers.
#pragma once

#include <algorithm>
#include <atomic>
#include <numeric>

#include "launch.h"
#include "sequence.cuh"
#include "tensor_map.h"

namespace mbrs {
namespace seq {

inline uint32_t wait_limit(int64_t wait_ns) {
    return (uint32_t)std::min<int64_t>(std::max<int64_t>(wait_ns, 1), 0x7fffffff);
}

// The call's geometry for tiles of `keys` keys: a copy's rows lie in one page.
inline bool fill_geometry(const AttnCall &c, int keys, Geometry *g) {
    const softmax_sequence_args_t &a = c.a;
    g->starts = a.q_starts;
    g->lens = c.paged ? a.kv_lens : nullptr;
    g->table = c.paged ? a.page_table : nullptr;
    g->table_stride = a.table_stride;
    g->v = (const uint16_t *)a.v;
    g->v_page = c.paged ? a.v_page_stride : 0;
    g->v_token = a.v_token_stride;
    g->v_head = a.v_head_stride;
    g->o = (uint16_t *)a.o;
    g->lse = a.lse;
    g->o_token = a.o_token_stride;
    g->o_head = a.o_head_stride;
    g->pages = c.paged ? a.pages : 1;
    g->tokens = (int)a.tokens;
    g->batch = (int)a.batch;
    g->heads = (int)a.heads;
    g->kv_heads = (int)a.kv_heads;
    g->group = (int)(a.heads / a.kv_heads);
    g->page_size = c.paged ? (int)a.page_size : 1;
    g->max_keys = c.paged ? (int)(a.max_pages * a.page_size) : (int)a.tokens;
    g->box = c.paged ? (int)std::gcd<int64_t>(a.page_size, keys) : keys;
    g->causal = a.causal;
    g->kscale = a.sm_scale * kLog2e;
    return g->box % 8 == 0;
}

// A 4-D map (innermost first: head dim, rows, heads, pages) with boxes of 64
// columns x `box` rows, 128-byte swizzled.  Strides of dimensions of size 1 are
// not used; the encoder still wants them in range.
inline bool make_map(CUtensorMap *map, const void *ptr, const softmax_sequence_args_t &a, const int64_t dims[4],
                     const int64_t strides[3], const int box_in[4]) {
    const EncodeTiled enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t d[4], st[3];
    cuuint32_t box[4], estr[4] = {1, 1, 1, 1};
    for (int i = 0; i < 4; ++i) d[i] = (cuuint64_t)dims[i], box[i] = (cuuint32_t)box_in[i];
    for (int i = 0; i < 3; ++i) st[i] = (cuuint64_t)(dims[i + 1] > 1 ? strides[i] : dims[0]) * 2;
    return enc(map, a.dtype == SOFTMAX_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
               const_cast<void *>(ptr), d, st, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               dims[0] * 2 >= 256 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// K and V for copies of whole rows: a 5-D map (64 columns, rows, column blocks,
// heads, pages) whose boxes hold all of a head's columns, [column block][row] of
// 128-byte rows.
inline bool make_row_map(CUtensorMap *map, const void *ptr, const AttnCall &c, int box, int64_t token, int64_t head,
                         int64_t page) {
    const EncodeTiled enc = tensor_map_encoder();
    if (!enc) return false;
    const softmax_sequence_args_t &a = c.a;
    const cuuint64_t halves = (cuuint64_t)a.head_dim / 64;
    const cuuint64_t d[5] = {64, (cuuint64_t)(c.paged ? a.page_size : a.tokens), halves, (cuuint64_t)a.kv_heads,
                             (cuuint64_t)(c.paged ? a.pages : 1)};
    const cuuint64_t row = (cuuint64_t)a.head_dim * 2;
    const cuuint64_t st[4] = {d[1] > 1 ? (cuuint64_t)token * 2 : row, 128, d[3] > 1 ? (cuuint64_t)head * 2 : row,
                              d[4] > 1 ? (cuuint64_t)page * 2 : row};
    const cuuint32_t b[5] = {64, (cuuint32_t)box, (cuuint32_t)halves, 1, 1}, estr[5] = {1, 1, 1, 1, 1};
    return enc(map, a.dtype == SOFTMAX_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5,
               const_cast<void *>(ptr), d, st, b, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               halves > 1 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline bool make_kv_maps(const AttnCall &c, int box, CUtensorMap *tk, CUtensorMap *tv) {
    const softmax_sequence_args_t &a = c.a;
    const int64_t dims[4] = {a.head_dim, c.paged ? a.page_size : a.tokens, a.kv_heads, c.paged ? a.pages : 1};
    const int64_t ks[3] = {a.k_token_stride, a.k_head_stride, a.k_page_stride};
    const int64_t vs[3] = {a.v_token_stride, a.v_head_stride, a.v_page_stride};
    const int b[4] = {64, box, 1, 1};
    return make_map(tk, a.k, a, dims, ks, b) && make_map(tv, a.v, a, dims, vs, b);
}

// Of `blocks` blocks, those that equal stretches of the whole work can occupy: no
// stretch is shorter than COST + 1 (see find_stretch), and there are about
// `row_blocks` row blocks of at most max_keys keys at each kv head.  (Offsets that
// do not rise can make more of them; the stretches are then longer.)
inline int64_t blocks_with_work(const Geometry &g, int64_t row_blocks, int keys, int cost, int64_t blocks) {
    const int64_t items = row_blocks * g.kv_heads, tiles = std::max(1, (g.max_keys + keys - 1) / keys);
    if (items >= blocks) return blocks;
    return std::min(blocks, std::max<int64_t>(1, (items * (cost + tiles) + cost) / (cost + 1)));
}

// Dynamic shared memory beyond 48 KB, opted in once per kernel and device.
inline cudaError_t opt_in_shared_memory(const void *kernel, int bytes, std::atomic<unsigned long long> &opted) {
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = device < 64 ? 1ull << device : 0ull;
    if (bit && (opted.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) opted.fetch_or(bit, std::memory_order_acq_rel);
    return e;
}

// launch_kernel with a two-dimensional grid, on the call's stream.
template <typename... P, typename... A>
cudaError_t launch_kernel_2d(void (*kernel)(P...), const AttnCall &c, dim3 grid, int threads, A &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.stream = c.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = c.overlap ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<A &&>(args)...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace seq
}  // namespace mbrs
