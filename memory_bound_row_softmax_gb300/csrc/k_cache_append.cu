// k_cache_append.cu -- new keys and values into the paged cache, the keys (and
// the queries, if given) rotated by their positions on the way.
//
// Pair m of a head turns by the angle p * inv_freq[m] at position p:
//     (x, y) -> (x cos - y sin, y cos + x sin).
// The angle is formed and reduced to turns in 64 bits (at p = 10^6 an angle in
// fp32 is off by up to 2^-5 rad), its sine and cosine and the rotation are fp32,
// and each element is rounded once.
//
// Every element is read once and written once, so HBM bounds it.  A block takes
// one token: its heads share the token's sines and cosines (computed once, by
// rotary_dim / 2 threads, kept in shared memory).  A thread moves two 16-byte
// vectors at a time: the two that hold a pair's halves, or neighbours where
// pairs are neighbours or nothing is rotated.  The first vectors are loaded
// before the token's sequence is looked up, so that the lookup (one count over
// q_starts) and the sines hide behind them.
#include "common.cuh"
#include "sequence_launch.h"
#include "launch.h"

namespace mbrs {
namespace seq {
namespace {

// Measured on 16,298 tokens of 32/8 heads of 128 (401 MB; a copy of as many bytes
// takes 64 us): 256 threads 68.6 us, 128 threads 61.3 us, 64 threads 62.8 us; of
// head dim 64: 49, 34 and 33 us.  Smaller blocks leave fewer warps at the barriers.
constexpr int kThreads = 128;
constexpr int kEarly = 2;  // vector pairs per thread loaded before the lookup

struct Params {
    const uint16_t *k, *v, *q;
    uint16_t *k_cache, *v_cache, *q_out;
    const int32_t *starts, *lens, *table;
    const float *inv_freq;
    int64_t kt, kh, vt, vh, qt, qh, ot, oh;
    int64_t kcp, kct, kch, vcp, vct, vch;
    int64_t table_stride;
    int64_t pages, max_pages;
    uint32_t page_size;
    int batch, heads, kv_heads, half;  // half = rotary_dim / 2
};

// Unit u of a head: the 16-byte vectors it moves.
template <bool INTERLEAVED>
__device__ __forceinline__ int2 unit_vectors(int u, int half, bool rotates) {
    if (INTERLEAVED || !rotates) return make_int2(2 * u, 2 * u + 1);
    const int h8 = half >> 3;
    if (u < h8) return make_int2(u, u + h8);
    const int first = 2 * h8 + 2 * (u - h8);
    return make_int2(first, first + 1);
}

template <typename T, int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) k_cache_append(const Params p) {
    constexpr int kUnits = D / 16;  // units of two vectors in a head
    __shared__ float s_cos[D / 2], s_sin[D / 2];
    pdl_enter();
    const int64_t token = blockIdx.x;
    const int rows = p.heads + 2 * p.kv_heads;  // the token's query, key and value heads
    const int total = rows * kUnits;

    const auto source = [&](int i, int2 &vec) -> const uint4 * {
        const int row = i / kUnits, u = i % kUnits;
        vec = unit_vectors<INTERLEAVED>(u, p.half, row < p.heads + p.kv_heads);
        const uint16_t *s = row < p.heads ? p.q + token * p.qt + row * p.qh
                            : row < p.heads + p.kv_heads
                                ? p.k + token * p.kt + (row - p.heads) * p.kh
                                : p.v + token * p.vt + (row - p.heads - p.kv_heads) * p.vh;
        return reinterpret_cast<const uint4 *>(s);
    };
    uint4 early[kEarly][2];
#pragma unroll
    for (int e = 0; e < kEarly; ++e) {
        const int i = (int)threadIdx.x + e * kThreads;
        if (i < total) {
            int2 vec;
            const uint4 *s = source(i, vec);
            early[e][0] = s[vec.x];
            early[e][1] = s[vec.y];
        }
    }

    // the token's sequence: the last one that starts at or before it
    int at_or_before = 0;
    for (int b0 = 0; b0 <= p.batch; b0 += kThreads) {
        const int b = b0 + (int)threadIdx.x;
        at_or_before += __syncthreads_count(b <= p.batch && (int64_t)p.starts[b] <= token);
    }
    const int b = at_or_before - 1;
    if (b < 0 || b >= p.batch) return;  // a row of no sequence
    const int64_t end = min((int64_t)p.starts[b + 1], (int64_t)gridDim.x);
    if (token >= end) return;
    const int64_t pos = (int64_t)p.lens[b] - end + token;
    if ((int)threadIdx.x < p.half) {
        // the angle in turns, reduced to [-1/2, 1/2]
        const double turns = (double)pos * (double)p.inv_freq[threadIdx.x] * 0.15915494309189533577;
        float sn, cs;
        sincospif((float)(2.0 * (turns - rint(turns))), &sn, &cs);
        s_cos[threadIdx.x] = cs;
        s_sin[threadIdx.x] = sn;
    }
    int64_t page = -1;
    uint32_t slot = 0;
    if (pos >= 0) {  // below 2^31: a length less a distance
        const uint32_t entry = (uint32_t)pos / p.page_size;
        slot = (uint32_t)pos % p.page_size;
        if (entry < p.max_pages) page = p.table[b * p.table_stride + entry];
    }
    const bool kept = page >= 0 && page < p.pages;
    __syncthreads();

    const auto put = [&](int i, uint4 a, uint4 c) {
        const int row = i / kUnits, u = i % kUnits;
        const bool is_q = row < p.heads, is_k = !is_q && row < p.heads + p.kv_heads;
        const int2 vec = unit_vectors<INTERLEAVED>(u, p.half, is_q || is_k);
        uint16_t *dst;
        if (is_q) {
            dst = p.q_out + token * p.ot + row * p.oh;
        } else if (!kept) {
            return;
        } else if (is_k) {
            dst = p.k_cache + page * p.kcp + slot * p.kct + (row - p.heads) * p.kch;
        } else {
            dst = p.v_cache + page * p.vcp + slot * p.vct + (row - p.heads - p.kv_heads) * p.vch;
        }
        if (is_q || is_k) {
            if (INTERLEAVED) {
                float x[8], y[8];
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const int m0 = (w ? vec.y : vec.x) * 4;  // the vector's first pair
                    if (m0 < p.half) {
                        Elem<T>::unpack(w ? c : a, x);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float cs = s_cos[m0 + e], sn = s_sin[m0 + e];
                            y[2 * e] = x[2 * e] * cs - x[2 * e + 1] * sn;
                            y[2 * e + 1] = x[2 * e + 1] * cs + x[2 * e] * sn;
                        }
                        (w ? c : a) = Elem<T>::pack(y);
                    }
                }
            } else if (u < (p.half >> 3)) {
                float x[8], y[8], xr[8], yr[8];
                Elem<T>::unpack(a, x);
                Elem<T>::unpack(c, y);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float cs = s_cos[8 * u + e], sn = s_sin[8 * u + e];
                    xr[e] = x[e] * cs - y[e] * sn;
                    yr[e] = y[e] * cs + x[e] * sn;
                }
                a = Elem<T>::pack(xr);
                c = Elem<T>::pack(yr);
            }
        }
        uint4 *d = reinterpret_cast<uint4 *>(dst);
        d[vec.x] = a;
        d[vec.y] = c;
    };
#pragma unroll
    for (int e = 0; e < kEarly; ++e) {
        const int i = (int)threadIdx.x + e * kThreads;
        if (i < total) put(i, early[e][0], early[e][1]);
    }
    for (int i = (int)threadIdx.x + kEarly * kThreads; i < total; i += kThreads) {
        int2 vec;
        const uint4 *s = source(i, vec);
        const uint4 a = s[vec.x], c = s[vec.y];
        put(i, a, c);
    }
}

template <typename T, int D, bool INTERLEAVED>
cudaError_t go(const Params &p, int64_t tokens, int overlap, cudaStream_t stream) {
    LaunchArgs l = {};
    l.stream = stream;
    l.overlap = overlap;
    return launch_kernel(k_cache_append<T, D, INTERLEAVED>, l, tokens, kThreads, 0, 0, p);
}

template <typename T, int D>
cudaError_t go_pairs(const Params &p, int64_t tokens, bool interleaved, int overlap, cudaStream_t stream) {
    return interleaved ? go<T, D, true>(p, tokens, overlap, stream) : go<T, D, false>(p, tokens, overlap, stream);
}

}  // namespace

cudaError_t launch_append(const softmax_append_args_t &a, int overlap, cudaStream_t stream) {
    Params p;
    p.k = (const uint16_t *)a.k;
    p.v = (const uint16_t *)a.v;
    p.q = (const uint16_t *)a.q;
    p.k_cache = (uint16_t *)a.k_cache;
    p.v_cache = (uint16_t *)a.v_cache;
    p.q_out = (uint16_t *)a.q_out;
    p.starts = a.q_starts;
    p.lens = a.kv_lens;
    p.table = a.page_table;
    p.inv_freq = a.inv_freq;
    p.kt = a.k_token_stride, p.kh = a.k_head_stride, p.vt = a.v_token_stride, p.vh = a.v_head_stride;
    p.qt = a.q_token_stride, p.qh = a.q_head_stride, p.ot = a.q_out_token_stride, p.oh = a.q_out_head_stride;
    p.kcp = a.k_cache_page_stride, p.kct = a.k_cache_token_stride, p.kch = a.k_cache_head_stride;
    p.vcp = a.v_cache_page_stride, p.vct = a.v_cache_token_stride, p.vch = a.v_cache_head_stride;
    p.table_stride = a.table_stride;
    p.pages = a.pages, p.max_pages = a.max_pages, p.page_size = (uint32_t)a.page_size;
    p.batch = (int)a.batch;
    p.heads = a.q ? (int)a.heads : 0;
    p.kv_heads = (int)a.kv_heads;
    p.half = a.inv_freq ? (int)(a.rotary_dim / 2) : 0;
    const bool il = a.interleaved != 0;
    if (a.dtype == SOFTMAX_BF16)
        return a.head_dim == 128 ? go_pairs<__nv_bfloat16, 128>(p, a.tokens, il, overlap, stream)
                                 : go_pairs<__nv_bfloat16, 64>(p, a.tokens, il, overlap, stream);
    return a.head_dim == 128 ? go_pairs<__half, 128>(p, a.tokens, il, overlap, stream)
                             : go_pairs<__half, 64>(p, a.tokens, il, overlap, stream);
}

}  // namespace seq
}  // namespace mbrs
