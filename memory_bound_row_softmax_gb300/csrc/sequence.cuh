// sequence.cuh -- what the sequence attention kernels share: the batch's
// geometry as it is read on the device, the tensor maps, the waits, and the
// layout in shared memory.
#pragma once

#include <type_traits>

#include "attention.cuh"
#include "common.cuh"
#include "launch.h"
#include "sequence_launch.h"

namespace mbrs {
namespace seq {

// What every sequence attention kernel is given (host: fill_geometry).
struct Geometry {
    const int32_t *starts, *lens, *table;  // lens and table null: packed prompts
    int64_t table_stride;
    const uint16_t *v;                      // for the values read back in repair_values
    int64_t v_page, v_token, v_head;
    uint16_t *o;
    float *lse;
    int64_t o_token, o_head;
    int64_t pages;
    int tokens, batch, heads, kv_heads, group;  // group = heads / kv_heads
    int page_size, max_keys;                    // max_keys: max_pages * page_size
    int box;                                    // keys of one K or V copy
    int causal;
    float kscale;                               // sm_scale * log2 e
};

// One sequence: its rows of q and o, its keys.
struct Sequence {
    int start, n;  // first row, number of rows
    int keys;
};
// (Plain loads, here and in locate: these arrays may be written by the kernel that
// a launch overlaps, up to its griddepcontrol.wait, so they are not constant.)
__device__ __forceinline__ Sequence load_sequence(const Geometry &g, int b) {
    Sequence s;
    s.start = min(max(g.starts[b], 0), g.tokens);
    const int end = min(max(g.starts[b + 1], s.start), g.tokens);
    s.n = end - s.start;
    s.keys = g.lens ? min(max(g.lens[b], 0), g.max_keys) : s.n;
    return s;
}
// a / b, a >= 0, b > 0.  Most are small: a 64-bit division takes some 250 cycles,
// and a block does several, one after the other, before its first copy (0.5 to 1 us
// of a short call of the tile kernel).
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    return ((uint64_t)(a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
// Keys that query i of a sequence keeps: [0, kept).
__device__ __forceinline__ int kept_keys(const Geometry &g, const Sequence &s, int i) {
    return g.causal ? max(s.keys - s.n + i + 1, 0) : s.keys;
}

// Index arrays towards L2, before the wait on the previous kernel (a hint: what
// the loads after it return does not change).  Every block names the small ones,
// and its share of the page table.
__device__ __forceinline__ void prefetch_line(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
__device__ __forceinline__ void prefetch_indices(const Geometry &g) {
    constexpr int kLine = 32;  // int32 in a 128-byte line
    for (int i = (int)threadIdx.x * kLine; i <= g.batch; i += (int)blockDim.x * kLine) prefetch_line(g.starts + i);
    if (!g.table) return;
    for (int i = (int)threadIdx.x * kLine; i < g.batch; i += (int)blockDim.x * kLine) prefetch_line(g.lens + i);
    const int64_t entries = (int64_t)(g.batch - 1) * g.table_stride + g.max_keys / g.page_size;
    const int64_t step = (int64_t)gridDim.x * blockDim.x * kLine;
    int64_t i = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * kLine;
    for (int n = 0; n < 4 && i < entries; ++n, i += step) prefetch_line(g.table + i);
}

// ---------------------------------------------------------------------------
// The order of work.  An item is a block of `rows` query rows (row r of a
// sequence: token r / group, head r % group) of one sequence at one key/value
// head, with its keys in tiles of KEYS.  An item's work is COST plus its tiles:
// what it costs to begin and end one, in tiles' time.  The work of all items, in
// the order (sequence, row block, kv head), is what the blocks of a grid share.
// ---------------------------------------------------------------------------
__device__ __forceinline__ int row_blocks(const Geometry &g, const Sequence &s, int rows) {
    return (int)quotient((int64_t)s.n * g.group + rows - 1, rows);
}
// Keys that some row of block rb keeps: those of its last row.
__device__ __forceinline__ int block_keys(const Geometry &g, const Sequence &s, int rb, int rows) {
    const int64_t last = min((int64_t)(rb + 1) * rows, (int64_t)s.n * g.group) - 1;
    return kept_keys(g, s, (int)quotient(last, g.group));
}
// at least one: an item without keys still writes its rows
template <int KEYS> __device__ __forceinline__ int tiles_of(int keys) { return max(1, (keys + KEYS - 1) / KEYS); }
// The work of row blocks lo .. hi - 1.
template <int KEYS, int COST>
__device__ __forceinline__ int64_t work_of(const Geometry &g, const Sequence &s, int lo, int hi, int rows) {
    int64_t t = 0;
    if (!g.causal) {
        t = (int64_t)(hi - lo) * (COST + tiles_of<KEYS>(s.keys));
    } else {
        for (int rb = lo; rb < hi; ++rb) t += COST + tiles_of<KEYS>(block_keys(g, s, rb, rows));
    }
    return t * g.kv_heads;
}

// A place in that order: `at` is how much of the item's work lies before it.
struct Place {
    int b, rb, h, at;
};
// To the next item (sequences without rows are passed over).
__device__ __forceinline__ void next_item(const Geometry &g, Place &p, Sequence &s, int rows) {
    p.at = 0;
    if (++p.h < g.kv_heads) return;
    p.h = 0;
    if (++p.rb < row_blocks(g, s, rows)) return;
    p.rb = 0;
    do {
        if (++p.b >= g.batch) return;
        s = load_sequence(g, p.b);
    } while (s.n == 0);
}

// What a stretch with `left` work to go takes of the item at `p`: key tiles
// [t0, t1), none if the stretch ends within the item's COST.
struct Piece {
    int count, t0, t1, tiles;  // count: the work taken
    __device__ bool empty() const { return t1 <= t0; }
    __device__ bool whole() const { return t0 == 0 && t1 == tiles; }
    // the part it writes if it is not whole: each block has one that continues
    // an item and one that begins one
    __device__ int part() const { return 2 * (int)blockIdx.x + (t0 == 0 ? 1 : 0); }
};
template <int KEYS, int COST>
__device__ __forceinline__ Piece take_piece(const Geometry &g, const Sequence &s, const Place &p, int rows, int64_t left) {
    Piece r;
    r.tiles = tiles_of<KEYS>(block_keys(g, s, p.rb, rows));
    r.count = (int)min(left, (int64_t)(COST + r.tiles - p.at));
    r.t0 = max(p.at - COST, 0);
    r.t1 = max(p.at + r.count - COST, 0);
    return r;
}
// The record of an item that begins in this block and ends in another: its
// last block.  `pos` is the place's position in the order.
template <int COST>
__device__ __forceinline__ int last_block(const Piece &c, const Place &p, int64_t pos, int64_t stretch) {
    return (int)quotient(pos - p.at + COST + c.tiles - 1, stretch);
}

// This block's stretch [first, first + mine) of all work, cut evenly over the
// grid, and the place it begins at.  Thread t counts the work of some consecutive
// sequences, or of some consecutive row blocks of one (so that a long sequence does
// not wait for one thread: 1184 causal tokens, 37 row blocks of 24/3 heads, 33.1 ->
// 20.0 us); a scan over the threads finds whose count the stretch begins in.  (A
// larger least stretch spares the join parts, but leaves a batch of many short
// sequences on few blocks: two tiles instead of one, 10.5 -> 13.8 us for 25 prompts
// of 42 tokens at most.)  Called by all THREADS threads; `scratch` is kScanBytes of 16-byte
// aligned shared memory.
constexpr int kScanBytes = 16 + 8 * 32;
struct Stretch {
    int64_t size, first, mine;
    Place at;
};
template <int KEYS, int COST, int THREADS>
__device__ __forceinline__ Stretch find_stretch(const Geometry &g, int rows, uint8_t *scratch) {
    int4 *const place = reinterpret_cast<int4 *>(scratch);
    int64_t *const scan = reinterpret_cast<int64_t *>(scratch + 16);
    const int warp = (int)(threadIdx.x >> 5), lane = (int)(threadIdx.x & 31);
    const int each = (g.batch + THREADS - 1) / THREADS;       // sequences to a thread
    const int split = each == 1 ? THREADS / g.batch : 1;      // threads to a sequence
    const int nth = (int)threadIdx.x / split, share = (int)threadIdx.x - nth * split;
    const int b_lo = (int)min((int64_t)nth * each, (int64_t)g.batch), b_hi = min(b_lo + each, g.batch);
    Sequence s{};            // the last of the thread's sequences,
    int lo = 0, hi = 0;      // and its row blocks there
    const auto enter = [&](int b) {
        s = load_sequence(g, b);
        const int nb = row_blocks(g, s, rows), per = (nb + split - 1) / split;
        lo = min(share * per, nb), hi = min(lo + per, nb);
        return work_of<KEYS, COST>(g, s, lo, hi, rows);
    };
    int64_t own = 0;
    for (int b = b_lo; b < b_hi; ++b) own += enter(b);
    int64_t upto = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) scan[warp] = upto;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) upto += scan[w];
        total += scan[w];
    }
    Stretch r;
    r.size = max(quotient(total + gridDim.x - 1, gridDim.x), (int64_t)(COST + 1));
    r.first = (int64_t)blockIdx.x * r.size;
    r.mine = min(r.size, total - r.first);
    if (r.mine > 0 && r.first >= upto - own && r.first < upto) {
        int64_t rest = r.first - (upto - own);
        int b = b_lo;
        if (each > 1) {
            int64_t n;
            while (rest >= (n = enter(b))) rest -= n, ++b;
        }
        int t = COST + tiles_of<KEYS>(block_keys(g, s, lo, rows));
        while (rest >= (int64_t)t * g.kv_heads) {
            rest -= (int64_t)t * g.kv_heads;
            t = COST + tiles_of<KEYS>(block_keys(g, s, ++lo, rows));
        }
        const int h = (int)quotient(rest, t);
        *place = make_int4(b, lo, h, (int)(rest - (int64_t)h * t));
    }
    __syncthreads();
    const int4 at = *place;
    r.at = Place{at.x, at.y, at.z, at.w};
    return r;
}

// Where key j of sequence b lies: a page (or the one run of packed rows) and
// the row in it.  A packed key is row start + j of page 0.
__device__ __forceinline__ int2 locate(const Geometry &g, const Sequence &s, int b, int j) {
    if (!g.table) return make_int2(0, s.start + j);
    const uint32_t entry = (uint32_t)j / (uint32_t)g.page_size;
    return make_int2(g.table[b * g.table_stride + entry], (int)((uint32_t)j - entry * (uint32_t)g.page_size));
}

// Tiled 4-D TMA load (coordinates innermost first); see attn::tma_load_3d.
// Elements outside the tensor (a page index that is none among them) read as
// zero.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int32_t x, int32_t y, int32_t z,
                                            int32_t w, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
        "%4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}

// The same in five dimensions.
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap *map, int32_t x, int32_t y, int32_t z,
                                            int32_t w, int32_t u, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
        "%4, %5, %6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(u), "r"(bar)
        : "memory");
}

// Writes of earlier kernels to global memory, seen by this thread, before its
// copies through the async proxy.
__device__ __forceinline__ void fence_proxy_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }

// A wait for phase `parity` of an mbarrier that gives up after limit_ns or
// once the block's abort flag is set; running out sets both the flag and the
// device error word.
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, volatile uint32_t *abort_flag,
                                           unsigned int *error_word, uint32_t limit_ns) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint32_t t0 = global_timer_lo();
    for (uint32_t it = 0; it < (1u << 30); ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        if (global_timer_lo() - t0 > limit_ns) break;
    }
    *abort_flag = 1u;
    atomicOr(error_word, kErrWaitTimeout);
    return false;
}
// The same for copies or products already in flight, which must end before
// the block lets go of its memory: the abort flag does not cut it short.
__device__ __forceinline__ void drain_phase(uint32_t bar, uint32_t parity, volatile uint32_t *abort_flag,
                                            unsigned int *error_word, uint32_t limit_ns) {
    if (mbar_try_wait(bar, parity)) return;
    const uint32_t t0 = global_timer_lo();
    for (uint32_t it = 0; it < (1u << 30); ++it) {
        if (mbar_try_wait(bar, parity)) return;
        if (global_timer_lo() - t0 > limit_ns) break;
    }
    *abort_flag = 1u;
    atomicOr(error_word, kErrWaitTimeout);
}

// How far a row's shift lies below the max that set it, in log2 units: a key of score x
// weighs P = 2^(x k - shift), rounded to the type for the second product.  fp16 loses
// bits below 2^-14 and everything below 2^-25, while many such keys (131000 of 2^-25
// beside one of 1: 0.004 of the row) count in the fp32 sum; with the max at 2^7, and at
// 2^15 where the shift lags behind by kShiftSlack, nothing is lost above 2^-32.  bf16
// has the range of fp32.
constexpr float kShiftSlack = 8.f;  // log2 units: the shift moves when a tile's max exceeds its own by this
template <typename T> constexpr float kShiftBelow = std::is_same<T, __half>::value ? 7.f : 0.f;

// The logarithm of a row's sum from its (shift, sum) state: the shift in log2
// units, the sum relative to it.
__device__ __forceinline__ float natural_lse(float shift, float sum) {
    return sum == 0.f ? -INFINITY : (shift + log2f(sum)) * 0.6931471805599453f;
}

template <typename T> __device__ __forceinline__ uint32_t pack2(float a, float b) { return Elem<T>::unpair(a, b); }

// x * 0 of two packed 16-bit values added to acc: a half of the result is NaN
// once an infinity or NaN has gone in, else zero.
template <typename T> __device__ __forceinline__ uint32_t add_times_zero(uint32_t acc, uint32_t x) {
    uint32_t r;
    if constexpr (std::is_same<T, __half>::value)
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(acc));
    else
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(acc));
    return r;
}
// Infinite and NaN halves of a packed pair are set to zero.
template <typename T> __device__ __forceinline__ constexpr uint32_t exponent_bits() {
    return std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
}
template <typename T> __device__ __forceinline__ uint32_t finite_or_zero(uint32_t w) {
    constexpr uint32_t e = exponent_bits<T>();
    if ((w & e) == e) w &= 0xffff0000u;
    if ((w & (e << 16)) == (e << 16)) w &= 0x0000ffffu;
    return w;
}

}  // namespace seq
}  // namespace mbrs
