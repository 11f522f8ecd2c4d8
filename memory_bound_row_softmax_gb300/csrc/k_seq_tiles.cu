// k_seq_tiles.cu -- attention of many query rows on the fifth-generation
// tensor cores: packed prompts, and chunks of new tokens over a paged cache.
//
// The rows of an item are up to 256 (token, head) pairs of one sequence that
// share one key/value head: two tiles A and B of 128 / group tokens times
// `group` heads, so K and V are loaded once for the whole group and the last,
// partly masked tiles are narrow in tokens.  Keys go by in tiles of 128:
//     S_t = Q_t K^T (TMEM)  ->  P_t = 2^(S_t k - m)  (TMEM, 16 bits)  ->  O_t += P_t V (TMEM)
// with the running shift m and sum l of a row in its thread's registers, and
// O_t / l written once.  The arithmetic is the dense kernel's (k_attention.cu:
// lazy shift, packed fp32 pairs).  What bounds it is the tensor pipe (78 % active
// on 8192 tokens of 32/8 heads of 128 without a mask: 619 us under the profiler, at
// 1.90 GHz, 629-644 us or 1707-1748 TFLOP/s in calls): a pair of tiles takes 2600
// cycles, 2048 of them products, and each group's softmax, 1110 between its S and its
// P, hides behind the other's products.  With head dim 64 the products are half, 1024
// a pair of tiles, and the thread that issues them is what is left: it serves both
// groups, 1100 cycles a tile and so 2200 a pair, where the groups' softmax, side by
// side, takes 1200.  Three S buffers, and one wait per tile landed, took 4 x 2048
// tokens of 16 heads of 64 from 89.7 to 82.5 us (833 TFLOP/s; 78-80 on another GB300),
// and from 59.7 to 55.1 us with the causal mask.
//
// Threads: warps 0-3 and 4-7 are the softmax groups of tiles A and B (thread r
// = row r = TMEM lane r); warp 8 fetches work and feeds TMA, one lane per copy
// (a copy: rows of one page, 64 columns, 128-byte swizzled); warp 9 issues the
// products.  One block per SM, persistent.
//
// Work: with many items (at least kItemsPerSm per SM) k_tiles_plan sorts the
// items by their key tiles and the blocks take them longest first from a
// counter; nothing is cut.  With few, or where one item is longer than an SM's
// fair share or the last wave would idle for long, each block takes an equal
// stretch of all work (find_stretch), and k_tiles_join merges the parts of the
// items that were cut, in order.
//
// Masked values (infinite or NaN) are taken out of the V tiles some row does
// not keep whole and added back to the rows that do keep them, as in
// k_seq_rows.cu.
//
// Every wait is bounded: one that runs out sets the device error word and an
// abort flag, outstanding copies and products are waited for (bounded), TMEM
// is released and the block returns.
#include <type_traits>

#include "attention_launch.h"
#include "launch.h"
#include "sequence.cuh"
#include "sequence_host.h"
#include "sequence_rules.h"

namespace mbrs {
namespace seq {

__device__ unsigned int g_tiles_error;

namespace {

using namespace attn;

constexpr int kTile = 128;     // rows of a query tile, keys of a key tile
constexpr int kThreads = 320;
constexpr int kWarpTma = 8, kWarpMma = 9;
constexpr int kItemsPerSm = 2;
constexpr int kItemCost = 2;   // beginning and ending an item, in tiles' time (about 2.4 us of 1.4 us each)
// Key tiles of an item that hold keys some row of it does not keep: its rows'
// kept keys end within 256 tokens of each other.
constexpr int kEdgeTiles = 3;

template <int D>
struct Layout {
    static constexpr int kSlots = D == 128 ? 4 : 8;              // K/V ring
    // Tensor memory, 512 columns: S tiles (P_t over the first 64 of each), then O_a and
    // O_b.  With head dim 64 there is room for a third S: see step_of.
    static constexpr int kBuffers = D == 128 ? 2 : 3;
    static constexpr uint32_t kColO = 128 * kBuffers;
    static constexpr uint32_t kHalf = kTile * 128;               // 64 columns of a tile: 128 rows of 128 bytes
    static constexpr uint32_t kTileBytes = kHalf * (D / 64);
    // from a 1024-byte aligned base
    static constexpr uint32_t kOffQ = 0;                         // Q_t at t kTileBytes
    static constexpr uint32_t kOffRing = 2 * kTileBytes;
    static constexpr uint32_t kOffStage = kOffRing + kSlots * kTileBytes;  // a warp's 32 rows of 64 columns of O
    static constexpr uint32_t kOffBar = kOffStage + 8 * 4096;
    static constexpr int kBarQ = 0, kBarQEmpty = 1, kBarUnit = 2, kBarRead = 3, kBarDrain = 4, kBarO = 5,
                         kBarS = 7, kBarP = 7 + kBuffers, kBarDone = 7 + 2 * kBuffers, kBarFull = 7 + 3 * kBuffers,
                         kBarEmpty = kBarFull + kSlots, kNumBars = kBarEmpty + kSlots;
    static constexpr uint32_t kOffUnits = (kOffBar + kNumBars * 8 + 15) / 16 * 16;  // two units
    static constexpr uint32_t kOffScan = kOffUnits + 2 * 64;
    static constexpr uint32_t kOffTmem = kOffScan + kScanBytes;
    static constexpr uint32_t kOffAbort = kOffTmem + 4;
    static constexpr uint32_t kOffBad = (kOffAbort + 4 + 15) / 16 * 16;  // per ring entry of units
    static constexpr size_t kBytes = kOffBad + 2 * 16 * kEdgeTiles + 1024;
};
static_assert(Layout<128>::kBytes <= 227 * 1024 && Layout<64>::kBytes <= 227 * 1024, "shared memory per block");
constexpr uint32_t kTmemCols = 512;
static_assert(Layout<128>::kColO + 2 * 128 <= kTmemCols && Layout<64>::kColO + 2 * 64 <= kTmemCols, "tensor memory");
__host__ __device__ constexpr uint32_t col_s(int buffer) { return 128u * (uint32_t)buffer; }
template <int D> __host__ __device__ constexpr uint32_t col_o(int t) {
    return Layout<D>::kColO + (uint32_t)(D * t);
}

// The steps of a unit: tile j of group A, tile j of group B, tile j + 1 of A, ...;
// where one group has fewer tiles, the other's follow one another.  With three buffers
// step i of the block has S and P in buffer i mod 3.
__device__ __forceinline__ int step_of(int n_a, int n_b, int t, int j) {
    const int both = min(n_a, n_b);
    return j < both ? 2 * j + t : both + j;
}

// What a block works on next: key tiles [j0, j0 + n_t) of the item's tile t.
struct Unit {
    int b, h;       // sequence (-1: no more work), kv head
    int start, i0;  // the sequence's first row, the item's first token in the sequence
    int n, keys;    // the sequence's tokens and keys
    int j0, n_a, n_b;
    int part;       // where the part's state goes; -1: the item is whole
    int kept_all;   // keys that every row of the item keeps
    int load;       // loads of the block before this unit's
    int step;       // steps of the block before this unit's
    int s[2];       // S tiles of each query tile before this unit's
    int o;          // bit t: parity of the O tiles of group t before this unit's
};
static_assert(sizeof(Unit) == 64, "two units in shared memory");

struct TilesParams {
    Geometry g;
    int tile_tokens;         // tokens of a query tile: 128 / group
    unsigned int *plan;      // {next unit, units, 1: cut into stretches}; null: cut
    const int4 *entries;     // two per planned row block: {sequence, row block, start, n}, {keys}
    int head_group;          // kv heads whose keys and values share L2
    int4 *records;           // per block: the cut item that begins in it
    float2 *states;          // [part][tile][row]
    float *parts;            // [part][tile][D / 4][row][4]
    uint32_t wait_ns;
    int starve;              // test hook: leave the first Q barrier unarmed
};

__device__ __forceinline__ Unit make_unit(const TilesParams &p, const Sequence &s, int b, int rb, int h, int j0, int count,
                                          int part) {
    const Geometry &g = p.g;
    Unit u;
    u.b = b, u.h = h, u.start = s.start, u.n = s.n, u.keys = s.keys;
    u.i0 = rb * 2 * p.tile_tokens;
    u.j0 = j0, u.part = part;
    const auto tiles = [&](int t) {  // key tiles of query tile t in [j0, j0 + count)
        const int first = u.i0 + t * p.tile_tokens;
        if (first >= s.n) return 0;
        const int kept = kept_keys(g, s, min(first + p.tile_tokens, s.n) - 1);
        return min(max((kept + kTile - 1) / kTile - j0, 0), count);
    };
    u.n_a = tiles(0);
    u.n_b = tiles(1);
    u.kept_all = kept_keys(g, s, u.i0);
    return u;
}

// Thread r of a softmax group looks over key r's values, row `v` of a V tile
// (`sw`: its place in the swizzle atom): x * 0 summed is NaN once one of them is
// infinite or NaN.  Such values are set to zero, the key's bit in the tile's mask
// `bad` first: whoever finds the zero finds the bit.  Rows past the last key
// (leftovers in shared memory) get no bit.  The fence comes last on every path, before
// the group lets its product read the tile: the other group looks at the same tile, so
// a thread that finds nothing bad may have found that group's zeros, which the product
// (async proxy) is sure to read only past a fence of this thread's.
template <typename T, int D>
__device__ __forceinline__ void zero_bad_values(uint8_t *v, int sw, uint32_t *bad, int r, bool real) {
    constexpr uint32_t kHalf = Layout<D>::kHalf;
    uint32_t acc[2] = {0u, 0u};
#pragma unroll
    for (int c = 0; c < D / 8; ++c) {
        const uint4 w = *reinterpret_cast<const uint4 *>(v + (c >> 3) * kHalf + (((c & 7) ^ sw) << 4));
        acc[0] = add_times_zero<T>(add_times_zero<T>(acc[0], w.x), w.y);
        acc[1] = add_times_zero<T>(add_times_zero<T>(acc[1], w.z), w.w);
    }
    if ((acc[0] | acc[1]) & 0x7fff7fffu) {
        if (real) {
            atomicOr(bad + (r >> 5), 1u << (r & 31));
            __threadfence_block();
        }
#pragma unroll 1
        for (int c = 0; c < D / 8; ++c) {
            uint4 *const w = reinterpret_cast<uint4 *>(v + (c >> 3) * kHalf + (((c & 7) ^ sw) << 4));
            *w = make_uint4(finite_or_zero<T>(w->x), finite_or_zero<T>(w->y), finite_or_zero<T>(w->z),
                            finite_or_zero<T>(w->w));
        }
    }
    mbrs::fence_proxy_async_smem();
}

// The values set to zero, added back to a row that keeps their keys [from, upto),
// as the caller's memory has them: `bad` holds the masks of the key tiles from
// from / 128 rounded down to `tile0` on.  The row has been written, to `o` or to
// its part's columns of four; added to an infinity or NaN it is one whatever it
// was.  (Out of line: rare work, kept out of the registers of the softmax loop.)
template <typename T, int D>
__device__ __noinline__ void add_bad_values(const Geometry &g, const Sequence &s, int b, int h, int tile0,
                                            const uint32_t *bad, int from, int upto, uint16_t *o, float *part) {
#pragma unroll 1
    for (int w = 0; w < 4 * kEdgeTiles; ++w) {
        for (uint32_t bits = *(const volatile uint32_t *)(bad + w); bits; bits &= bits - 1) {
            const int j = tile0 * kTile + 32 * w + __ffs((int)bits) - 1;
            if (j < from || j >= upto) continue;
            const int2 place = locate(g, s, b, j);
            if (place.x < 0 || place.x >= g.pages) continue;
            const uint16_t *v = g.v + place.x * g.v_page + place.y * g.v_token + h * g.v_head;
#pragma unroll 1
            for (int c = 0; c < D / 8; ++c) {
                const uint4 four = *reinterpret_cast<const uint4 *>(v + 8 * c);
                const uint32_t pairs[4] = {four.x, four.y, four.z, four.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (finite_or_zero<T>(pairs[e]) == pairs[e]) continue;
                    const float2 f = Elem<T>::pair(pairs[e] ^ finite_or_zero<T>(pairs[e]));  // its finite half as 0
                    const int d = 8 * c + 2 * e;
                    if (o) {
                        const float2 x = Elem<T>::pair(*reinterpret_cast<const uint32_t *>(o + d));
                        *reinterpret_cast<uint32_t *>(o + d) = pack2<T>(x.x + f.x, x.y + f.y);
                    } else {
                        float *const x = part + (int64_t)(d / 4) * kTile * 4 + d % 4;
                        x[0] += f.x, x[1] += f.y;
                    }
                }
            }
        }
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    k_seq_tiles(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                const __grid_constant__ CUtensorMap tv, const __grid_constant__ TilesParams p) {
    using L = Layout<D>;
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr int kHalves = D / 64;
    constexpr bool kAhead = L::kBuffers == 3;  // S a step ahead of its group
    const Geometry &g = p.g;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *const gbase = smem_raw + (base - raw);
    volatile uint32_t *const abort_flag = reinterpret_cast<volatile uint32_t *>(gbase + L::kOffAbort);
    // unit k's masks of keys with infinite or NaN values, from its first edge tile on
    const auto bad_keys = [gbase](int k) {
        return reinterpret_cast<uint32_t *>(gbase + L::kOffBad) + 4 * kEdgeTiles * (k & 1);
    };
    volatile Unit *const units = reinterpret_cast<volatile Unit *>(gbase + L::kOffUnits);
    const auto bar = [base](int i) { return base + L::kOffBar + 8u * (uint32_t)i; };
    const auto wait = [&](int i, int phase) {
        return wait_phase(bar(i), (uint32_t)phase & 1u, abort_flag, &g_tiles_error, p.wait_ns);
    };
    const auto drain = [&](int i, int phase) {
        drain_phase(bar(i), (uint32_t)phase & 1u, abort_flag, &g_tiles_error, p.wait_ns);
    };
    const int warp = (int)(threadIdx.x >> 5), lane = (int)(threadIdx.x & 31);

    if (threadIdx.x == 0) {
        for (int i = 0; i < L::kNumBars; ++i)
            mbar_init(bar(i), i >= L::kBarP && i < L::kBarP + L::kBuffers ? 4 : i == L::kBarRead ? 9 : 1);
        *abort_flag = 0u;
        fence_mbar_init();
        tma_prefetch_desc(&tq);
        tma_prefetch_desc(&tk);
        tma_prefetch_desc(&tv);
    }
    if (warp == kWarpMma) {
        tmem_alloc(base + L::kOffTmem, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(gbase + L::kOffTmem);
    pdl_enter();
    const bool cut = !p.plan || p.plan[2];
    const int item_rows = 2 * p.tile_tokens * g.group;
    Stretch st{};
    if (cut) st = find_stretch<kTile, kItemCost, kThreads>(g, item_rows, gbase + L::kOffScan);

    if (warp == kWarpTma) {
        // ---- work and TMA ---------------------------------------------------
        fence_proxy_async_global();
        const uint32_t box_bytes = (uint32_t)g.box * 128u;
        const int boxes = kTile / g.box;
        const int half = lane % kHalves, box = lane / kHalves;
        const uint32_t to = (uint32_t)half * L::kHalf + (uint32_t)box * box_bytes;
        const uint32_t q_half_bytes = (uint32_t)(p.tile_tokens * g.group) * 128u;
        int4 record = make_int4(-1, 0, 0, 0);
        Place at = st.at;
        Sequence s{};
        int64_t left = cut ? st.mine : 0, pos = st.first;
        if (left > 0) s = load_sequence(g, at.b);
        bool first = true;
        // the next unit (every lane has it); b = -1 when there is none
        const auto fetch = [&]() {
            Unit u;
            u.b = -1;
            if (cut) {
                if (left <= 0) return u;
                if (!first) next_item(g, at, s, item_rows);
                first = false;
                const Piece c = take_piece<kTile, kItemCost>(g, s, at, item_rows, left);
                if (!c.empty()) {
                    u = make_unit(p, s, at.b, at.rb, at.h, c.t0, c.t1 - c.t0, c.whole() ? -1 : c.part());
                    if (!c.whole() && c.t0 == 0)
                        record = make_int4(at.b, at.rb, at.h, last_block<kItemCost>(c, at, pos, st.size));
                }
                pos += c.count;
                left -= c.count;  // an empty piece is the stretch's last
                return u;
            }
            unsigned int i = 0;
            if (lane == 0) i = atomicAdd(p.plan, 1u);
            i = __shfl_sync(0xffffffffu, i, 0);
            const unsigned int total = p.plan[1];
            if (i >= total) return u;
            // kv heads in groups whose keys and values fit in L2 together
            const unsigned int entries = total / (unsigned int)g.kv_heads, per = entries * (unsigned int)p.head_group;
            const unsigned int grp = i / per, within = i - grp * per;
            const unsigned int here = min((unsigned int)p.head_group, (unsigned int)g.kv_heads - grp * p.head_group);
            const int4 e = p.entries[2 * (within / here)], k = p.entries[2 * (within / here) + 1];
            s.start = e.z, s.n = e.w, s.keys = k.x;
            return make_unit(p, s, e.x, e.y, (int)(grp * p.head_group + within % here), 0, 0x7fffffff, -1);
        };
        int n = 0;  // loads issued so far
        int k = 0;  // units published so far
        int s_before[2] = {0, 0}, o_before = 0;
        bool ok = true;
        Unit next = fetch();
        for (;; ++k) {
            // the previous unit's S products are done with Q, and every role
            // has read its entry, so the ring is never two entries ahead
            if (k > 0 && ok) ok = wait(L::kBarQEmpty, k - 1) && wait(L::kBarRead, k - 1);
            ok = __all_sync(0xffffffffu, ok);
            Unit u = next;
            if (!ok) u.b = -1;
            if (lane < 4 * kEdgeTiles) bad_keys(k)[lane] = 0u;
            __syncwarp();
            if (lane == 0) {
                volatile Unit &e = units[k & 1];
                e.b = u.b, e.h = u.h, e.start = u.start, e.i0 = u.i0, e.n = u.n, e.keys = u.keys, e.j0 = u.j0;
                e.n_a = u.n_a, e.n_b = u.n_b, e.part = u.part, e.kept_all = u.kept_all, e.load = n;
                e.s[0] = s_before[0], e.s[1] = s_before[1], e.step = s_before[0] + s_before[1], e.o = o_before;
                mbar_arrive(bar(L::kBarUnit));  // release: the entry is visible to whoever waits
            }
            if (u.b < 0) break;
            s_before[0] += u.n_a, s_before[1] += u.n_b;
            o_before ^= (u.n_a > 0 ? 1 : 0) | (u.n_b > 0 ? 2 : 0);
            if (!(p.starve && k == 0)) {  // the test hook leaves the first Q barrier unarmed
                if (lane == 0) mbar_arrive_expect_tx(bar(L::kBarQ), 2 * kHalves * q_half_bytes);
                __syncwarp();
                if (lane < 2 * kHalves) {
                    const int t = lane / kHalves;
                    tma_load_4d(base + L::kOffQ + (uint32_t)t * L::kTileBytes + (uint32_t)half * L::kHalf, &tq, half * 64, 0,
                                u.h, u.start + u.i0 + t * p.tile_tokens, bar(L::kBarQ));
                }
            }
            const int loads = 2 * max(u.n_a, u.n_b);
            Sequence us{u.start, u.n, u.keys};
            // where this lane's box of key tile j lies; asked for one tile ahead, so that
            // the page table's latency passes while the ring is full
            const auto find = [&](int j, int2 &at_page) {
                const int key = (u.j0 + j) * kTile + box * g.box;
                const bool in = box < boxes && key < u.keys && 2 * j < loads;
                if (in) at_page = locate(g, us, u.b, key);
                return in;
            };
            int2 place = make_int2(0, 0), place_next = place;
            bool live = false, live_next = find(0, place_next);
            for (int i = 0; i < loads && ok; ++i, ++n) {
                if (!(i & 1)) {  // K and V of a tile lie at the same places
                    place = place_next, live = live_next;
                    live_next = find((i >> 1) + 1, place_next);
                }
                const int slot = n % L::kSlots;
                // the slot last held load n - kSlots; its products must be done
                if (n >= L::kSlots) ok = wait(L::kBarEmpty + slot, n / L::kSlots - 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                const uint32_t copies = (uint32_t)__popc(__ballot_sync(0xffffffffu, live));
                if (lane == 0) mbar_arrive_expect_tx(bar(L::kBarFull + slot), copies * box_bytes);
                __syncwarp();
                if (live)
                    tma_load_4d(base + L::kOffRing + (uint32_t)slot * L::kTileBytes + to, (i & 1) ? &tv : &tk, half * 64,
                                place.y, u.h, place.x, bar(L::kBarFull + slot));
                if (i == 1) next = fetch();  // its latency passes while the ring holds work
            }
            if (loads < 2) next = fetch();
        }
        if (lane == 0) {
            // every copy issued lands before the block may exit
            if (k > 0 && !(p.starve && k == 1)) drain(L::kBarQ, k - 1);
            for (int m = n > L::kSlots ? n - L::kSlots : 0; m < n; ++m) drain(L::kBarFull + m % L::kSlots, m / L::kSlots);
            if (cut) p.records[blockIdx.x] = *abort_flag ? make_int4(-1, 0, 0, 0) : record;
        }
    } else if (warp == kWarpMma) {
        // ---- products -------------------------------------------------------
        // (one thread, by elect.sync: chosen by lane == 0 the same code took 7 % longer)
        if (elect_one()) {
            constexpr uint32_t id_s = f16_idesc(kBf16, false, kTile, kTile);  // S = Q K^T
            constexpr uint32_t id_o = f16_idesc(kBf16, true, kTile, D);       // O += P V
            // Between a group's P and its next S lies what this thread does, so that is
            // little: descriptors are made once, and a step adds to their low words (the
            // address field, in 16-byte units, stays below its 14 bits).
            const uint64_t desc_k = sw128_desc(base + L::kOffRing, 16, 1024);        // K-major: K, Q
            const uint64_t desc_v = sw128_desc(base + L::kOffRing, L::kHalf, 1024);  // MN-major: V
            const uint32_t hi = (uint32_t)(desc_k >> 32);  // of both: layout and stride
            const uint32_t k_lo = (uint32_t)desc_k, v_lo = (uint32_t)desc_v;
            const uint32_t q_lo = (uint32_t)sw128_desc(base + L::kOffQ, 16, 1024);
            int nb = 0;             // first load of the current unit
            int p_cnt[2] = {0, 0};  // P tiles consumed so far, per group (two buffers)
            int step_at = 0, step_turn = 0;  // the next step's buffer, and its time there (three buffers)
            const auto landed = [&](int m) { return wait(L::kBarFull + m % L::kSlots, m / L::kSlots); };
            const auto slot = [&](int m) { return (uint32_t)(m % L::kSlots) * (L::kTileBytes >> 4); };
            // S in buffer `to` of query tile q and K load m; both operands in shared memory
            const auto issue_s = [&](int to, int q, int m) {
                const uint32_t k = k_lo + slot(m), qd = q_lo + (uint32_t)q * (L::kTileBytes >> 4);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = ((uint32_t)(kk >> 2) * L::kHalf + (uint32_t)(kk & 3) * 32u) >> 4;
                    mma_ss_lo(tmem + col_s(to), qd + off, hi, k + off, hi, id_s, kk > 0);
                }
                mma_commit(bar(L::kBarS + to));
            };
            // O_t (+)= P V of load m; P in TMEM, buffer `from`
            const auto issue_pv = [&](int t, int from, int m, bool first) {
                const uint32_t v = v_lo + slot(m);
#pragma unroll
                for (int kk = 0; kk < kTile / 16; ++kk)
                    mma_ts_lo(tmem + col_o<D>(t), tmem + col_s(from) + (uint32_t)kk * 8u, v + (uint32_t)kk * 128u, hi, id_o,
                              (!first || kk > 0));
            };
            const auto free_load = [&](int m) { mma_commit(bar(L::kBarEmpty + m % L::kSlots)); };
            const auto wait_p = [&](int t) { return wait(L::kBarP + t, p_cnt[t]++); };
            bool ok = true;
            for (int k = 0; ok; ++k) {
                if (!(ok = wait(L::kBarUnit, k))) break;
                const int b = units[k & 1].b, n_a = units[k & 1].n_a, n_b = units[k & 1].n_b;
                mbar_arrive(bar(L::kBarRead));
                if (b < 0) break;
                const int count = max(n_a, n_b);
                if (!(ok = wait(L::kBarQ, k))) break;
                if (count == 0) mma_commit(bar(L::kBarQEmpty));
                // S of a unit overwrites P of the one before only after the product that
                // reads it, which was issued before it
                if constexpr (kAhead) {
                    // Step i has S and P in buffer i mod 3, so S of step i + 3 may follow P V
                    // of step i, and a group finds the S of its next tile made while it was
                    // busy with this one.  (In two buffers S follows the group's own P V: the
                    // group waits for both, 820 of the 2400 cycles of a pair of tiles of
                    // head dim 64.)
                    const int both = min(n_a, n_b), steps = n_a + n_b, tail = n_b > n_a ? 1 : 0;
                    const auto group_of = [&](int i) { return i < 2 * both ? i & 1 : tail; };
                    const auto tile_of = [&](int i) { return i < 2 * both ? i >> 1 : i - both; };
                    int k_seen = 0, v_seen = 0;  // key tiles whose K and V have been waited for
                    const auto next_s = [&](int i, int to) {
                        const int t = group_of(i), j = tile_of(i), m = nb + 2 * j;
                        if (j >= k_seen) {
                            if (!landed(m)) return false;
                            k_seen = j + 1;
                            tc_fence_after();
                        }
                        issue_s(to, t, m);
                        if (t == 1 || j >= n_b) free_load(m);  // the last to use K_j
                        if (i + 1 == steps) mma_commit(bar(L::kBarQEmpty));
                        return true;
                    };
                    int at = step_at;
                    for (int i = 0; i < min(3, steps) && ok; ++i) ok = next_s(i, (at + i) % 3);
                    for (int i = 0; i < steps && ok; ++i) {
                        const int t = group_of(i), j = tile_of(i), v = nb + 2 * j + 1;
                        if (j >= v_seen) {
                            if (!(ok = landed(v))) break;
                            v_seen = j + 1;
                        }
                        if (!(ok = wait(L::kBarP + at, step_turn))) break;
                        tc_fence_after();
                        issue_pv(t, at, v, j == 0);
                        mma_commit(bar(L::kBarDone + at));
                        if (t == 1 || j >= n_b) free_load(v);
                        if (j + 1 == (t ? n_b : n_a)) mma_commit(bar(L::kBarO + t));
                        if (i + 3 < steps) ok = next_s(i + 3, at);
                        if (++at == 3) at = 0, ++step_turn;
                    }
                    step_at = at;
                } else if (count > 0) {
                    if (!(ok = landed(nb))) break;
                    tc_fence_after();
                    if (n_a > 0) issue_s(0, 0, nb);
                    if (n_b > 0) issue_s(1, 1, nb);
                    free_load(nb);
                    if (count == 1) mma_commit(bar(L::kBarQEmpty));
                    for (int j = 0; j < count; ++j) {
                        const int v = nb + 2 * j + 1, next = v + 1;  // V_j, K_{j+1}
                        if (!(ok = landed(v))) break;
                        bool k_here = false;  // K_{j+1} has been waited for
                        if (j < n_a) {
                            if (!(ok = wait_p(0))) break;
                            tc_fence_after();
                            issue_pv(0, 0, v, j == 0);
                            if (j + 1 < n_a) {
                                if (!(ok = landed(next))) break;
                                k_here = true;
                                tc_fence_after();
                                issue_s(0, 0, next);
                            } else {
                                mma_commit(bar(L::kBarO + 0));
                            }
                        }
                        if (j < n_b) {
                            if (!(ok = wait_p(1))) break;
                            tc_fence_after();
                            issue_pv(1, 1, v, j == 0);
                        }
                        free_load(v);
                        if (j < n_b) {
                            if (j + 1 < n_b) {
                                if (!k_here && !(ok = landed(next))) break;
                                tc_fence_after();
                                issue_s(1, 1, next);
                            } else {
                                mma_commit(bar(L::kBarO + 1));
                            }
                        }
                        if (j + 1 < count) {
                            free_load(next);
                            if (j + 2 == count) mma_commit(bar(L::kBarQEmpty));  // the unit's last S
                        }
                    }
                }
                nb += 2 * count;
            }
            // every product issued completes before TMEM is released
            mma_commit(bar(L::kBarDrain));
            drain(L::kBarDrain, 0);
        }
    } else {
        // ---- softmax: thread r of group t owns row r of query tile t ---------
        const int t = warp >> 2;
        const int r = (int)(threadIdx.x & 127);
        const uint32_t lane_addr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        bool ok = true;
        for (int k = 0; ok; ++k) {
            ok = __all_sync(0xffffffffu, wait(L::kBarUnit, k));
            if (!ok) break;
            const volatile Unit &u = units[k & 1];
            // What the loop over tiles needs, and no more: the rest is read from the
            // unit again at its end (its entry stays until this warp has read the next
            // one): the loop holds 128 scores in 168 registers.
            const bool last = u.b < 0;
            int lim;                                     // kept columns of the tile: [0, lim)
            {
                const int row_token = r / g.group, i = u.i0 + t * p.tile_tokens + row_token;
                const Sequence s{0, u.n, u.keys};
                lim = (row_token < p.tile_tokens && i < s.n ? kept_keys(g, s, i) : 0) - u.j0 * kTile;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::kBarRead));
            if (last) break;
            const int edge = u.kept_all / kTile - u.j0;
            float m_run = -INFINITY;                 // the shift, in log2 units
            float l_run = 0.f;
            for (int j = 0; j < (t ? u.n_b : u.n_a); ++j, lim -= kTile) {
                if (j >= edge) {  // some row keeps not every key of this tile
                    // Thread r looks over key r's values: x * 0 summed is NaN once one of them is
                    // infinite or NaN.  Each group does so before it lets its product read the
                    // tile; a value is flagged before it is zeroed, so that whoever finds the
                    // zero finds the flag.
                    // (The unit's S products before this one, or the ones of the unit before,
                    // have used every load up to the slot's previous one, so its barrier is
                    // in this load's phase or the next, which the parity tells apart.)
                    const int load = u.load + 2 * j + 1;
                    ok = __all_sync(0xffffffffu, wait(L::kBarFull + load % L::kSlots, load / L::kSlots));
                    if (!ok) break;
                    zero_bad_values<T, D>(gbase + L::kOffRing + (uint32_t)(load % L::kSlots) * L::kTileBytes + r * 128, r & 7,
                                          bad_keys(k) + 4 * (u.j0 + j - u.kept_all / kTile), r,
                                          (u.j0 + j) * kTile + r < u.keys);
                }
                // where S_t of the tile lies (and its barriers), and for which time
                int at = t, turn = u.s[t] + j;
                if constexpr (kAhead) {
                    const int step = u.step + step_of(u.n_a, u.n_b, t, j);
                    at = step % 3, turn = step / 3;
                }
                ok = __all_sync(0xffffffffu, wait(L::kBarS + at, turn));
                if (!ok) break;
                tc_fence_after();
                float x[kTile];
                tmem_load128(lane_addr + col_s(at), x);
                if (lim < kTile) {
#pragma unroll
                    for (int c = 0; c < kTile; ++c)
                        if (c >= lim) x[c] = -INFINITY;
                }
                float mx[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) mx[e] = fmaxf(x[e], x[4 + e]);
#pragma unroll
                for (int c = 8; c < kTile; c += 8) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], x[c + e], x[c + 4 + e]);
                }
                const float m_tile = max3(mx[0], mx[1], fmaxf(mx[2], mx[3])) * g.kscale;
                float alpha = 1.f;
                bool moved = false;
                if (m_tile > m_run + (kShiftBelow<T> + kShiftSlack)) {
                    const float to = m_tile - kShiftBelow<T>;
                    alpha = ex2(m_run - to);  // 0 on the first tile with keys
                    l_run *= alpha;
                    m_run = to;
                    moved = j > 0;
                }
                const float shift = safe_shift(m_run);
                const uint64_t k2 = f2(g.kscale, g.kscale), nm2 = f2(-shift, -shift);
                uint64_t sum2[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t pk[16];
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const float2 a = f2_split(fma_f2(f2(x[32 * q + 2 * c], x[32 * q + 2 * c + 1]), k2, nm2));
                        const float p0 = ex2(a.x), p1 = ex2(a.y);
                        sum2[c & 1] = add_f2(sum2[c & 1], f2(p0, p1));
                        pk[c] = pack2<T>(p0, p1);
                    }
                    tmem_st16(lane_addr + col_s(at) + 16 * q, pk);
                }
                const float2 sa = f2_split(sum2[0]), sb = f2_split(sum2[1]);
                l_run += (sa.x + sa.y) + (sb.x + sb.y);
                if (__any_sync(0xffffffffu, moved)) {
                    // O_t's previous update has completed: S_t of this tile was issued after
                    // it, or it is waited for
                    if constexpr (kAhead) {
                        const int step = u.step + step_of(u.n_a, u.n_b, t, j - 1);
                        ok = __all_sync(0xffffffffu, wait(L::kBarDone + step % 3, step / 3));
                        if (!ok) break;
                        tc_fence_after();
                    }
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        float ov[32];
                        tmem_load32(lane_addr + col_o<D>(t) + c * 32, ov);
#pragma unroll
                        for (int e = 0; e < 32; ++e) ov[e] *= alpha;
                        tmem_st32(lane_addr + col_o<D>(t) + c * 32, ov);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::kBarP + at));
            }
            if (!ok) break;
            // ---- the unit's rows: O / l, or the part's O with its (m, l) ------
            // (what does not need O, before the wait for it)
            const int n_t = t ? u.n_b : u.n_a, part = u.part, h = u.h;
            const int row_token = r / g.group, i = u.i0 + t * p.tile_tokens + row_token;
            const bool valid = row_token < p.tile_tokens && i < u.n;
            const int64_t token = (int64_t)u.start + i, head = (int64_t)h * g.group + (r - row_token * g.group);
            if (valid) {
                if (part >= 0)
                    p.states[((int64_t)part * 2 + t) * kTile + r] = make_float2(m_run, l_run);
                else if (g.lse)
                    g.lse[token * g.heads + head] = natural_lse(m_run, l_run);
            }
            if (part >= 0 && n_t == 0) continue;  // a part without keys: its state says so
            const float inv = l_run == 0.f ? 0.f : 1.f / l_run;
            const int64_t row_at = valid ? token * g.o_token + head * g.o_head : -1;
            // a warp stores its rows four at a time, 128 bytes of each: this lane's are 4 e + lane / 8
            uint16_t *store_to[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int64_t to = __shfl_sync(0xffffffffu, row_at, 4 * e + (lane >> 3));
                store_to[e] = to >= 0 ? g.o + to + 8 * (lane & 7) : nullptr;
            }
            uint8_t *const stage = gbase + L::kOffStage + warp * 4096;
            float *const part_at = p.parts + (((int64_t)part * 2 + t) * (D / 4) * kTile + r) * 4;
            bool mend = false;
            if (n_t > 0) {
                ok = __all_sync(0xffffffffu, wait(L::kBarO + t, u.o >> t));
                if (!ok) break;
                tc_fence_after();
                uint4 any = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int w = 0; w < kEdgeTiles; ++w) {
                    const uint4 b4 = reinterpret_cast<const uint4 *>(bad_keys(k))[w];
                    any.x |= b4.x | b4.y | b4.z | b4.w;
                }
                mend = any.x != 0u;
            }
#pragma unroll 1
            for (int c2 = 0; c2 < kHalves; ++c2) {  // 64 columns of O at a time
                float ov[64];
                if (n_t > 0) {
                    tmem_load64(lane_addr + col_o<D>(t) + 64 * c2, ov);
                } else {
#pragma unroll
                    for (int e = 0; e < 64; ++e) ov[e] = 0.f;
                }
                if (part >= 0) {
                    if (valid) {
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            *reinterpret_cast<float4 *>(part_at + (int64_t)(16 * c2 + e) * kTile * 4) =
                                make_float4(ov[4 * e], ov[4 * e + 1], ov[4 * e + 2], ov[4 * e + 3]);
                    }
                    continue;
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    uint4 w;
                    w.x = pack2<T>(ov[8 * e + 0] * inv, ov[8 * e + 1] * inv);
                    w.y = pack2<T>(ov[8 * e + 2] * inv, ov[8 * e + 3] * inv);
                    w.z = pack2<T>(ov[8 * e + 4] * inv, ov[8 * e + 5] * inv);
                    w.w = pack2<T>(ov[8 * e + 6] * inv, ov[8 * e + 7] * inv);
                    *reinterpret_cast<uint4 *>(stage + lane * 128 + ((e ^ (lane & 7)) << 4)) = w;
                }
                __syncwarp();
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int row = 4 * e + (lane >> 3);
                    const uint4 w = *reinterpret_cast<const uint4 *>(stage + row * 128 + (((lane & 7) ^ (row & 7)) << 4));
                    if (store_to[e]) *reinterpret_cast<uint4 *>(store_to[e] + 64 * c2) = w;
                }
                __syncwarp();
            }
            if (mend && valid) {
                const Sequence s{u.start, u.n, u.keys};
                const int tile0 = u.kept_all / kTile;
                add_bad_values<T, D>(g, s, u.b, h, tile0, bad_keys(k), max(u.j0, tile0) * kTile,
                                     min(kept_keys(g, s, i), (u.j0 + n_t) * kTile),
                                     part >= 0 ? nullptr : g.o + row_at, part_at);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// One block: the items' row blocks sorted by their key tiles, most first (a
// counting sort in kBins bins of 2^shift tiles), for the blocks to take in turn;
// or the decision to cut, where one row block has more than an SM's fair share.
// Warp w takes the sequences w, w + 32, ...; its lanes load 32 of them at once
// and share out the row blocks of each.
constexpr int kBins = 1024;
struct PlanParams {
    Geometry g;
    unsigned int *plan;
    int4 *entries;
    int capacity;  // of entries: enough for offsets that rise
    int rows;      // of an item
    int sms, shift;
    unsigned int cut_cost;  // of cutting and joining, in tiles' time of an SM
};
__global__ void __launch_bounds__(1024) k_tiles_plan(const __grid_constant__ PlanParams p) {
    __shared__ unsigned int bins[kBins], warp_sum[32];
    __shared__ unsigned long long total, total_blocks;
    __shared__ int most, least;
    const Geometry &g = p.g;
    pdl_enter();
    const int warp = (int)(threadIdx.x >> 5), lane = (int)(threadIdx.x & 31);
    bins[threadIdx.x] = 0u;
    if (threadIdx.x == 0) total = 0ull, total_blocks = 0ull, most = 0, least = 0x7fffffff;
    __syncthreads();
    const auto walk = [&](auto &&each) {
        for (int64_t b0 = warp; b0 < g.batch; b0 += 32 * 32) {
            const int64_t b = b0 + 32 * lane;
            Sequence s{0, 0, 0};
            if (b < g.batch) s = load_sequence(g, (int)b);
            for (int l = 0; l < 32 && b0 + 32 * l < g.batch; ++l) {
                const Sequence o{__shfl_sync(0xffffffffu, s.start, l), __shfl_sync(0xffffffffu, s.n, l),
                                 __shfl_sync(0xffffffffu, s.keys, l)};
                const int nb = row_blocks(g, o, p.rows);
                for (int rb = lane; rb < nb; rb += 32)
                    each((int)(b0 + 32 * l), rb, o, tiles_of<kTile>(block_keys(g, o, rb, p.rows)));
            }
        }
    };
    unsigned long long own = 0, blocks = 0;
    int top = 0, low = 0x7fffffff;
    walk([&](int, int, const Sequence &, int tiles) {
        own += (unsigned long long)tiles;
        ++blocks;
        top = max(top, tiles);
        low = min(low, tiles);
        atomicAdd(&bins[kBins - 1 - min(tiles >> p.shift, kBins - 1)], 1u);
    });
    for (int o = 16; o; o >>= 1) {
        own += __shfl_xor_sync(0xffffffffu, own, o);
        blocks += __shfl_xor_sync(0xffffffffu, blocks, o);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        low = min(low, __shfl_xor_sync(0xffffffffu, low, o));
    }
    if (lane == 0 && own) {
        atomicAdd(&total, own);
        atomicAdd(&total_blocks, blocks);
        atomicMax(&most, top);
        atomicMin(&least, low);
    }
    __syncthreads();
    const unsigned int mine = bins[threadIdx.x];
    unsigned int upto = mine;
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) warp_sum[warp] = upto;
    __syncthreads();
    unsigned int all = 0;
    for (int w = 0; w < 32; ++w) {
        if (w < warp) upto += warp_sum[w];
        all += warp_sum[w];
    }
    bins[threadIdx.x] = upto - mine;
    // (a plan that does not cut has at most `capacity` row blocks: its bins and `all`, in
    // 32 bits, are exact)
    const PlanCounts counts{total_blocks, total, (uint32_t)most, (uint32_t)least};
    const bool cut = plan_cuts(counts, (uint32_t)g.kv_heads, (uint32_t)p.sms, (uint32_t)p.capacity, p.cut_cost);
    if (threadIdx.x == 0) {
        p.plan[0] = 0u;
        p.plan[1] = all * (unsigned)g.kv_heads;
        p.plan[2] = cut ? 1u : 0u;
    }
    __syncthreads();
    if (cut) return;
    walk([&](int b, int rb, const Sequence &s, int tiles) {
        const unsigned int at = atomicAdd(&bins[kBins - 1 - min(tiles >> p.shift, kBins - 1)], 1u);
        p.entries[2 * at] = make_int4(b, rb, s.start, s.n);
        p.entries[2 * at + 1] = make_int4(s.keys, 0, 0, 0);
    });
}

// The cut items: block (x, y) merges 16 columns of one query tile of the item
// that begins in block x of k_seq_tiles, part by part in order.
template <typename T, int D>
__global__ void __launch_bounds__(kTile) k_tiles_join(const __grid_constant__ TilesParams p) {
    pdl_enter();
    const Geometry &g = p.g;
    if (p.plan && !p.plan[2]) return;
    const int4 rec = p.records[blockIdx.x];
    if (rec.x < 0) return;
    const int t = (int)blockIdx.y / (D / 16), c0 = (int)blockIdx.y % (D / 16) * 16;
    const int r = (int)threadIdx.x;
    const Sequence s = load_sequence(g, rec.x);
    const int row_token = r / g.group;
    const int64_t i = (int64_t)rec.y * 2 * p.tile_tokens + t * p.tile_tokens + row_token;
    if (row_token >= p.tile_tokens || i >= s.n) return;
    const int first = (int)blockIdx.x, last = rec.w;
    const auto state = [&](int b) { return p.states[((int64_t)(2 * b + (b == first ? 1 : 0)) * 2 + t) * kTile + r]; };
    float shift = -INFINITY, all = 0.f;
    for (int b = first; b <= last; ++b) shift = fmaxf(shift, state(b).x);
    float4 acc[4] = {};
#pragma unroll 4
    for (int b = first; b <= last; ++b) {
        const float2 st = state(b);
        const float w = ex2(st.x - safe_shift(shift));
        // a part without keys has no O; one far below the others has, and its infinite
        // and NaN values reach the row
        if (st.x == -INFINITY && st.y == 0.f) continue;
        all += st.y * w;
        const float *o = p.parts + (((int64_t)(2 * b + (b == first ? 1 : 0)) * 2 + t) * (D / 4) * kTile + r) * 4;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float4 v = *reinterpret_cast<const float4 *>(o + (int64_t)(c0 / 4 + e) * kTile * 4);
            acc[e].x += v.x * w, acc[e].y += v.y * w, acc[e].z += v.z * w, acc[e].w += v.w * w;
        }
    }
    const int64_t token = s.start + i, head = (int64_t)rec.z * g.group + (r - row_token * g.group);
    const float inv = all == 0.f ? 0.f : 1.f / all;
    uint16_t *const o = g.o + token * g.o_token + head * g.o_head + c0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        uint4 w;
        w.x = pack2<T>(acc[2 * e].x * inv, acc[2 * e].y * inv);
        w.y = pack2<T>(acc[2 * e].z * inv, acc[2 * e].w * inv);
        w.z = pack2<T>(acc[2 * e + 1].x * inv, acc[2 * e + 1].y * inv);
        w.w = pack2<T>(acc[2 * e + 1].z * inv, acc[2 * e + 1].w * inv);
        *reinterpret_cast<uint4 *>(o + 8 * e) = w;
    }
    if (g.lse && c0 == 0) g.lse[token * g.heads + head] = natural_lse(shift, all);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
int tile_tokens(const softmax_sequence_args_t &a) { return (int)(kTile / (a.heads / a.kv_heads)); }

// Row blocks of the batch: at most this many, and about `least` of them.
int64_t most_blocks(const softmax_sequence_args_t &a) { return a.tokens / (2 * tile_tokens(a)) + a.batch; }
int64_t least_blocks(const softmax_sequence_args_t &a) { return a.tokens / (2 * tile_tokens(a)); }
bool planned(const softmax_sequence_args_t &a, int sms) {
    return least_blocks(a) * a.kv_heads >= (int64_t)kItemsPerSm * sms && most_blocks(a) * a.kv_heads < 0x7fffffff;
}

struct Space {
    int64_t plan, entries, records, states, parts, bytes;
};
Space space(const softmax_sequence_args_t &a, int sms) {
    const auto up = [](int64_t n) { return (n + 255) / 256 * 256; };
    Space s;
    s.plan = 0;
    s.entries = 256;
    s.records = s.entries + (planned(a, sms) ? up(most_blocks(a) * 2 * (int64_t)sizeof(int4)) : 0);
    s.states = s.records + up(sms * (int64_t)sizeof(int4));
    s.parts = s.states + up(2 * (int64_t)sms * 2 * kTile * (int64_t)sizeof(float2));
    s.bytes = s.parts + up(2 * (int64_t)sms * 2 * kTile * a.head_dim * (int64_t)sizeof(float));
    return s;
}

template <typename T, int D>
cudaError_t go(const AttnCall &c) {
    using L = Layout<D>;
    const softmax_sequence_args_t &a = c.a;
    static std::atomic<unsigned long long> opted{0};
    cudaError_t e = opt_in_shared_memory((const void *)k_seq_tiles<T, D>, (int)L::kBytes, opted);
    if (e != cudaSuccess) return e;
    TilesParams p;
    CUtensorMap tq, tk, tv;
    if (!fill_geometry(c, kTile, &p.g) || !make_kv_maps(c, p.g.box, &tk, &tv)) return cudaErrorInvalidValue;
    p.tile_tokens = tile_tokens(a);
    const int64_t qdims[4] = {a.head_dim, p.g.group, a.kv_heads, a.tokens};
    const int64_t qst[3] = {a.q_head_stride, a.q_head_stride * p.g.group, a.q_token_stride};
    const int qbox[4] = {64, p.g.group, 1, p.tile_tokens};
    if (!make_map(&tq, a.q, a, qdims, qst, qbox)) return cudaErrorInvalidValue;
    const Space sp = space(a, c.sms);
    uint8_t *const w = (uint8_t *)c.workspace;
    const bool plan = planned(a, c.sms);
    p.plan = plan ? reinterpret_cast<unsigned int *>(w + sp.plan) : nullptr;
    p.entries = reinterpret_cast<const int4 *>(w + sp.entries);
    const int64_t head_bytes = 4 * a.head_dim *
                               (c.paged ? std::min<int64_t>(a.pages * a.page_size, a.batch * (int64_t)p.g.max_keys) : a.tokens);
    p.head_group = (int)std::max<int64_t>(1, std::min<int64_t>(attn::kAttnGroupBytes / head_bytes, a.kv_heads));
    p.records = reinterpret_cast<int4 *>(w + sp.records);
    p.states = reinterpret_cast<float2 *>(w + sp.states);
    p.parts = reinterpret_cast<float *>(w + sp.parts);
    p.wait_ns = wait_limit(c.wait_ns);
    p.starve = c.starve;
    LaunchArgs l = {};
    l.stream = c.stream;
    l.overlap = c.overlap;
    if (plan) {
        PlanParams q;
        q.g = p.g;
        q.plan = p.plan;
        q.entries = reinterpret_cast<int4 *>(w + sp.entries);
        q.capacity = (int)most_blocks(a);
        q.rows = 2 * p.tile_tokens * p.g.group;
        q.sms = c.sms;
        q.shift = 0;
        // measured: 4096 tokens, 32/8 heads, no mask (20 tiles idle, head dim 128): 228 us whole,
        // 214 us cut; 8192 tokens (17 idle): 757 and 753; 4 x 2048, 16 heads, head dim 64 (10
        // idle): 104 and 95
        q.cut_cost = D == 128 ? 14 : 8;
        const int64_t top = ((c.paged ? p.g.max_keys : a.tokens) + kTile - 1) / kTile;
        while ((top >> q.shift) >= kBins) ++q.shift;
        e = launch_kernel(k_tiles_plan, l, 1, 1024, 0, 0, q);
        if (e != cudaSuccess) return e;
    }
    const int64_t blocks = plan ? c.sms : blocks_with_work(p.g, most_blocks(a), kTile, kItemCost, c.sms);
    e = launch_kernel(k_seq_tiles<T, D>, l, blocks, kThreads, L::kBytes, 0, tq, tk, tv, p);
    if (e != cudaSuccess) return e;
    return launch_kernel_2d(k_tiles_join<T, D>, c, dim3((unsigned)blocks, 2 * D / 16), kTile, p);
}

}  // namespace

int64_t tiles_workspace_bytes(const softmax_sequence_args_t &a, int sms) { return space(a, sms).bytes; }

cudaError_t launch_tiles(const AttnCall &c) {
    if (c.a.dtype == SOFTMAX_BF16) return c.a.head_dim == 128 ? go<__nv_bfloat16, 128>(c) : go<__nv_bfloat16, 64>(c);
    return c.a.head_dim == 128 ? go<__half, 128>(c) : go<__half, 64>(c);
}

cudaError_t read_clear_tiles_error_word(unsigned int *word) {
    cudaError_t e = cudaMemcpyFromSymbol(word, g_tiles_error, sizeof(unsigned int), 0, cudaMemcpyDeviceToHost);
    if (e != cudaSuccess) return e;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(g_tiles_error, &zero, sizeof(unsigned int), 0, cudaMemcpyHostToDevice);
}

}  // namespace seq
}  // namespace mbrs
