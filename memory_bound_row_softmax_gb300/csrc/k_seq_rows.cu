// k_seq_rows.cu -- attention of a few query rows against many keys: single
// tokens and short chunks over a paged cache, and short packed prompts.
//
// The rows of one item are the new tokens of one sequence times the query
// heads that share one key/value head (row r: token r / group, head r % group),
// 16 or 32 of them; its keys go by in tiles of 64.  With so few rows every
// K and V byte is used once, so HBM bounds the call (64 tokens over 37 to 8000
// keys, 988 MB, 159-165 us: 6.0-6.2 TB/s, 0.88-0.91 of a copy's rate), and the products
// need far less than the tensor cores have: 16-row mma.sync tiles, whose accumulators are
// registers, keep the warps independent of each other (a 128-row tcgen05 tile
// would be seven eighths empty).
//
// Work split: the work of all items, in the order (sequence, row block, kv head),
// is cut into equal stretches, one per block, whatever the sequences' lengths.  Each
// block finds its stretch from q_starts and kv_lens itself (one scan over the batch).
// A block walks its stretch item by item; an item it holds whole is finished there, of
// a cut one the part's (shift, sum, O) goes to the workspace in fp32 and k_rows_join
// merges the parts in order (the merge rule of common.cuh), so results do not depend on
// timing.
//
// Roles: the last warp feeds a ring of K/V tiles with TMA (one lane per copy: a
// copy is a box of whole rows within one page, 128-byte swizzled).  Four warps
// share 16 rows: each owns 16 keys of every tile, with its own running shift, sum
// and O, so nothing is exchanged until the item's end: S = Q K^T with Q from shared
// memory, the softmax on S's registers, which are then P's registers for P V.  At
// the item's end the four states are merged through shared memory.  32 rows take
// two such groups of warps side by side on the same tiles (one group with two row
// tiles each spilled: 32 x 4 tokens over 4000 keys 131 us where two groups take 106).
//
// Masked values: a tile that holds keys some row does not keep is looked over
// first; infinite and NaN values in it are set to zero in shared memory (a
// masked P is 0, and 0 times them would be NaN) and, at the item's end, added
// back to the rows that do keep them.
#include <type_traits>

#include "launch.h"
#include "sequence.cuh"
#include "sequence_host.h"

namespace mbrs {
namespace seq {

__device__ unsigned int g_rows_error;

namespace {

constexpr int kKeys = 64;      // keys per tile
constexpr int kWarpKeys = 16;  // a warp's share of them
constexpr int kWarps = kKeys / kWarpKeys;
constexpr int kGroupThreads = kWarps * 32;
// The ring: 128 KB of keys and values on their way to an SM, by two blocks of one
// row group or one of two.  (More is slower: three stages instead of two 167 us
// where two take 163.)
template <int NG> constexpr int kStages = NG == 1 ? 2 : 4;
template <int NG> constexpr int kBlocksPerSm = NG == 1 ? 2 : 1;
template <int NG> constexpr int kThreads = NG * kGroupThreads + 32;
constexpr int kItemCost = 1;   // beginning and ending an item, in tiles' time

template <int D, int NG>
struct Layout {
    static constexpr int kRows = 16 * NG;
    static constexpr uint32_t kTile = kKeys * D * 2;              // a K or V tile: boxes of [64 columns][row]
    static constexpr uint32_t kQPitch = D * 2 + 16;               // padded: ldmatrix without bank conflicts
    static constexpr int kCols = 32;                              // columns of O merged at a time
    static constexpr int kColPitch = kCols + 4;
    static constexpr uint32_t kQBytes = 16 * kQPitch;
    static constexpr uint32_t kMergeBytes = kWarps * 16 * kColPitch * 4;
    static constexpr uint32_t kGroupBytes = kQBytes > kMergeBytes ? kQBytes : kMergeBytes;
    // from a 1024-byte aligned base; a group's Q and merge buffer take turns
    static constexpr uint32_t kOffRing = 0;
    static constexpr uint32_t kOffQ = kOffRing + kStages<NG> * 2 * kTile;
    static constexpr uint32_t kOffStates = kOffQ + NG * kGroupBytes;
    static constexpr uint32_t kOffBar = kOffStates + NG * kWarps * 16 * 8;
    static constexpr uint32_t kOffScan = kOffBar + 2 * kStages<NG> * 8;
    static constexpr uint32_t kOffAbort = kOffScan + kScanBytes;
    static constexpr uint32_t kOffBad = kOffAbort + 4;            // infinite or NaN values have been set to zero
    static constexpr size_t kBytes = kOffBad + 4 + 1024;
};
static_assert(Layout<128, 1>::kBytes <= 115200 && Layout<128, 2>::kBytes <= 232448, "shared memory per block");

struct RowsParams {
    Geometry g;
    const uint16_t *q;
    int64_t q_token, q_head;
    int4 *records;    // per block: the cut item that begins in it {sequence or -1, row block, kv head, last block}
    float2 *states;   // per part and row: (shift, sum), the shift in log2 units
    float *parts;     // per part: kRows x D
    uint32_t wait_ns;
    int starve;       // test hook: leave the first tile's barrier unarmed
};

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t *r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t *r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
template <typename T>
__device__ __forceinline__ void mma16816(float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same<T, __half>::value)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                     "{%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                     "{%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The four warps of a row group.  (A barrier named in a register would reserve
// all sixteen.)
__device__ __forceinline__ void group_barrier(int group) {
    if (group == 0)
        asm volatile("bar.sync 1, %0;" ::"n"(kGroupThreads) : "memory");
    else
        asm volatile("bar.sync 2, %0;" ::"n"(kGroupThreads) : "memory");
}

template <typename T, int D, int NG>
__global__ void __launch_bounds__(kThreads<NG>, kBlocksPerSm<NG>)
    k_seq_rows(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
               const __grid_constant__ RowsParams p) {
    using L = Layout<D, NG>;
    constexpr int kRows = L::kRows, kStages = mbrs::seq::kStages<NG>;
    const Geometry &g = p.g;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *const gbase = smem_raw + (base - raw);
    volatile uint32_t *const abort_flag = reinterpret_cast<volatile uint32_t *>(gbase + L::kOffAbort);
    volatile uint32_t *const bad = reinterpret_cast<volatile uint32_t *>(gbase + L::kOffBad);
    const auto full = [base](int s) { return base + L::kOffBar + 8u * (uint32_t)s; };
    const auto empty = [base](int s) { return base + L::kOffBar + 8u * (uint32_t)(kStages + s); };
    const int warp = (int)(threadIdx.x >> 5), lane = (int)(threadIdx.x & 31);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), NG * kWarps);
        }
        *abort_flag = 0u;
        *bad = 0u;
        fence_mbar_init();
        attn::tma_prefetch_desc(&tk);
        attn::tma_prefetch_desc(&tv);
    }
    prefetch_indices(g);
    pdl_enter();

    const Stretch st = find_stretch<kKeys, kItemCost, kThreads<NG>>(g, kRows, gbase + L::kOffScan);
    const int64_t stretch = st.size, first = st.first, mine = st.mine;
    if (mine <= 0) {
        if (threadIdx.x == 0) p.records[blockIdx.x] = make_int4(-1, 0, 0, 0);
        return;
    }
    Place at = st.at;
    Sequence s = load_sequence(g, at.b);

    if (warp == NG * kWarps) {
        // ---- TMA producer: lane u copies box u of the tile ----------------
        const int boxes = kKeys / g.box;
        const int which = lane & 1, box = lane >> 1;
        fence_proxy_async_global();
        const uint32_t box_bytes = (uint32_t)g.box * D * 2;
        const uint32_t to = (uint32_t)which * L::kTile + (uint32_t)box * box_bytes;
        int n = 0;
        bool ok = true;
        for (int64_t left = mine; left > 0 && ok;) {
            const int keys = block_keys(g, s, at.rb, kRows);
            const Piece piece = take_piece<kKeys, kItemCost>(g, s, at, kRows, left);
            // where this lane's box of tile t lies; asked for one tile ahead
            const auto find = [&](int t, int2 &page) {
                const int j = t * kKeys + box * g.box;
                const bool in = box < boxes && j < keys && t < piece.t1;
                if (in) page = locate(g, s, at.b, j);
                return in;
            };
            int2 place = make_int2(0, 0), place_next = place;
            bool live = false, live_next = find(piece.t0, place_next);
            for (int t = piece.t0; t < piece.t1; ++t, ++n) {
                const int stage = n % kStages;
                place = place_next, live = live_next;
                live_next = find(t + 1, place_next);
                if (n >= kStages)
                    ok = wait_phase(empty(stage), ((n / kStages) - 1) & 1, abort_flag, &g_rows_error, p.wait_ns);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (p.starve && n == 0) continue;  // the test hook: this tile never lands
                const uint32_t copies = (uint32_t)__popc(__ballot_sync(0xffffffffu, live));
                if (lane == 0) {
                    if (copies) mbar_arrive_expect_tx(full(stage), copies * box_bytes);
                    else mbar_arrive(full(stage));
                }
                __syncwarp();
                if (live)
                    tma_load_5d(base + L::kOffRing + (uint32_t)stage * 2u * L::kTile + to, which ? &tv : &tk, 0, place.y, 0,
                                at.h, place.x, full(stage));
            }
            left -= piece.count;
            if (left > 0) next_item(g, at, s, kRows);
        }
        // every copy issued lands before the block may exit
        if (lane == 0)
            for (int m = n > kStages ? n - kStages : p.starve ? 1 : 0; m < n; ++m)
                drain_phase(full(m % kStages), (m / kStages) & 1, abort_flag, &g_rows_error, p.wait_ns);
        return;
    }

    // ---- products and softmax ----------------------------------------------
    const int group = NG == 1 ? 0 : warp / kWarps, slice = warp % kWarps;  // 16 rows of the item, 16 keys of a tile
    const int tid = (int)threadIdx.x % kGroupThreads;
    float2 *const merge_state = reinterpret_cast<float2 *>(gbase + L::kOffStates) + group * kWarps * 16;  // [slice][row]
    uint8_t *const q_smem = gbase + L::kOffQ + group * L::kGroupBytes;
    float *const merge = reinterpret_cast<float *>(q_smem);                               // [slice][row][kColPitch]
    const uint32_t q_lane = base + L::kOffQ + (uint32_t)group * L::kGroupBytes +
                            (uint32_t)((lane & 7) + ((lane >> 3) & 1) * 8) * L::kQPitch + (uint32_t)(lane >> 4) * 16u;
    const int k_row = (lane & 7) + (lane >> 4) * 8, k_chunk = (lane >> 3) & 1;
    const int v_row = (lane & 7) + ((lane >> 3) & 1) * 8, v_chunk = lane >> 4;
    const int sw = lane & 7;  // the row's place in its swizzle atom, of k_row and v_row alike
    // where a tile's row begins (its first 64 columns; the next ones `half` bytes on)
    const uint32_t half = (uint32_t)g.box * 128u;
    const auto row_at = [&](int row) {
        const uint32_t box = (uint32_t)row / (uint32_t)g.box;
        return box * (uint32_t)g.box * (uint32_t)(D * 2) + ((uint32_t)row - box * (uint32_t)g.box) * 128u;
    };
    const uint32_t k_at = row_at(slice * kWarpKeys + k_row), v_at = row_at(slice * kWarpKeys + v_row);
    // an item's queries (rows past the last are zero): asked for while the item before
    // is being merged
    constexpr int kQLoads = 16 * (D / 8) / kGroupThreads;
    uint4 queries[kQLoads];
    const auto load_queries = [&](const Place &at, const Sequence &s) {
        const int64_t row0 = (int64_t)at.rb * kRows + 16 * group;
#pragma unroll
        for (int e = 0; e < kQLoads; ++e) {
            const int i = tid + e * kGroupThreads;
            const int64_t row = row0 + i / (D / 8);
            queries[e] = make_uint4(0, 0, 0, 0);
            if (row < (int64_t)s.n * g.group) {
                const int64_t token = s.start + row / g.group, head = (int64_t)at.h * g.group + row % g.group;
                queries[e] = *reinterpret_cast<const uint4 *>(p.q + token * p.q_token + head * p.q_head + i % (D / 8) * 8);
            }
        }
    };
    load_queries(at, s);
    int n = 0;
    bool ok = true;
    int4 record = make_int4(-1, 0, 0, 0);
    int64_t pos = first;
    for (int64_t left = mine; left > 0;) {
        const int keys = block_keys(g, s, at.rb, kRows);
        const Piece piece = take_piece<kKeys, kItemCost>(g, s, at, kRows, left);
        if (piece.empty()) break;  // the stretch ends here, before the item's first tile
        const int64_t row0 = (int64_t)at.rb * kRows + 16 * group;  // the group's first row
        const int rows = (int)min((int64_t)16, max((int64_t)0, (int64_t)s.n * g.group - row0));
        group_barrier(group);  // the previous item's merge has been read
#pragma unroll
        for (int e = 0; e < kQLoads; ++e) {
            const int i = tid + e * kGroupThreads;
            *reinterpret_cast<uint4 *>(q_smem + i / (D / 8) * L::kQPitch + i % (D / 8) * 16) = queries[e];
        }
        int kept[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = 8 * e + (lane >> 2);
            kept[e] = r < rows ? kept_keys(g, s, (int)((row0 + r) / g.group)) : 0;
        }
        // every row of the item keeps the keys below this
        const int kept_all = kept_keys(g, s, (int)((int64_t)at.rb * kRows / g.group));
        group_barrier(group);

        float o[D / 8][4], shift[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
#pragma unroll
        for (int c = 0; c < D / 8; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[c][e] = 0.f;
        for (int t = piece.t0; t < piece.t1; ++t, ++n) {
            const int stage = n % kStages;
            if (ok)
                ok = __all_sync(0xffffffffu,
                                wait_phase(full(stage), (n / kStages) & 1, abort_flag, &g_rows_error, p.wait_ns));
            if (!ok) break;
            const uint32_t ks = base + L::kOffRing + (uint32_t)stage * 2u * L::kTile;
            const uint32_t vs = ks + L::kTile;
            const int j0 = t * kKeys + slice * kWarpKeys;  // this warp's first key
            float x[2][4];
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[c][e] = 0.f;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                uint32_t kf[4], qf[4];
                const int chunk = 2 * kk + k_chunk;
                ldmatrix4(ks + k_at + (uint32_t)(chunk >> 3) * half + (uint32_t)(((chunk & 7) ^ sw) << 4), kf);
                ldmatrix4(q_lane + (uint32_t)kk * 32u, qf);
                mma16816<T>(x[0], qf, kf[0], kf[1]);
                mma16816<T>(x[1], qf, kf[2], kf[3]);
            }
            if (j0 + kWarpKeys > kept_all) {
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (j0 + 8 * c + 2 * (lane & 3) + (e & 1) >= kept[e >> 1]) x[c][e] = -INFINITY;
                // infinite and NaN values of this warp's keys out of the tile; each group
                // does so before it uses the tile, the flag first: whoever finds a zero
                // in a value's place finds the flag
                for (int i = lane; i < kWarpKeys * (D / 8); i += 32) {
                    const int r = slice * kWarpKeys + i / (D / 8), c = i % (D / 8);
                    uint4 *const at_v = reinterpret_cast<uint4 *>(gbase + (vs - base) + row_at(r) + (c >> 3) * half +
                                                                  (((c & 7) ^ (r & 7)) << 4));
                    const uint4 w = *at_v;
                    const uint4 f = make_uint4(finite_or_zero<T>(w.x), finite_or_zero<T>(w.y), finite_or_zero<T>(w.z),
                                               finite_or_zero<T>(w.w));
                    if (f.x != w.x || f.y != w.y || f.z != w.z || f.w != w.w) {
                        if (t * kKeys + r < s.keys) {  // (rows past the last key are leftovers)
                            *bad = 1u;
                            __threadfence_block();
                        }
                        *at_v = f;
                    }
                }
                fence_proxy_async_smem();  // before the next copy into this tile
                __syncwarp();
            }
            uint32_t pf[4];
            bool moved = false;
            float scale[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float mx = fmaxf(fmaxf(x[0][2 * e], x[0][2 * e + 1]), fmaxf(x[1][2 * e], x[1][2 * e + 1]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)) * g.kscale;
                scale[e] = 1.f;
                if (mx > shift[e] + (kShiftBelow<T> + kShiftSlack)) {
                    const float to = mx - kShiftBelow<T>;
                    scale[e] = ex2(shift[e] - to);  // 0 from -inf
                    shift[e] = to;
                    sum[e] *= scale[e];
                    moved = true;
                }
                const float below = safe_shift(shift[e]);
                const float p0 = ex2(fmaf(x[0][2 * e], g.kscale, -below));
                const float p1 = ex2(fmaf(x[0][2 * e + 1], g.kscale, -below));
                const float p2 = ex2(fmaf(x[1][2 * e], g.kscale, -below));
                const float p3 = ex2(fmaf(x[1][2 * e + 1], g.kscale, -below));
                sum[e] += (p0 + p1) + (p2 + p3);
                pf[e] = pack2<T>(p0, p1);
                pf[2 + e] = pack2<T>(p2, p3);
            }
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int c = 0; c < D / 8; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[c][e] *= scale[e >> 1];
            }
#pragma unroll
            for (int cc = 0; cc < D / 16; ++cc) {
                uint32_t vf[4];
                const int chunk = 2 * cc + v_chunk;
                ldmatrix4_trans(vs + v_at + (uint32_t)(chunk >> 3) * half + (uint32_t)(((chunk & 7) ^ sw) << 4), vf);
                mma16816<T>(o[2 * cc], pf, vf[0], vf[1]);
                mma16816<T>(o[2 * cc + 1], pf, vf[2], vf[3]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty(stage));
        }
        if (*bad) {
            // values set to zero (in this item or an earlier one) back to the rows that
            // keep them, as the caller's memory has them
            for (int t = max(piece.t0, kept_all / kKeys); t < piece.t1; ++t)
                for (int i = 0; i < kWarpKeys; ++i) {
                    const int j = t * kKeys + slice * kWarpKeys + i;
                    if (j < kept_all / kWarpKeys * kWarpKeys || j >= keys) continue;
                    const int2 place = locate(g, s, at.b, j);
                    if (place.x < 0 || place.x >= g.pages) continue;
                    const uint16_t *v = g.v + place.x * g.v_page + place.y * g.v_token + at.h * g.v_head;
#pragma unroll
                    for (int c = 0; c < D / 8; ++c)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t bits = v[8 * c + 2 * (lane & 3) + e];
                            if (finite_or_zero<T>(bits) == bits) continue;
                            const float f = Elem<T>::pair(bits).x;
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                if (j < kept[h]) o[c][2 * h + e] += f;
                        }
                }
        }

        Place next = at;
        Sequence next_s = s;
        if (left > piece.count) {
            next_item(g, next, next_s, kRows);
            load_queries(next, next_s);
        }

        // ---- the four warps' states become the group's ----------------------
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float l = sum[e];
            l += __shfl_xor_sync(0xffffffffu, l, 1);
            l += __shfl_xor_sync(0xffffffffu, l, 2);
            if ((lane & 3) == 0) merge_state[slice * 16 + 8 * e + (lane >> 2)] = make_float2(shift[e], l);
        }
        const bool whole = piece.whole();
        const int64_t part = piece.part();
        static_assert(16 * L::kCols / 4 == kGroupThreads, "four columns of a row to each thread");
        const int r = tid / (L::kCols / 4), c4 = tid % (L::kCols / 4) * 4;
        float weight[kWarps], all = 0.f, common = -INFINITY;
        bool good = ok;  // and every other warp of the group has had its tiles
#pragma unroll
        for (int c0 = 0; c0 < D; c0 += L::kCols) {
            group_barrier(group);  // Q (or the previous columns) has been read
#pragma unroll
            for (int c = 0; c < L::kCols / 8; ++c)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    *reinterpret_cast<float2 *>(merge + (slice * 16 + 8 * e + (lane >> 2)) * L::kColPitch + 8 * c +
                                                2 * (lane & 3)) =
                        make_float2(o[c0 / 8 + c][2 * e], o[c0 / 8 + c][2 * e + 1]);
            group_barrier(group);
            if (c0 == 0) {
                good = ok && !*abort_flag;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) common = fmaxf(common, merge_state[w * 16 + r].x);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float2 st = merge_state[w * 16 + r];
                    weight[w] = ex2(st.x - safe_shift(common));
                    all += st.y * weight[w];
                }
            }
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                // a weight of zero too: infinite and NaN values of keys that the row keeps
                // reach it (a warp whose keys it does not keep holds zeros)
                const float4 v = *reinterpret_cast<const float4 *>(merge + (w * 16 + r) * L::kColPitch + c4);
                acc.x += v.x * weight[w], acc.y += v.y * weight[w];
                acc.z += v.z * weight[w], acc.w += v.w * weight[w];
            }
            if (r < rows && good) {
                if (whole) {
                    const int64_t row = row0 + r;
                    const int64_t token = s.start + row / g.group, head = (int64_t)at.h * g.group + row % g.group;
                    const float inv = all == 0.f ? 0.f : 1.f / all;
                    uint2 w;
                    w.x = pack2<T>(acc.x * inv, acc.y * inv);
                    w.y = pack2<T>(acc.z * inv, acc.w * inv);
                    *reinterpret_cast<uint2 *>(g.o + token * g.o_token + head * g.o_head + c0 + c4) = w;
                    if (g.lse && c0 == 0 && c4 == 0) g.lse[token * g.heads + head] = natural_lse(common, all);
                } else {
                    const int64_t row = part * kRows + 16 * group + r;
                    *reinterpret_cast<float4 *>(p.parts + row * D + c0 + c4) = acc;
                    if (c0 == 0 && c4 == 0) p.states[row] = make_float2(common, all);
                }
            }
        }
        if (!whole && piece.t0 == 0 && good)
            record = make_int4(at.b, at.rb, at.h, last_block<kItemCost>(piece, at, pos, stretch));
        pos += piece.count;
        left -= piece.count;
        at = next;
        s = next_s;
    }
    if (threadIdx.x == 0) p.records[blockIdx.x] = *abort_flag ? make_int4(-1, 0, 0, 0) : record;
}

// The cut items: block (x, y) merges rows y, y + gridDim.y, ... of the item that
// begins in block x of the kernel above.  A warp takes every kJoinWarps-th part
// of a row, lane by lane D / 32 columns, so that all parts are on their way at
// once (a thread that walks 19 parts of a long context one by one took 8 us);
// the warps' sums are added in order.
// (gridDim.y: the rows of an average item, at most 8 of each row group.  8 instead of
// 4: five tokens of 40/8 heads, 25 rows, 3394 keys, 22.8 -> 14.1 us; 14970 keys of
// one head, 27.2 -> 22.7; 16 where items have few rows are blocks for nothing, 10.6 ->
// 12.8 for one token of 32/8 heads.  What it costs: items that are not cut get their
// blocks all the same, 9.7 -> 11.7 for 14 prompts of 18 rows on average.)
constexpr int kJoinWarps = 8;
template <typename T, int D, int NG>
__global__ void __launch_bounds__(kJoinWarps * 32) k_rows_join(const __grid_constant__ RowsParams p) {
    constexpr int kRows = 16 * NG, V = D / 32;
    __shared__ float sums[kJoinWarps][D];
    pdl_enter();
    const Geometry &g = p.g;
    const int4 rec = p.records[blockIdx.x];
    if (rec.x < 0) return;
    const Sequence s = load_sequence(g, rec.x);
    const int rows = (int)min((int64_t)kRows, (int64_t)s.n * g.group - (int64_t)rec.y * kRows);
    const int warp = (int)(threadIdx.x >> 5), lane = (int)(threadIdx.x & 31);
    const int first = (int)blockIdx.x, last = rec.w;
    // part of block b: it holds the item's beginning only if b is the first
    const auto part = [first](int b) { return 2 * (int64_t)b + (b == first ? 1 : 0); };
    for (int r = (int)blockIdx.y; r < rows; r += (int)gridDim.y) {
        float acc[V], shift = -INFINITY, all = 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = 0.f;
        for (int b = first + lane; b <= last; b += 32) shift = fmaxf(shift, p.states[part(b) * kRows + r].x);
#pragma unroll
        for (int o = 16; o; o >>= 1) shift = fmaxf(shift, __shfl_xor_sync(0xffffffffu, shift, o));
        const float base = safe_shift(shift);
        for (int b = first + lane; b <= last; b += 32) {
            const float2 st = p.states[part(b) * kRows + r];
            all += st.y * ex2(st.x - base);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
#pragma unroll 4
        for (int b = first + warp; b <= last; b += kJoinWarps) {
            const float w = ex2(p.states[part(b) * kRows + r].x - base);
            const float *o = p.parts + (part(b) * kRows + r) * D + lane * V;
            float v[V];
            if constexpr (V == 4) *reinterpret_cast<float4 *>(v) = *reinterpret_cast<const float4 *>(o);
            else *reinterpret_cast<float2 *>(v) = *reinterpret_cast<const float2 *>(o);
#pragma unroll
            for (int e = 0; e < V; ++e) acc[e] += v[e] * w;
        }
        __syncthreads();  // the previous row's sums have been read
#pragma unroll
        for (int e = 0; e < V; ++e) sums[warp][lane * V + e] = acc[e];
        __syncthreads();
        const int c = 2 * (int)threadIdx.x;
        if (c < D) {
            float2 o = make_float2(0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kJoinWarps; ++w) o.x += sums[w][c], o.y += sums[w][c + 1];
            const int64_t row = (int64_t)rec.y * kRows + r;
            const int64_t token = s.start + row / g.group, head = (int64_t)rec.z * g.group + row % g.group;
            const float inv = all == 0.f ? 0.f : 1.f / all;
            *reinterpret_cast<uint32_t *>(g.o + token * g.o_token + head * g.o_head + c) = pack2<T>(o.x * inv, o.y * inv);
            if (g.lse && c == 0) g.lse[token * g.heads + head] = natural_lse(shift, all);
        }
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// Row groups of a block: by the query rows that an average sequence has at one
// key/value head.
int row_groups(const softmax_sequence_args_t &a) {
    const int64_t rows = a.tokens * (a.heads / a.kv_heads);
    return rows <= 16 * a.batch ? 1 : 2;
}
int blocks_of(int groups, int sms) { return (groups == 1 ? kBlocksPerSm<1> : kBlocksPerSm<2>)*sms; }

int64_t align256(int64_t n) { return (n + 255) / 256 * 256; }

struct Space {
    int64_t records, states, parts, bytes;
};
Space space(int64_t blocks, int64_t rows, int64_t head_dim) {
    Space s;
    s.records = 0;
    s.states = s.records + align256(blocks * (int64_t)sizeof(int4));
    s.parts = s.states + align256(2 * blocks * rows * (int64_t)sizeof(float2));
    s.bytes = s.parts + align256(2 * blocks * rows * head_dim * (int64_t)sizeof(float));
    return s;
}

template <typename T, int D, int NG>
cudaError_t go(const AttnCall &c) {
    using L = Layout<D, NG>;
    static std::atomic<unsigned long long> opted{0};
    cudaError_t e = opt_in_shared_memory((const void *)k_seq_rows<T, D, NG>, (int)L::kBytes, opted);
    if (e != cudaSuccess) return e;
    RowsParams p;
    CUtensorMap tk, tv;
    if (!fill_geometry(c, kKeys, &p.g) ||
        !make_row_map(&tk, c.a.k, c, p.g.box, c.a.k_token_stride, c.a.k_head_stride, c.a.k_page_stride) ||
        !make_row_map(&tv, c.a.v, c, p.g.box, c.a.v_token_stride, c.a.v_head_stride, c.a.v_page_stride))
        return cudaErrorInvalidValue;
    const Space sp = space(blocks_of(NG, c.sms), L::kRows, D);
    uint8_t *const w = (uint8_t *)c.workspace;
    p.q = (const uint16_t *)c.a.q;
    p.q_token = c.a.q_token_stride;
    p.q_head = c.a.q_head_stride;
    p.records = reinterpret_cast<int4 *>(w + sp.records);
    p.states = reinterpret_cast<float2 *>(w + sp.states);
    p.parts = reinterpret_cast<float *>(w + sp.parts);
    p.wait_ns = wait_limit(c.wait_ns);
    p.starve = c.starve;
    const int64_t rows = c.a.tokens * p.g.group;
    const int64_t blocks = blocks_with_work(p.g, rows / L::kRows + c.a.batch, kKeys, kItemCost, blocks_of(NG, c.sms));
    const int64_t join_rows = std::min<int64_t>((rows + c.a.batch - 1) / c.a.batch, 8 * NG);
    LaunchArgs l = {};
    l.stream = c.stream;
    l.overlap = c.overlap;
    e = launch_kernel(k_seq_rows<T, D, NG>, l, blocks, kThreads<NG>, L::kBytes, 0, tk, tv, p);
    if (e != cudaSuccess) return e;
    return launch_kernel_2d(k_rows_join<T, D, NG>, c, dim3((unsigned)blocks, (unsigned)join_rows), kJoinWarps * 32, p);
}

template <typename T, int D>
cudaError_t go_rows(const AttnCall &c) {
    return row_groups(c.a) == 1 ? go<T, D, 1>(c) : go<T, D, 2>(c);
}

}  // namespace

int64_t rows_workspace_bytes(const softmax_sequence_args_t &a, int sms) {
    const int groups = row_groups(a);
    return space(blocks_of(groups, sms), 16 * groups, a.head_dim).bytes;
}

cudaError_t launch_rows(const AttnCall &c) {
    if (c.a.dtype == SOFTMAX_BF16)
        return c.a.head_dim == 128 ? go_rows<__nv_bfloat16, 128>(c) : go_rows<__nv_bfloat16, 64>(c);
    return c.a.head_dim == 128 ? go_rows<__half, 128>(c) : go_rows<__half, 64>(c);
}

cudaError_t read_clear_rows_error_word(unsigned int *word) {
    cudaError_t e = cudaMemcpyFromSymbol(word, g_rows_error, sizeof(unsigned int), 0, cudaMemcpyDeviceToHost);
    if (e != cudaSuccess) return e;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(g_rows_error, &zero, sizeof(unsigned int), 0, cudaMemcpyHostToDevice);
}

}  // namespace seq
}  // namespace mbrs
