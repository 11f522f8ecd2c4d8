// sequence_abi.cu -- the C ABI declared in include/mbrs_sequence.h: argument
// checks, then the launches (k_seq_rows.cu, k_seq_tiles.cu,
// k_cache_append.cu).
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "attention_launch.h"
#include "launch.h"
#include "mbrs_sequence.h"
#include "sequence_launch.h"
#include "sequence_rules.h"

using namespace mbrs;

namespace {

constexpr int64_t kInt = 0x7fffffff;
constexpr int64_t kMaxStride = (1ll << 39);  // elements: 2^40 bytes

// A 16-bit tensor of up to four dimensions, the last one `inner` contiguous
// elements: dimensions of size 1 have no stride to check.
struct View {
    const void *ptr;
    int64_t inner;
    int64_t n[3], stride[3];
};

int check_view(const View &v, bool written, uint64_t *bytes) {
    int64_t last = v.inner;  // elements up to the end of the last row
    int64_t size[3], step[3];
    int d = 0;
    for (int i = 0; i < 3; ++i) {
        if (v.n[i] <= 1) continue;
        if (v.stride[i] < v.inner || v.stride[i] % 8 != 0 || v.stride[i] >= kMaxStride) return SOFTMAX_ERR_STRIDE;
        if (v.n[i] - 1 > (INT64_MAX / 4 - last) / v.stride[i]) return SOFTMAX_ERR_SHAPE;
        last += (v.n[i] - 1) * v.stride[i];
        size[d] = v.n[i], step[d] = v.stride[i], ++d;
    }
    if (written) {  // no two rows share elements: sorted by stride, each dimension steps over the ones inside it
        for (int i = 0; i < d; ++i)
            for (int j = i + 1; j < d; ++j)
                if (step[j] < step[i]) std::swap(step[i], step[j]), std::swap(size[i], size[j]);
        int64_t extent = v.inner;
        for (int i = 0; i < d; ++i) {
            if (step[i] < extent) return SOFTMAX_ERR_STRIDE;
            extent += (size[i] - 1) * step[i];
        }
    }
    *bytes = (uint64_t)last * 2;
    return SOFTMAX_OK;
}

// Whether two views share an element, `delta` elements from a's first to b's
// first, looking at their dimensions from `level` on (strides falling).  Views
// that step together (the queries and keys of one fused buffer, the halves of
// one cache) are told apart by where they lie within the step; others count as
// sharing where their extents meet.
struct Steps {
    int64_t inner;
    int count = 0;
    int64_t n[3], stride[3];
    explicit Steps(const View &v) : inner(v.inner) {
        for (int i = 0; i < 3; ++i)
            if (v.n[i] > 1) n[count] = v.n[i], stride[count] = v.stride[i], ++count;
        for (int i = 0; i < count; ++i)
            for (int j = i + 1; j < count; ++j)
                if (stride[j] > stride[i]) std::swap(stride[i], stride[j]), std::swap(n[i], n[j]);
    }
    int64_t extent(int level) const {
        int64_t e = inner;
        for (int i = level; i < count; ++i) e += (n[i] - 1) * stride[i];
        return e;
    }
};
bool steps_meet(const Steps &a, const Steps &b, int level, int64_t delta) {
    if (delta >= a.extent(level) || -delta >= b.extent(level)) return false;
    if (level >= a.count || level >= b.count || a.stride[level] != b.stride[level]) return true;
    const int64_t step = a.stride[level];
    if (a.extent(level + 1) > step || b.extent(level + 1) > step) return true;
    const int64_t r = ((delta % step) + step) % step;
    return steps_meet(a, b, level + 1, r) || steps_meet(a, b, level + 1, r - step);
}
bool views_meet(const View &a, const View &b) {
    const int64_t delta = (int64_t)((uint64_t)(uintptr_t)b.ptr - (uint64_t)(uintptr_t)a.ptr) / 2;
    return steps_meet(Steps(a), Steps(b), 0, delta);
}

struct Span {
    uint64_t lo, hi;
};
bool meet(const Span &a, const Span &b) { return a.lo < b.hi && b.lo < a.hi; }

// The span of a pointer's bytes: SOFTMAX_ERR_NULL, _ALIGN or _SHAPE where it has none.
int span_of(const void *p, uint64_t bytes, uint64_t align, Span *s) {
    if (!p) return SOFTMAX_ERR_NULL;
    const uint64_t a = (uint64_t)(uintptr_t)p;
    if (a % align) return SOFTMAX_ERR_ALIGN;
    if (a > UINT64_MAX - bytes) return SOFTMAX_ERR_SHAPE;
    *s = Span{a, a + bytes};
    return SOFTMAX_OK;
}

int check_types(int dtype, int64_t head_dim) {
    if (dtype != SOFTMAX_F32 && dtype != SOFTMAX_F16 && dtype != SOFTMAX_BF16) return SOFTMAX_ERR_DTYPE;
    if (dtype == SOFTMAX_F32 || (head_dim != 64 && head_dim != 128)) return SOFTMAX_ERR_UNSUPPORTED;
    return SOFTMAX_OK;
}

int check_pages(int64_t pages, int64_t page_size, int64_t max_pages) {
    if (pages < 1 || page_size < 1 || max_pages < 1 || pages > kInt || page_size > kInt) return SOFTMAX_ERR_SHAPE;
    if (max_pages > (kInt - 1024) / page_size) return SOFTMAX_ERR_SHAPE;  // room to round a key count up
    return page_size % 8 ? SOFTMAX_ERR_UNSUPPORTED : SOFTMAX_OK;
}

int check_sizes(const softmax_sequence_args_t &a, bool paged) {
    if (a.tokens < 0 || a.batch < 0 || a.heads < 1 || a.kv_heads < 1 || a.head_dim < 1) return SOFTMAX_ERR_SHAPE;
    int st = check_types(a.dtype, a.head_dim);
    if (st != SOFTMAX_OK) return st;
    if (a.causal != 0 && a.causal != 1) return SOFTMAX_ERR_ARG;
    if (a.heads % a.kv_heads) return SOFTMAX_ERR_SHAPE;
    if (a.heads / a.kv_heads > 128) return SOFTMAX_ERR_UNSUPPORTED;
    if (a.tokens > kInt - 1024 || a.batch > kInt - 1024 || a.heads > 65535) return SOFTMAX_ERR_SHAPE;
    return paged ? check_pages(a.pages, a.page_size, a.max_pages) : SOFTMAX_OK;
}

bool few_rows(const softmax_sequence_args_t &a) { return seq::few_rows(a.tokens, a.batch, a.heads / a.kv_heads); }

int64_t workspace_bytes_of(const softmax_sequence_args_t &a, int sms) {
    return few_rows(a) ? seq::rows_workspace_bytes(a, sms) : seq::tiles_workspace_bytes(a, sms);
}

int attention_call(const softmax_sequence_args_t *args, bool paged, void *workspace, int64_t workspace_bytes,
                   cudaStream_t stream) {
    if (!args) return SOFTMAX_ERR_ARG;
    const softmax_sequence_args_t &a = *args;
    int st = check_sizes(a, paged);
    if (st != SOFTMAX_OK) return st;
    if (!(a.sm_scale > 0.f) || !std::isfinite(a.sm_scale)) return SOFTMAX_ERR_ARG;
    if (!paged && (a.kv_lens || a.page_table || a.pages || a.page_size || a.max_pages)) return SOFTMAX_ERR_ARG;
    if (a.tokens == 0 || a.batch == 0) return SOFTMAX_OK;
    const int64_t d = a.head_dim;
    uint64_t qb, kb, vb, ob;
    const View q{a.q, d, {a.tokens, a.heads, 1}, {a.q_token_stride, a.q_head_stride, 0}};
    const View o{a.o, d, {a.tokens, a.heads, 1}, {a.o_token_stride, a.o_head_stride, 0}};
    const int64_t rows = paged ? a.page_size : a.tokens, pages = paged ? a.pages : 1;
    const View k{a.k, d, {rows, a.kv_heads, pages}, {a.k_token_stride, a.k_head_stride, a.k_page_stride}};
    const View v{a.v, d, {rows, a.kv_heads, pages}, {a.v_token_stride, a.v_head_stride, a.v_page_stride}};
    if ((st = check_view(q, false, &qb)) || (st = check_view(k, false, &kb)) || (st = check_view(v, false, &vb)) ||
        (st = check_view(o, true, &ob)))
        return st;
    if (paged && (a.table_stride < a.max_pages || a.table_stride >= kMaxStride)) return SOFTMAX_ERR_STRIDE;
    Span sq, sk, sv, so, sl{0, 0}, ss, sn{0, 0}, sp{0, 0}, sw;
    if ((st = span_of(a.q, qb, 16, &sq)) || (st = span_of(a.k, kb, 16, &sk)) || (st = span_of(a.v, vb, 16, &sv)) ||
        (st = span_of(a.o, ob, 16, &so)) || (st = span_of(a.q_starts, (uint64_t)(a.batch + 1) * 4, 4, &ss)))
        return st;
    if (a.lse && (st = span_of(a.lse, (uint64_t)(a.tokens * a.heads) * 4, 4, &sl))) return st;
    if (paged && ((st = span_of(a.kv_lens, (uint64_t)a.batch * 4, 4, &sn)) ||
                  (st = span_of(a.page_table, (uint64_t)((a.batch - 1) * a.table_stride + a.max_pages) * 4, 4, &sp))))
        return st;
    const Span in[6] = {sq, sk, sv, ss, sn, sp};
    if (a.lse)
        for (const Span &x : in)
            if (meet(sl, x)) return SOFTMAX_ERR_OVERLAP;
    if (views_meet(o, q) || views_meet(o, k) || views_meet(o, v) || meet(so, ss) || meet(so, sn) || meet(so, sp) ||
        (a.lse && meet(so, sl)))
        return SOFTMAX_ERR_OVERLAP;
    int sms = 0;
    st = host_device_sms(&sms);
    if (st != SOFTMAX_OK) return st;
    const int64_t need = workspace_bytes_of(a, sms);
    if (workspace_bytes < need) return SOFTMAX_ERR_SCRATCH_LIMIT;
    if ((st = span_of(workspace, (uint64_t)need, 256, &sw))) return st;
    for (const Span &x : in)
        if (meet(sw, x)) return SOFTMAX_ERR_OVERLAP;
    if (meet(sw, so) || (a.lse && meet(sw, sl))) return SOFTMAX_ERR_OVERLAP;
    const seq::AttnCall call{a, paged, workspace, sms, host_wait_ns(), attn::attention_starve(),
                             host_launch_overlap(), stream};
    const cudaError_t e = few_rows(a) ? seq::launch_rows(call) : seq::launch_tiles(call);
    return e == cudaSuccess ? SOFTMAX_OK : SOFTMAX_ERR_CUDA;
}

}  // namespace

cudaError_t mbrs::seq::read_clear_sequence_error_word(unsigned int *word) {
    unsigned int rows = 0, tiles = 0;
    cudaError_t e = read_clear_rows_error_word(&rows);
    if (e == cudaSuccess) e = read_clear_tiles_error_word(&tiles);
    *word = rows | tiles;
    return e;
}

extern "C" {

int softmax_attention_varlen_fwd(const softmax_sequence_args_t *args, void *workspace, int64_t workspace_bytes,
                                 cudaStream_t stream) {
    return attention_call(args, false, workspace, workspace_bytes, stream);
}

int softmax_attention_paged_fwd(const softmax_sequence_args_t *args, void *workspace, int64_t workspace_bytes,
                                cudaStream_t stream) {
    return attention_call(args, true, workspace, workspace_bytes, stream);
}

int64_t softmax_sequence_workspace_bytes(const softmax_sequence_args_t *args) {
    if (!args) return -SOFTMAX_ERR_ARG;
    int st = check_sizes(*args, args->page_table != nullptr);
    if (st != SOFTMAX_OK) return -st;
    if (args->tokens == 0 || args->batch == 0) return 0;
    int sms = 0;
    st = host_device_sms(&sms);
    if (st != SOFTMAX_OK) return -st;
    return workspace_bytes_of(*args, sms);
}

int softmax_kv_cache_append(const softmax_append_args_t *args, cudaStream_t stream) {
    if (!args) return SOFTMAX_ERR_ARG;
    const softmax_append_args_t &a = *args;
    if (a.tokens < 0 || a.batch < 0 || a.kv_heads < 1 || a.head_dim < 1 || a.heads < 0) return SOFTMAX_ERR_SHAPE;
    int st = check_types(a.dtype, a.head_dim);
    if (st != SOFTMAX_OK) return st;
    if ((a.q != nullptr) != (a.q_out != nullptr) || (a.q != nullptr) != (a.heads > 0)) return SOFTMAX_ERR_ARG;
    if (a.interleaved != 0 && a.interleaved != 1) return SOFTMAX_ERR_ARG;
    if (a.rotary_dim < 0 || a.rotary_dim > a.head_dim || a.rotary_dim % 16 ||
        (a.inv_freq != nullptr) != (a.rotary_dim > 0))
        return SOFTMAX_ERR_ARG;
    if (a.tokens > kInt - 1024 || a.batch > kInt - 1024 || a.heads > 65535 || a.kv_heads > 65535)
        return SOFTMAX_ERR_SHAPE;
    st = check_pages(a.pages, a.page_size, a.max_pages);
    if (st != SOFTMAX_OK) return st;
    if (a.tokens == 0 || a.batch == 0) return SOFTMAX_OK;
    const int64_t d = a.head_dim;
    uint64_t kb, vb, kcb, vcb, qb = 0, ob = 0;
    const View k{a.k, d, {a.tokens, a.kv_heads, 1}, {a.k_token_stride, a.k_head_stride, 0}};
    const View v{a.v, d, {a.tokens, a.kv_heads, 1}, {a.v_token_stride, a.v_head_stride, 0}};
    const View kc{a.k_cache, d, {a.page_size, a.kv_heads, a.pages},
                  {a.k_cache_token_stride, a.k_cache_head_stride, a.k_cache_page_stride}};
    const View vc{a.v_cache, d, {a.page_size, a.kv_heads, a.pages},
                  {a.v_cache_token_stride, a.v_cache_head_stride, a.v_cache_page_stride}};
    if ((st = check_view(k, false, &kb)) || (st = check_view(v, false, &vb)) || (st = check_view(kc, true, &kcb)) ||
        (st = check_view(vc, true, &vcb)))
        return st;
    const View q{a.q, d, {a.tokens, a.heads, 1}, {a.q_token_stride, a.q_head_stride, 0}};
    const View o{a.q_out, d, {a.tokens, a.heads, 1}, {a.q_out_token_stride, a.q_out_head_stride, 0}};
    Span sk, sv, skc, svc, sq, so{0, 0}, ss, sn, sp, sf{0, 0};
    if ((st = span_of(a.k, kb, 16, &sk)) || (st = span_of(a.v, vb, 16, &sv)) ||
        (st = span_of(a.k_cache, kcb, 16, &skc)) || (st = span_of(a.v_cache, vcb, 16, &svc)))
        return st;
    if (a.q) {
        if ((st = check_view(q, false, &qb)) || (st = check_view(o, true, &ob)) || (st = span_of(a.q, qb, 16, &sq)) ||
            (st = span_of(a.q_out, ob, 16, &so)))
            return st;
    }
    if (a.table_stride < a.max_pages || a.table_stride >= kMaxStride) return SOFTMAX_ERR_STRIDE;
    if ((st = span_of(a.q_starts, (uint64_t)(a.batch + 1) * 4, 4, &ss)) ||
        (st = span_of(a.kv_lens, (uint64_t)a.batch * 4, 4, &sn)) ||
        (st = span_of(a.page_table, (uint64_t)((a.batch - 1) * a.table_stride + a.max_pages) * 4, 4, &sp)))
        return st;
    if (a.inv_freq && (st = span_of(a.inv_freq, (uint64_t)a.rotary_dim * 2, 4, &sf))) return st;
    // the caches and q_out are written; q_out may be q itself, row for row
    const Span in[4] = {ss, sn, sp, sf};
    for (const Span &x : in)
        if (meet(skc, x) || meet(svc, x) || meet(so, x)) return SOFTMAX_ERR_OVERLAP;
    const View *cache[2] = {&kc, &vc}, *source[2] = {&k, &v};
    for (const View *c : cache)
        if (views_meet(*c, k) || views_meet(*c, v) || (a.q && (views_meet(*c, q) || views_meet(*c, o))))
            return SOFTMAX_ERR_OVERLAP;
    if (views_meet(kc, vc)) return SOFTMAX_ERR_OVERLAP;
    if (a.q) {
        for (const View *s : source)
            if (views_meet(o, *s)) return SOFTMAX_ERR_OVERLAP;
        const bool in_place = a.q == a.q_out && (a.tokens == 1 || a.q_token_stride == a.q_out_token_stride) &&
                              (a.heads == 1 || a.q_head_stride == a.q_out_head_stride);
        if (!in_place && views_meet(q, o)) return SOFTMAX_ERR_OVERLAP;
    }
    return seq::launch_append(a, host_launch_overlap(), stream) == cudaSuccess ? SOFTMAX_OK : SOFTMAX_ERR_CUDA;
}

}  // extern "C"
