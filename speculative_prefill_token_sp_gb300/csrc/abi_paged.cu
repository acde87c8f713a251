// extern "C" entry points of the rotary positions, the paged cache and the
// attention over it (declared in include/specprefill.h).  Arguments are checked
// here, before anything is enqueued.
#include "paged.cuh"

#include <float.h>
#include <string.h>

#include <algorithm>
#include <atomic>
#include <initializer_list>

namespace sp {

// Implemented in rotary.cu, cache.cu and attend_*.cu.
sp_status rotary_launch(const sp_rotary_plan& plan, const int32_t* pos, int64_t pos_stride, int64_t T, int d,
                        sp_dtype dtype, bool inverse, const sp_rows& q, const sp_rows& qo, int H, const sp_rows& k,
                        const sp_rows& ko, int Hk, cudaStream_t st);
sp_status cache_write_launch(const sp_cache& c, const sp_batch& b, const sp_rows& k, const sp_rows& v, void* ws,
                             cudaStream_t st);
sp_status cache_read_launch(const sp_cache& c, const sp_batch& b, const sp_rows& k, const sp_rows& v, void* ws,
                            cudaStream_t st);
size_t attend_general_ws_bytes(const sp_cache& c);
sp_status attend_general_launch(const AttendProblem& p, void* ws, cudaStream_t st);
bool attend_step_supported(const sp_cache& c);
size_t attend_step_ws_bytes(const sp_cache& c);
sp_status attend_step_launch(const AttendProblem& p, void* ws, cudaStream_t st);
bool attend_tc_supported(const sp_cache& c, const sp_batch& b, int G);
size_t attend_tc_ws_bytes(const sp_cache& c);
sp_status attend_tc_launch(const AttendProblem& p, int min_rows, void* ws, size_t offset, cudaStream_t st);
// Implemented in weights_*.cu, tree.cu and evict.cu.
sp_status weights_general_launch(const WeightsProblem& w, void* ws, cudaStream_t st);
sp_status weights_step_launch(const WeightsProblem& w, void* ws, cudaStream_t st);
bool weights_tc_supported(const sp_cache& c, const sp_batch& b, int G);
size_t weights_tc_ws_bytes();
sp_status weights_tc_launch(const WeightsProblem& w, void* ws, cudaStream_t st);
sp_status tree_seen_launch(const sp_batch& b, const int32_t* parent, uint32_t* seen, int64_t stride, int words, int32_t* positions,
                           void* ws, cudaStream_t st);
sp_status tree_accept_launch(const sp_batch& b, const int32_t* parent, const int32_t* draft, const int32_t* target, int32_t* path,
                             int64_t stride, int64_t* n_path, int32_t* next, void* ws, cudaStream_t st);
sp_status cache_choose_launch(const sp_cache& c, const sp_batch& b, const float* weights, bool shared, int64_t budget, int64_t first,
                              int64_t last, int32_t* kept, int64_t stride_seq, int64_t stride_head, int64_t* n_kept, void* ws,
                              cudaStream_t st);
sp_status cache_keep_launch(const sp_cache& c, const sp_batch& b, const int32_t* kept, int heads, int64_t stride_seq,
                            int64_t stride_head, const int64_t* n_kept, int64_t most, bool drafted, const int32_t* to, int to_width,
                            int64_t to_stride, float* weights, int64_t* kv_out, void* ws, cudaStream_t st);

namespace {

int esize(sp_dtype t) { return t == SP_BF16 ? 2 : 4; }

sp_status check_dim(const char* fn, int d, sp_dtype dtype) {
    if (d < 8 || d > 256 || d % 8 != 0) {
        set_error("%s: head dim d must be a multiple of 8 in [8, 256] (got %d)", fn, d);
        return d < 1 ? SP_EINVAL : SP_EUNSUPPORTED;
    }
    if (dtype != SP_BF16 && dtype != SP_F32) {
        set_error("%s: unknown dtype %d", fn, (int)dtype);
        return SP_EINVAL;
    }
    return SP_OK;
}

sp_status check_rows(const char* fn, const char* what, const sp_rows* r, sp_dtype dtype, int64_t rows) {
    if (r && rows == 0) return SP_OK;           // an empty tensor may have no address
    if (!r || !r->data) {
        set_error("%s: null %s", fn, what);
        return SP_EINVAL;
    }
    const int64_t step = 16 / esize(dtype);
    if (reinterpret_cast<uintptr_t>(r->data) % 16 || r->stride_row % step || r->stride_head % step) {
        set_error("%s: %s must be 16-byte aligned, with strides of a multiple of 16 bytes", fn, what);
        return SP_EINVAL;
    }
    return SP_OK;
}

// Whether places i0 * stride0 + i1 * stride1 + ... of `width` entries each lie apart, as in every tensor that slices and permutations
// make of a contiguous one: the steps of each axis pass over all that the axes of smaller steps span.
struct Axis {
    int64_t extent, stride;
};
template <int N>
bool apart(Axis (&axis)[N], int width) {
    std::sort(axis, axis + N, [](const Axis& a, const Axis& b) { return a.stride < b.stride; });
    __int128 span = width;
    for (const Axis& a : axis) {
        if (a.extent <= 1) continue;
        if (a.stride < span) return false;
        span += (__int128)(a.extent - 1) * a.stride;
    }
    return true;
}

// Rows that are written, or that a tensor map describes, must not overlap.
sp_status check_apart(const char* fn, const char* what, const sp_rows* r, int64_t rows, int heads, int d) {
    const int64_t most = (int64_t)1 << 38;
    Axis axis[2] = {{rows, r->stride_row}, {heads, r->stride_head}};
    if (rows == 0) return SP_OK;
    if ((rows > 1 && r->stride_row > most) || (heads > 1 && r->stride_head > most) || !apart(axis, d)) {
        set_error("%s: the rows of %s must not overlap, and its strides must be at most 2^38", fn, what);
        return SP_EINVAL;
    }
    return SP_OK;
}

sp_status check_workspace(const char* fn, const void* ws, size_t have, size_t need) {
    if (!ws || reinterpret_cast<uintptr_t>(ws) % 16) {
        set_error("%s: null or misaligned workspace", fn);
        return SP_EINVAL;
    }
    if (have < need) {
        set_error("%s: workspace of %zu bytes is smaller than the %zu required", fn, have, need);
        return SP_ENOMEM;
    }
    return SP_OK;
}

// f / 2 pi modulo 1 in units of 2^-64, to one and a half of them for |f| <= 2^40: a position of 2^31 multiplies the error.  1 / 2 pi is
// the sum of two doubles, and so is the product; taken of |f|, since the fraction of a small negative number would be rounded.
uint64_t fraction_of_turn(double f) {
    constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;
    const double x = fabs(f);
    const volatile double rounded = x * kHi;        // volatile: a compiler may fuse the product with what follows, and count lo twice
    const double hi = rounded, lo = fma(x, kHi, -hi) + x * kLo;
    const uint64_t u = (uint64_t)ldexp(hi - floor(hi), 64) + (uint64_t)llrint(ldexp(lo, 64));
    return f < 0 ? 0 - u : u;
}

// Which kernels a call takes.
enum Path {
    kGeneral,       // the general one
    kStep,          // every sequence has at most the 16 rows per KV head of the step kernel
    kChunks,        // one sequence with more, or a cache that the step kernel does not take
    kMixed          // the step kernel for the sequences with few rows, the tensor-core one for the others
};
Path path_of(const sp_cache& c, const sp_batch& b, int H) {
    const int G = H / c.H_kv;
    if (b.T == 0) return kGeneral;          // nothing to do but the check
    // (its join has a block for each sequence and KV head)
    const bool step = attend_step_supported(c) && (int64_t)b.B * c.H_kv <= INT32_MAX;
    if (step && (int64_t)b.max_new * G <= 16) return kStep;
    if (!attend_tc_supported(c, b, G)) return kGeneral;
    return step && b.B > 1 ? kMixed : kChunks;
}

size_t path_bytes(Path path, const sp_cache& c) {
    switch (path) {
        case kStep: return attend_step_ws_bytes(c);
        case kChunks: return attend_tc_ws_bytes(c);
        case kMixed: return attend_step_ws_bytes(c) + attend_tc_ws_bytes(c);
        default: return attend_general_ws_bytes(c);
    }
}

// Which kernel sp_attend_weights takes: as sp_attend, but a mixed batch goes to the tensor cores' kernel as a whole.
Path weights_path(const sp_cache& c, const sp_batch& b, int H) {
    const Path path = path_of(c, b, H);
    if (path == kGeneral || path == kStep) return path;
    return weights_tc_supported(c, b, H / c.H_kv) ? kChunks : kGeneral;
}

// Pages, heads and slots of a cache that is written lie apart.
sp_status check_no_overlap(const char* fn, const sp_cache* c) {
    Axis axis[3] = {{c->pages, c->stride_page}, {c->H_kv, c->stride_head}, {c->page, c->stride_slot}};
    if (apart(axis, c->d)) return SP_OK;
    set_error("%s: pages, heads or slots of the cache overlap", fn);
    return SP_EINVAL;
}

sp_status check_heads(const char* fn, const sp_cache* c, int H) {
    if (H >= 1 && H % c->H_kv == 0) return SP_OK;
    set_error("%s: H (%d) must be a multiple of H_kv (%d)", fn, H, c->H_kv);
    return SP_EINVAL;
}

sp_status check_ints(const char* fn, const char* what, const void* p) {
    if (p && reinterpret_cast<uintptr_t>(p) % 4 == 0) return SP_OK;
    set_error("%s: null or misaligned %s", fn, what);
    return SP_EINVAL;
}

sp_status check_counts(const char* fn, const char* what, const void* p) {
    if (p && reinterpret_cast<uintptr_t>(p) % 8 == 0) return SP_OK;
    set_error("%s: null or misaligned %s", fn, what);
    return SP_EINVAL;
}

// An output that is written while the inputs are read is in none of their places.
struct Span {
    const void* p;
    int64_t bytes;
};
sp_status check_apart(const char* fn, const char* what, Span out, std::initializer_list<Span> inputs) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(out.p);
    for (const Span& in : inputs) {
        const uintptr_t b = reinterpret_cast<uintptr_t>(in.p);
        if (!a || !b || a >= b + (uintptr_t)in.bytes || b >= a + (uintptr_t)out.bytes) continue;
        set_error("%s: %s is in the place of an array that is read meanwhile", fn, what);
        return SP_EINVAL;
    }
    return SP_OK;
}
Span starts_of(const sp_batch* b) { return {b->cu_new, 8 * ((int64_t)b->B + 1)}; }
Span lengths_of(const sp_batch* b) { return {b->kv_len, 8 * (int64_t)b->B}; }
// n rows of `wide` words
Span words_of(const void* p, int64_t n, int64_t stride, int64_t wide) {
    return {p, n > 0 ? 4 * ((n - 1) * std::min<int64_t>(n > 1 ? stride : 0, (int64_t)1 << 28) + wide) : 0};
}

sp_status check_weights(const char* fn, const float* w) { return check_ints(fn, "weights", w); }

// A kernel has a cluster of up to 8 CTAs for each.
sp_status check_items(const char* fn, int64_t items) {
    if (items < (int64_t)1 << 27) return SP_OK;
    set_error("%s: too many sequences and KV heads (%lld)", fn, (long long)items);
    return SP_EUNSUPPORTED;
}

sp_status check_words(const char* fn, const sp_batch* b, const uint32_t* seen, int64_t stride, int words) {
    if (b->T == 0) return SP_OK;
    sp_status s = check_ints(fn, "seen", seen);
    if (s != SP_OK) return s;
    if (words < 1 || (int64_t)32 * words < b->max_new || stride < 0) {
        set_error("%s: %d words a row do not hold %d tokens (row stride %lld)", fn, words, b->max_new, (long long)stride);
        return SP_EINVAL;
    }
    return SP_OK;
}

size_t attend_bytes(const char* fn, const sp_cache* cache, const sp_batch* batch, int H) {
    if (check_cache(fn, cache) != SP_OK || check_batch_args(fn, batch) != SP_OK || check_heads(fn, cache, H) != SP_OK) return 0;
    return path_bytes(path_of(*cache, *batch, H), *cache);
}

// What sp_attend, sp_attend_tree and sp_attend_weights have in common: checks it and fills in the problem.
sp_status attend_problem(const char* fn, const sp_rows* q, const sp_cache* cache, const sp_batch* batch, int H, double scale,
                         int64_t window, AttendProblem* out) {
    sp_status s;
    if ((s = check_cache(fn, cache)) != SP_OK || (s = check_batch_args(fn, batch)) != SP_OK || (s = check_heads(fn, cache, H)) != SP_OK)
        return s;
    const float factor = (float)scale * 1.4426950408889634f;        // the kernels': logits to base 2
    if (!(factor >= FLT_MIN) || !isfinite(factor)) {
        set_error("%s: scale must be positive, and a normal fp32 number times log2(e) (got %g)", fn, scale);
        return SP_EINVAL;
    }
    if (window < 0) {
        set_error("%s: window must be >= 0 (got %lld)", fn, (long long)window);
        return SP_EINVAL;
    }
    if ((s = check_rows(fn, "q", q, cache->dtype, batch->T)) != SP_OK || (s = check_apart(fn, "q", q, batch->T, H, cache->d)) != SP_OK)
        return s;
    AttendProblem p;
    memset(&p, 0, sizeof(p));
    if (q) p.q = *q;
    p.cache = *cache; p.batch = *batch; p.H = H; p.scale = (float)scale;
    p.window = window >= (int64_t)1 << 30 ? 0 : (int)window;       // kv_len is at most 2^30: no limit at all
    p.page_shift = -1;
    for (int i = 0; i < 31; ++i)
        if (cache->page == 1 << i) p.page_shift = i;
    *out = p;
    return SP_OK;
}

// seen: null for causal attention.
sp_status attend(const char* fn, const sp_rows* q, const sp_cache* cache, const sp_batch* batch, int H, double scale, int64_t window,
                 const uint32_t* seen, int64_t seen_stride, const sp_rows* out, float* lse, int64_t lse_stride_row,
                 int64_t lse_stride_head, void* ws, size_t ws_bytes, void* stream) {
    AttendProblem p;
    sp_status s;
    if ((s = attend_problem(fn, q, cache, batch, H, scale, window, &p)) != SP_OK) return s;
    if ((s = check_rows(fn, "out", out, cache->dtype, batch->T)) != SP_OK) return s;
    if (reinterpret_cast<uintptr_t>(lse) % 4) {
        set_error("%s: lse must be 4-byte aligned", fn);
        return SP_EINVAL;
    }
    if ((s = check_apart(fn, "out", out, batch->T, H, cache->d)) != SP_OK) return s;
    if ((s = check_workspace(fn, ws, ws_bytes, attend_bytes(fn, cache, batch, H))) != SP_OK) return s;
    if (out) p.out = *out;
    p.lse = lse; p.lse_stride_row = lse_stride_row; p.lse_stride_head = lse_stride_head;
    p.seen = seen; p.seen_stride = seen_stride;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (path_of(*cache, *batch, H)) {
        case kGeneral: s = attend_general_launch(p, ws, st); break;
        case kStep: s = attend_step_launch(p, ws, st); break;
        case kChunks: s = attend_tc_launch(p, 0, ws, 0, st); break;
        case kMixed:
            s = attend_step_launch(p, ws, st);
            if (s == SP_OK) s = attend_tc_launch(p, 16, ws, attend_step_ws_bytes(*cache), st);
            break;
    }
    if (s == SP_OK) clear_error();
    return s;
}

}  // namespace

int sm_count() {
    static std::atomic<int> known[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 152;
    if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 152;
    if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
    return n;
}

sp_status check_cache(const char* fn, const sp_cache* c) {
    if (!c || !c->k || !c->v) {
        set_error("%s: null cache, or null keys or values of it", fn);
        return SP_EINVAL;
    }
    sp_status s = check_dim(fn, c->d, c->dtype);
    if (s != SP_OK) return s;
    if (c->H_kv > 65535) {
        set_error("%s: at most 65535 KV heads (got %d)", fn, c->H_kv);
        return SP_EUNSUPPORTED;
    }
    if (c->H_kv < 1 || c->page < 1 || c->pages < 1 || c->pages > INT32_MAX) {
        set_error("%s: the cache needs H_kv, page and pages >= 1 (got %d, %d, %lld)", fn, c->H_kv, c->page,
                  (long long)c->pages);
        return SP_EINVAL;
    }
    if (c->kind != SP_CACHE_SAME && c->kind != SP_CACHE_E4M3 && c->kind != SP_CACHE_INT8) {
        set_error("%s: unknown cache kind %d", fn, (int)c->kind);
        return SP_EINVAL;
    }
    const bool same = c->kind == SP_CACHE_SAME;
    if (!same && (!c->k_scale || !c->v_scale)) {
        set_error("%s: a cache of 8-bit codes needs k_scale and v_scale", fn);
        return SP_EINVAL;
    }
    if (!same && (reinterpret_cast<uintptr_t>(c->k_scale) % 4 || reinterpret_cast<uintptr_t>(c->v_scale) % 4)) {
        set_error("%s: k_scale and v_scale must be 4-byte aligned", fn);
        return SP_EINVAL;
    }
    const int64_t align = same ? 16 : 8, step = same ? 16 / esize(c->dtype) : 8;
    if (reinterpret_cast<uintptr_t>(c->k) % align || reinterpret_cast<uintptr_t>(c->v) % align ||
        c->stride_page % step || c->stride_head % step || c->stride_slot % step) {
        set_error("%s: cache pointers must be %lld-byte aligned, with strides of a multiple of that", fn, (long long)align);
        return SP_EINVAL;
    }
    if (c->stride_page < 0 || c->stride_head < 0 || c->stride_slot < c->d) {
        set_error("%s: cache strides must not be negative, and stride_slot at least d", fn);
        return SP_EINVAL;
    }
    return SP_OK;
}

sp_status check_batch_args(const char* fn, const sp_batch* b) {
    if (!b) {
        set_error("%s: null batch", fn);
        return SP_EINVAL;
    }
    if (b->B < 1 || b->T < 0 || b->T > INT32_MAX || b->max_new < 0 || b->table_width < 1 || b->table_stride < 0) {
        set_error("%s: the batch needs B and table_width >= 1, 0 <= T <= 2^31-1, max_new >= 0 and table_stride >= 0 "
                  "(got %d, %d, %lld, %d, %lld)", fn, b->B, b->table_width, (long long)b->T, b->max_new,
                  (long long)b->table_stride);
        return SP_EINVAL;
    }
    if (b->B > 65535) {
        set_error("%s: at most 65535 sequences (got %d)", fn, b->B);
        return SP_EUNSUPPORTED;
    }
    if (!b->cu_new || !b->kv_len || !b->table) {
        set_error("%s: null cu_new, kv_len or table", fn);
        return SP_EINVAL;
    }
    if (reinterpret_cast<uintptr_t>(b->cu_new) % 8 || reinterpret_cast<uintptr_t>(b->kv_len) % 8 ||
        reinterpret_cast<uintptr_t>(b->table) % 4) {
        set_error("%s: misaligned cu_new, kv_len or table", fn);
        return SP_EINVAL;
    }
    return SP_OK;
}

}  // namespace sp

using namespace sp;

extern "C" {

sp_status sp_rotary_plan_init(sp_rotary_plan* plan, int rot, const double* inv_freq_host,
                              const uint8_t* axis_of_pair_host, int axes, int interleaved) {
    const char* fn = "sp_rotary_plan_init";
    if (!plan || !inv_freq_host) {
        set_error("%s: null plan or frequencies", fn);
        return SP_EINVAL;
    }
    if (rot < 16 || rot > 256 || rot % 16 != 0) {
        set_error("%s: rot must be a multiple of 16 in [16, 256] (got %d)", fn, rot);
        return rot < 2 ? SP_EINVAL : SP_EUNSUPPORTED;
    }
    if (axes < 1 || axes > 8) {
        set_error("%s: 1 to 8 axes (got %d)", fn, axes);
        return SP_EINVAL;
    }
    sp_rotary_plan p;
    memset(&p, 0, sizeof(p));
    p.rot = rot;
    p.interleaved = interleaved != 0;
    p.axes = axes;
    for (int i = 0; i < rot / 2; ++i) {
        const double f = inv_freq_host[i];
        if (!isfinite(f)) {
            set_error("%s: frequency %d is not finite", fn, i);
            return SP_EINVAL;
        }
        if (fabs(f) > 0x1p40) {
            set_error("%s: frequency %d is above 2^40 radians a position (%g)", fn, i, f);
            return SP_EUNSUPPORTED;
        }
        p.turns[i] = fraction_of_turn(f);
        p.axis[i] = axis_of_pair_host ? axis_of_pair_host[i] : 0;
        if (p.axis[i] >= axes) {
            set_error("%s: pair %d has axis %d of %d", fn, i, (int)p.axis[i], axes);
            return SP_EINVAL;
        }
    }
    *plan = p;
    clear_error();
    return SP_OK;
}

sp_status sp_rotary(const sp_rotary_plan* plan, const int32_t* positions, int64_t pos_stride, int64_t T, int d,
                    sp_dtype dtype, int inverse, const sp_rows* q, const sp_rows* q_out, int H, const sp_rows* k,
                    const sp_rows* k_out, int H_kv, void* stream) {
    const char* fn = "sp_rotary";
    sp_status s = check_dim(fn, d, dtype);
    if (s != SP_OK) return s;
    if (!plan || plan->rot < 16 || plan->rot > 256 || plan->rot % 16 || plan->axes < 1 || plan->axes > 8) {
        set_error("%s: null plan, or one that sp_rotary_plan_init has not filled", fn);
        return SP_EINVAL;
    }
    if (plan->rot > d) {
        set_error("%s: the plan rotates %d entries of a head of %d", fn, plan->rot, d);
        return SP_EINVAL;
    }
    if (T < 0 || H < 0 || H_kv < 0 || T > INT32_MAX) {
        set_error("%s: T, H and H_kv must be >= 0, T at most 2^31-1 (got %lld, %d, %d)", fn, (long long)T, H, H_kv);
        return SP_EINVAL;
    }
    if (H > 65535 || H_kv > 65535) {
        set_error("%s: at most 65535 heads (got %d, %d)", fn, H, H_kv);
        return SP_EUNSUPPORTED;
    }
    const sp_rows none{nullptr, 0, 0};
    if (T > 0 && H + H_kv > 0) {
        if (!positions || reinterpret_cast<uintptr_t>(positions) % 4) {
            set_error("%s: null or misaligned positions", fn);
            return SP_EINVAL;
        }
        if (H > 0 && ((s = check_rows(fn, "q", q, dtype, T)) != SP_OK || (s = check_rows(fn, "q_out", q_out, dtype, T)) != SP_OK ||
                      (s = check_apart(fn, "q_out", q_out, T, H, d)) != SP_OK))
            return s;
        if (H_kv > 0 &&
            ((s = check_rows(fn, "k", k, dtype, T)) != SP_OK || (s = check_rows(fn, "k_out", k_out, dtype, T)) != SP_OK ||
             (s = check_apart(fn, "k_out", k_out, T, H_kv, d)) != SP_OK))
            return s;
    }
    s = rotary_launch(*plan, positions, pos_stride, T, d, dtype, inverse != 0, H > 0 && q ? *q : none,
                      H > 0 && q_out ? *q_out : none, H, H_kv > 0 && k ? *k : none, H_kv > 0 && k_out ? *k_out : none,
                      H_kv, static_cast<cudaStream_t>(stream));
    if (s == SP_OK) clear_error();
    return s;
}

size_t sp_cache_workspace_size(void) { return sizeof(WsHeader); }

sp_status sp_cache_write(const sp_cache* cache, const sp_batch* batch, const sp_rows* k_new, const sp_rows* v_new,
                         void* ws, size_t ws_bytes, void* stream) {
    const char* fn = "sp_cache_write";
    sp_status s;
    if ((s = check_cache(fn, cache)) != SP_OK || (s = check_batch_args(fn, batch)) != SP_OK) return s;
    if ((s = check_no_overlap(fn, cache)) != SP_OK) return s;
    if ((s = check_rows(fn, "k_new", k_new, cache->dtype, batch->T)) != SP_OK ||
        (s = check_rows(fn, "v_new", v_new, cache->dtype, batch->T)) != SP_OK)
        return s;
    if ((s = check_workspace(fn, ws, ws_bytes, sizeof(WsHeader))) != SP_OK) return s;
    s = cache_write_launch(*cache, *batch, *k_new, *v_new, ws, static_cast<cudaStream_t>(stream));
    if (s == SP_OK) clear_error();
    return s;
}

sp_status sp_cache_read(const sp_cache* cache, const sp_batch* batch, const sp_rows* out_k, const sp_rows* out_v,
                        void* ws, size_t ws_bytes, void* stream) {
    const char* fn = "sp_cache_read";
    sp_status s;
    if ((s = check_cache(fn, cache)) != SP_OK || (s = check_batch_args(fn, batch)) != SP_OK) return s;
    if (!out_k && !out_v) {
        set_error("%s: neither keys nor values are asked for", fn);
        return SP_EINVAL;
    }
    if ((out_k && (s = check_rows(fn, "out_k", out_k, cache->dtype, batch->T)) != SP_OK) ||
        (out_v && (s = check_rows(fn, "out_v", out_v, cache->dtype, batch->T)) != SP_OK) ||
        (out_k && (s = check_apart(fn, "out_k", out_k, batch->T, cache->H_kv, cache->d)) != SP_OK) ||
        (out_v && (s = check_apart(fn, "out_v", out_v, batch->T, cache->H_kv, cache->d)) != SP_OK))
        return s;
    if ((s = check_workspace(fn, ws, ws_bytes, sizeof(WsHeader))) != SP_OK) return s;
    const sp_rows none{nullptr, 0, 0};
    s = cache_read_launch(*cache, *batch, out_k ? *out_k : none, out_v ? *out_v : none, ws,
                          static_cast<cudaStream_t>(stream));
    if (s == SP_OK) clear_error();
    return s;
}

size_t sp_attend_workspace_size(const sp_cache* cache, const sp_batch* batch, int H) {
    return attend_bytes("sp_attend_workspace_size", cache, batch, H);
}

size_t sp_attend_tree_workspace_size(const sp_cache* cache, const sp_batch* batch, int H) {
    return attend_bytes("sp_attend_tree_workspace_size", cache, batch, H);
}

sp_status sp_attend(const sp_rows* q, const sp_cache* cache, const sp_batch* batch, int H, double scale,
                    int64_t window, const sp_rows* out, float* lse, int64_t lse_stride_row,
                    int64_t lse_stride_head, void* ws, size_t ws_bytes, void* stream) {
    return attend("sp_attend", q, cache, batch, H, scale, window, nullptr, 0, out, lse, lse_stride_row, lse_stride_head, ws, ws_bytes,
                  stream);
}

sp_status sp_attend_tree(const sp_rows* q, const sp_cache* cache, const sp_batch* batch, int H, double scale,
                         int64_t window, const uint32_t* seen, int64_t seen_stride, int seen_words, const sp_rows* out, float* lse,
                         int64_t lse_stride_row, int64_t lse_stride_head, void* ws, size_t ws_bytes, void* stream) {
    const char* fn = "sp_attend_tree";
    sp_status s;
    if ((s = check_batch_args(fn, batch)) != SP_OK || (s = check_words(fn, batch, seen, seen_stride, seen_words)) != SP_OK) return s;
    static const uint32_t none = 0;         // of an empty batch: never read
    return attend(fn, q, cache, batch, H, scale, window, seen ? seen : &none, seen_stride, out, lse, lse_stride_row, lse_stride_head, ws,
                  ws_bytes, stream);
}

size_t sp_tree_workspace_size(void) { return sizeof(WsHeader); }

sp_status sp_tree_seen(const sp_batch* batch, const int32_t* parent, uint32_t* seen, int64_t seen_stride, int seen_words,
                       int32_t* positions, void* ws, size_t ws_bytes, void* stream) {
    const char* fn = "sp_tree_seen";
    sp_status s;
    if ((s = check_batch_args(fn, batch)) != SP_OK) return s;
    if (!seen && !positions) {
        set_error("%s: neither seen nor positions are asked for", fn);
        return SP_EINVAL;
    }
    if (seen && (s = check_words(fn, batch, seen, seen_stride, seen_words)) != SP_OK) return s;
    if (seen && batch->T > 1 && seen_stride < seen_words) {
        set_error("%s: the rows of seen overlap (stride %lld of %d words)", fn, (long long)seen_stride, seen_words);
        return SP_EINVAL;
    }
    if (batch->T > 0 && (s = check_ints(fn, "parent", parent)) != SP_OK) return s;
    if (reinterpret_cast<uintptr_t>(positions) % 4) {
        set_error("%s: misaligned positions", fn);
        return SP_EINVAL;
    }
    const Span parents = words_of(parent, batch->T, 1, 1);
    if ((s = check_apart(fn, "seen", words_of(seen, batch->T, seen_stride, seen_words), {parents, starts_of(batch), lengths_of(batch)})) != SP_OK ||
        (s = check_apart(fn, "positions", words_of(positions, batch->T, 1, 1), {parents, starts_of(batch), lengths_of(batch)})) != SP_OK)
        return s;
    if ((s = check_workspace(fn, ws, ws_bytes, sizeof(WsHeader))) != SP_OK) return s;
    s = tree_seen_launch(*batch, parent, seen, seen_stride, seen ? seen_words : 1, positions, ws, static_cast<cudaStream_t>(stream));
    if (s == SP_OK) clear_error();
    return s;
}

sp_status sp_tree_accept(const sp_batch* batch, const int32_t* parent, const int32_t* draft, const int32_t* target, int32_t* path,
                         int64_t path_stride, int64_t* n_path, int32_t* next, void* ws, size_t ws_bytes, void* stream) {
    const char* fn = "sp_tree_accept";
    sp_status s;
    if ((s = check_batch_args(fn, batch)) != SP_OK) return s;
    if (batch->T > 0 && ((s = check_ints(fn, "parent", parent)) != SP_OK || (s = check_ints(fn, "draft", draft)) != SP_OK ||
                         (s = check_ints(fn, "target", target)) != SP_OK))
        return s;
    if ((batch->max_new > 0 && (s = check_ints(fn, "path", path)) != SP_OK) || (s = check_counts(fn, "n_path", n_path)) != SP_OK) return s;
    if (batch->B > 1 && path_stride < batch->max_new) {
        set_error("%s: the sequences' paths overlap (stride %lld for %d tokens)", fn, (long long)path_stride, batch->max_new);
        return SP_EINVAL;
    }
    if (reinterpret_cast<uintptr_t>(next) % 4) {
        set_error("%s: misaligned next", fn);
        return SP_EINVAL;
    }
    const Span p = words_of(parent, batch->T, 1, 1), d = words_of(draft, batch->T, 1, 1), t = words_of(target, batch->T, 1, 1);
    const Span starts = starts_of(batch), lengths = lengths_of(batch);
    if ((s = check_apart(fn, "path", words_of(path, batch->B, path_stride, batch->max_new), {p, d, t, starts, lengths})) != SP_OK ||
        (s = check_apart(fn, "n_path", {n_path, 8 * (int64_t)batch->B}, {p, d, t, starts, lengths})) != SP_OK ||
        (s = check_apart(fn, "next", words_of(next, batch->B, 1, 1), {p, d, t, starts, lengths})) != SP_OK)
        return s;
    if ((s = check_workspace(fn, ws, ws_bytes, sizeof(WsHeader))) != SP_OK) return s;
    s = tree_accept_launch(*batch, parent, draft, target, path, path_stride, n_path, next, ws, static_cast<cudaStream_t>(stream));
    if (s == SP_OK) clear_error();
    return s;
}

size_t sp_attend_weights_workspace_size(const sp_cache* cache, const sp_batch* batch, int H) {
    const char* fn = "sp_attend_weights_workspace_size";
    if (check_cache(fn, cache) != SP_OK || check_batch_args(fn, batch) != SP_OK || check_heads(fn, cache, H) != SP_OK) return 0;
    return weights_path(*cache, *batch, H) == kChunks ? weights_tc_ws_bytes() : sizeof(WsHeader);
}

sp_status sp_attend_weights(const sp_rows* q, const sp_cache* cache, const sp_batch* batch, int H, double scale, int64_t window,
                            const float* lse, int64_t lse_stride_row, int64_t lse_stride_head, double decay, float* weights,
                            void* ws, size_t ws_bytes, void* stream) {
    const char* fn = "sp_attend_weights";
    sp_status s;
    AttendProblem a;
    if ((s = attend_problem(fn, q, cache, batch, H, scale, window, &a)) != SP_OK) return s;
    if (batch->T > 0 && !lse) {
        set_error("%s: null lse", fn);
        return SP_EINVAL;
    }
    if ((s = check_weights(fn, weights)) != SP_OK) return s;
    if (reinterpret_cast<uintptr_t>(lse) % 4) {
        set_error("%s: lse must be 4-byte aligned", fn);
        return SP_EINVAL;
    }
    if (!(decay >= 0 && decay <= 1)) {
        set_error("%s: decay must be in [0, 1] (got %g)", fn, decay);
        return SP_EINVAL;
    }
    if ((s = check_workspace(fn, ws, ws_bytes, sp_attend_weights_workspace_size(cache, batch, H))) != SP_OK) return s;
    a.lse = const_cast<float*>(lse);        // read only
    a.lse_stride_row = lse_stride_row;
    a.lse_stride_head = lse_stride_head;
    const WeightsProblem w{a, (float)decay, weights};
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (weights_path(*cache, *batch, H)) {
        case kStep: s = weights_step_launch(w, ws, st); break;
        case kChunks: s = weights_tc_launch(w, ws, st); break;
        default: s = weights_general_launch(w, ws, st); break;
    }
    if (s == SP_OK) clear_error();
    return s;
}

sp_status sp_cache_choose(const sp_cache* cache, const sp_batch* batch, const float* weights, int shared, int64_t budget,
                          int64_t first, int64_t last, int32_t* kept, int64_t kept_stride_seq, int64_t kept_stride_head,
                          int64_t* n_kept, void* ws, size_t ws_bytes, void* stream) {
    const char* fn = "sp_cache_choose";
    sp_status s;
    if ((s = check_cache(fn, cache)) != SP_OK || (s = check_batch_args(fn, batch)) != SP_OK || (s = check_weights(fn, weights)) != SP_OK)
        return s;
    if (budget < 0 || budget > (int64_t)1 << 30 || first < 0 || last < 0 || first > budget || last > budget - first) {
        set_error("%s: 0 <= first + last <= budget <= 2^30 (got %lld, %lld, %lld)", fn, (long long)first, (long long)last,
                  (long long)budget);
        return SP_EINVAL;
    }
    const int heads = shared ? 1 : cache->H_kv;
    if ((s = check_items(fn, (int64_t)batch->B * heads)) != SP_OK) return s;
    if ((budget > 0 && (s = check_ints(fn, "kept", kept)) != SP_OK) || (s = check_counts(fn, "n_kept", n_kept)) != SP_OK) return s;
    Axis axis[2] = {{batch->B, kept_stride_seq}, {heads, kept_stride_head}};
    if (budget > 0 && !apart(axis, (int)budget)) {
        set_error("%s: the lists of kept overlap", fn);
        return SP_EINVAL;
    }
    if ((s = check_apart(fn, "n_kept", {n_kept, 8 * (int64_t)batch->B}, {starts_of(batch), lengths_of(batch)})) != SP_OK) return s;
    if ((s = check_workspace(fn, ws, ws_bytes, sizeof(WsHeader))) != SP_OK) return s;
    s = cache_choose_launch(*cache, *batch, weights, shared != 0, budget, first, last, kept, kept_stride_seq, kept_stride_head, n_kept,
                            ws, static_cast<cudaStream_t>(stream));
    if (s == SP_OK) clear_error();
    return s;
}

sp_status sp_cache_keep(const sp_cache* cache, const sp_batch* batch, const int32_t* kept, int heads, int64_t kept_stride_seq,
                        int64_t kept_stride_head, const int64_t* n_kept, int64_t most, int drafted, const int32_t* to, int to_width,
                        int64_t to_stride, float* weights, int64_t* kv_out, void* ws, size_t ws_bytes, void* stream) {
    const char* fn = "sp_cache_keep";
    sp_status s;
    if ((s = check_cache(fn, cache)) != SP_OK || (s = check_batch_args(fn, batch)) != SP_OK || (s = check_no_overlap(fn, cache)) != SP_OK)
        return s;
    if (heads != 1 && heads != cache->H_kv) {
        set_error("%s: a list for every KV head (%d) or 1 that they share (got %d)", fn, cache->H_kv, heads);
        return SP_EINVAL;
    }
    if ((s = check_items(fn, 2 * (int64_t)batch->B * cache->H_kv)) != SP_OK) return s;
    if (most < 0 || most > (int64_t)1 << 30) {
        set_error("%s: lists of 0 to 2^30 entries (got %lld)", fn, (long long)most);
        return SP_EINVAL;
    }
    if ((most > 0 && (s = check_ints(fn, "kept", kept)) != SP_OK) || (s = check_counts(fn, "n_kept", n_kept)) != SP_OK ||
        (s = check_counts(fn, "kv_out", kv_out)) != SP_OK)
        return s;
    if ((s = check_apart(fn, "kv_out", {kv_out, 8 * (int64_t)batch->B}, {starts_of(batch), lengths_of(batch), {n_kept, 8 * (int64_t)batch->B}})) != SP_OK)
        return s;
    if (reinterpret_cast<uintptr_t>(to) % 4 || (to && (to_width < 1 || to_stride < 0))) {
        set_error("%s: to must be 4-byte aligned, with to_width >= 1 and to_stride >= 0", fn);
        return SP_EINVAL;
    }
    if (to == batch->table) to = nullptr;       // the same places
    if (weights && (s = check_weights(fn, weights)) != SP_OK) return s;
    if ((s = check_workspace(fn, ws, ws_bytes, sizeof(WsHeader))) != SP_OK) return s;
    s = cache_keep_launch(*cache, *batch, kept, heads, kept_stride_seq, kept_stride_head, n_kept, most, drafted != 0, to, to_width,
                          to_stride, weights, kv_out, ws, static_cast<cudaStream_t>(stream));
    if (s == SP_OK) clear_error();
    return s;
}

}  // extern "C"
