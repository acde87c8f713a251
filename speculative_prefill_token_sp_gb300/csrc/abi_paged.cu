// extern "C" entry points of the rotary positions, the paged cache and the
// attention over it (declared in include/specprefill.h).  Arguments are checked
// here, before anything is enqueued.
#include "paged.cuh"

#include <float.h>
#include <string.h>

#include <algorithm>
#include <atomic>

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
    Axis axis[3] = {{cache->pages, cache->stride_page}, {cache->H_kv, cache->stride_head}, {cache->page, cache->stride_slot}};
    if (!apart(axis, cache->d)) {
        set_error("%s: pages, heads or slots of the cache overlap", fn);
        return SP_EINVAL;
    }
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
    const char* fn = "sp_attend_workspace_size";
    if (check_cache(fn, cache) != SP_OK || check_batch_args(fn, batch) != SP_OK) return 0;
    if (H < 1 || H % cache->H_kv) {
        set_error("%s: H (%d) must be a multiple of H_kv (%d)", fn, H, cache->H_kv);
        return 0;
    }
    return path_bytes(path_of(*cache, *batch, H), *cache);
}

sp_status sp_attend(const sp_rows* q, const sp_cache* cache, const sp_batch* batch, int H, double scale,
                    int64_t window, const sp_rows* out, float* lse, int64_t lse_stride_row,
                    int64_t lse_stride_head, void* ws, size_t ws_bytes, void* stream) {
    const char* fn = "sp_attend";
    sp_status s;
    if ((s = check_cache(fn, cache)) != SP_OK || (s = check_batch_args(fn, batch)) != SP_OK) return s;
    if (H < 1 || H % cache->H_kv) {
        set_error("%s: H (%d) must be a multiple of H_kv (%d)", fn, H, cache->H_kv);
        return SP_EINVAL;
    }
    const float factor = (float)scale * 1.4426950408889634f;        // the kernels': logits to base 2
    if (!(factor >= FLT_MIN) || !isfinite(factor)) {
        set_error("%s: scale must be positive, and a normal fp32 number times log2(e) (got %g)", fn, scale);
        return SP_EINVAL;
    }
    if (window < 0) {
        set_error("%s: window must be >= 0 (got %lld)", fn, (long long)window);
        return SP_EINVAL;
    }
    if ((s = check_rows(fn, "q", q, cache->dtype, batch->T)) != SP_OK || (s = check_rows(fn, "out", out, cache->dtype, batch->T)) != SP_OK)
        return s;
    if (reinterpret_cast<uintptr_t>(lse) % 4) {
        set_error("%s: lse must be 4-byte aligned", fn);
        return SP_EINVAL;
    }
    if ((s = check_apart(fn, "q", q, batch->T, H, cache->d)) != SP_OK || (s = check_apart(fn, "out", out, batch->T, H, cache->d)) != SP_OK)
        return s;
    const size_t need = sp_attend_workspace_size(cache, batch, H);
    if ((s = check_workspace(fn, ws, ws_bytes, need)) != SP_OK) return s;
    AttendProblem p;
    p.q = *q; p.out = *out; p.cache = *cache; p.batch = *batch; p.H = H; p.scale = (float)scale;
    p.window = window >= (int64_t)1 << 30 ? 0 : (int)window;       // kv_len is at most 2^30: no limit at all
    p.page_shift = -1;
    for (int i = 0; i < 31; ++i)
        if (cache->page == 1 << i) p.page_shift = i;
    p.lse = lse; p.lse_stride_row = lse_stride_row; p.lse_stride_head = lse_stride_head;
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

}  // extern "C"
