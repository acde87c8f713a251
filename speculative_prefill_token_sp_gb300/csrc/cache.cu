// The paged key/value cache: writing new tokens (quantised on the way) and
// reading tokens back.
//
// Both directions move each row once and compute next to nothing, so they are
// bound by memory, or by the launch for a decode step's few rows.  A group of
// 2^g lanes (the smallest power of two that covers d / 8) holds one row, eight
// entries a lane; the row's largest magnitude is a shuffle maximum over the
// group, so a row is read once and quantised in registers.  The last block
// checks what the batch's arrays say and is the only writer of the status.
#include "paged.cuh"

namespace sp {
namespace {

constexpr int kCacheThreads = 256;

struct MoveArgs {
    sp_cache c;
    sp_batch b;
    sp_rows k, v;           // data may be null (read)
    int lg;                 // log2 of the lanes of a row
    WsHeader* hdr;
};

template <typename T, int kKind>
__device__ __forceinline__ void write_row(const MoveArgs& p, const float (&x)[8], void* data, float* scales, int64_t at,
                                          int64_t scale_at, int lane, bool act, bool there) {
    if constexpr (kKind == SP_CACHE_SAME) {
        if (act && there) store8(static_cast<T*>(data) + at + lane * 8, x);
    } else {
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max_nan(top, fabsf(x[i]));
        for (int o = 1; o < (1 << p.lg); o <<= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float scale = row_scale<kKind>(top);
        if (!act || !there) return;
        const bool fine = scale == scale;
        const uint2 u = fine ? encode8<kKind>(x, __int_as_float(0x7f000000 - __float_as_int(scale))) : make_uint2(0, 0);
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(data) + at + lane * 8) = u;
        if (lane == 0) scales[scale_at] = scale;
    }
}

template <typename T, int kKind>
__global__ void __launch_bounds__(kCacheThreads) write_kernel(const __grid_constant__ MoveArgs p) {
    if (blockIdx.x == gridDim.x - 1) {
        check_batch(p.b, p.c, p.hdr);
        return;
    }
    const int64_t i = ((int64_t)blockIdx.x * kCacheThreads + threadIdx.x) >> p.lg;
    const int lane = threadIdx.x & ((1 << p.lg) - 1);
    const bool act = i < p.b.T * p.c.H_kv && lane * 8 < p.c.d;
    const int64_t r = act ? i / p.c.H_kv : 0;
    const int h = act ? (int)(i - r * p.c.H_kv) : 0;
    float x[8] = {}, y[8] = {};
    if (act) {
        load8(static_cast<const T*>(p.k.data) + r * p.k.stride_row + h * p.k.stride_head + lane * 8, x);
        load8(static_cast<const T*>(p.v.data) + r * p.v.stride_row + h * p.v.stride_head + lane * 8, y);
    }
    const Place pl = act ? place_of_row(p.b, p.c, r) : Place{-1, 0, false};
    const bool there = pl.page >= 0;
    const int64_t at = row_offset(p.c, pl.page, h, pl.slot), sat = scale_offset(p.c, pl.page, h, pl.slot);
    write_row<T, kKind>(p, x, p.c.k, p.c.k_scale, at, sat, lane, act, there);
    write_row<T, kKind>(p, y, p.c.v, p.c.v_scale, at, sat, lane, act, there);
}

template <typename T, int kKind>
__device__ __forceinline__ void read_row(const void* data, const float* scales, int64_t at, int64_t scale_at, int lane,
                                         bool there, T* dst) {
    float x[8] = {};
    if (there) {
        if constexpr (kKind == SP_CACHE_SAME) {
            load8(static_cast<const T*>(data) + at + lane * 8, x);
        } else {
            decode8<kKind>(*reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(data) + at + lane * 8), x);
            const float s = scales[scale_at];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] *= s;
        }
    }
    store8(dst + lane * 8, x);
}

template <typename T, int kKind>
__global__ void __launch_bounds__(kCacheThreads) read_kernel(const __grid_constant__ MoveArgs p) {
    if (blockIdx.x == gridDim.x - 1) {
        if (blockIdx.y == 0) check_batch(p.b, p.c, p.hdr);
        return;
    }
    const int64_t r = ((int64_t)blockIdx.x * kCacheThreads + threadIdx.x) >> p.lg;
    const int lane = threadIdx.x & ((1 << p.lg) - 1), h = blockIdx.y;
    if (r >= p.b.T || lane * 8 >= p.c.d) return;
    const Place pl = place_of_row(p.b, p.c, r);
    if (!pl.token) return;
    const bool there = pl.page >= 0;
    const int64_t at = row_offset(p.c, pl.page, h, pl.slot), sat = scale_offset(p.c, pl.page, h, pl.slot);
    if (p.k.data)
        read_row<T, kKind>(p.c.k, p.c.k_scale, at, sat, lane, there,
                           static_cast<T*>(p.k.data) + r * p.k.stride_row + h * p.k.stride_head);
    if (p.v.data)
        read_row<T, kKind>(p.c.v, p.c.v_scale, at, sat, lane, there,
                           static_cast<T*>(p.v.data) + r * p.v.stride_row + h * p.v.stride_head);
}

template <typename T>
void launch_kind(bool write, const MoveArgs& a, dim3 grid, cudaStream_t st) {
    switch (a.c.kind) {
        case SP_CACHE_SAME:
            if (write) write_kernel<T, SP_CACHE_SAME><<<grid, kCacheThreads, 0, st>>>(a);
            else read_kernel<T, SP_CACHE_SAME><<<grid, kCacheThreads, 0, st>>>(a);
            break;
        case SP_CACHE_E4M3:
            if (write) write_kernel<T, SP_CACHE_E4M3><<<grid, kCacheThreads, 0, st>>>(a);
            else read_kernel<T, SP_CACHE_E4M3><<<grid, kCacheThreads, 0, st>>>(a);
            break;
        case SP_CACHE_INT8:
            if (write) write_kernel<T, SP_CACHE_INT8><<<grid, kCacheThreads, 0, st>>>(a);
            else read_kernel<T, SP_CACHE_INT8><<<grid, kCacheThreads, 0, st>>>(a);
            break;
    }
}

sp_status move_launch(bool write, const sp_cache& c, const sp_batch& b, const sp_rows& k, const sp_rows& v, void* ws,
                      cudaStream_t st) {
    MoveArgs a{c, b, k, v, 0, static_cast<WsHeader*>(ws)};
    while ((8 << a.lg) < c.d) ++a.lg;
    const int64_t rows = write ? b.T * c.H_kv : b.T;
    const int64_t blocks = ((rows << a.lg) + kCacheThreads - 1) / kCacheThreads + 1;
    if (blocks > INT32_MAX) {
        set_error("%s: %lld rows are too many for one call", write ? "sp_cache_write" : "sp_cache_read", (long long)rows);
        return SP_EUNSUPPORTED;
    }
    const dim3 grid((unsigned)blocks, write ? 1u : (unsigned)c.H_kv);
    if (c.dtype == SP_BF16) launch_kind<__nv_bfloat16>(write, a, grid, st);
    else launch_kind<float>(write, a, grid, st);
    SP_LAUNCH_CHECK();
    return SP_OK;
}

}  // namespace

sp_status cache_write_launch(const sp_cache& c, const sp_batch& b, const sp_rows& k, const sp_rows& v, void* ws,
                             cudaStream_t st) {
    return move_launch(true, c, b, k, v, ws, st);
}

sp_status cache_read_launch(const sp_cache& c, const sp_batch& b, const sp_rows& k, const sp_rows& v, void* ws,
                            cudaStream_t st) {
    return move_launch(false, c, b, k, v, ws, st);
}

}  // namespace sp
