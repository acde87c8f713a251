// The paged key/value cache: writing new tokens (quantised on the way) and
// reading tokens back.
//
// Both directions move each row once and compute next to nothing, so they are
// bound by memory, or by the launch for a decode step's few rows.  A block takes
// some tokens (of one head to read, so that its rows lie side by side on both
// sides; of all heads to write, as the new rows come token by token) and works
// out their places once, into shared memory.  A row is then held by a group of
// 2^g lanes, kE entries a lane (16 codes of an 8-bit cache, 8 entries otherwise),
// and a thread has several rows' loads, keys and values, under way at once.  A
// row's largest magnitude is a shuffle maximum over its group, so it is read
// once and quantised in registers.  The last block checks what the batch's
// arrays say and is the only writer of the status.
// Reading 131072 tokens of 8 heads of 128 from e4m3 to bf16 takes 132 us (6.2 TB/s),
// 16 prompts of 2K to 32K of a bf16 cache with 4 heads of 64 80 us (6.6 TB/s);
// writing 16 tokens and reading them back 6.1 us.
#include "paged.cuh"

#include <algorithm>

namespace sp {
namespace {

constexpr int kCacheThreads = 256;
// Rows whose loads a thread has under way.  Reading one layer of 131072 tokens (e4m3, 8 heads of 128) took 178, 137, 147 us with
// 1, 2, 4 of them; writing and reading back 8192 tokens took 35 us with 2 in the writing, 31 us with 1.
constexpr int kAheadRead = 2, kAheadWrite = 1;
constexpr int kMaxTokens = 256;     // tokens of a block

struct MoveArgs {
    sp_cache c;
    sp_batch b;
    sp_rows k, v;           // data may be null (read)
    int lg;                 // log2 of the lanes of a row
    int tokens;             // of a block
    WsHeader* hdr;
};

// kE entries as fp32.
template <typename T, int kE>
__device__ __forceinline__ void load_entries(const T* p, float (&x)[kE]) {
#pragma unroll
    for (int i = 0; i < kE; i += 8) load8(p + i, *reinterpret_cast<float(*)[8]>(x + i));
}
template <typename T, int kE>
__device__ __forceinline__ void store_entries(T* p, const float (&x)[kE]) {
#pragma unroll
    for (int i = 0; i < kE; i += 8) store8(p + i, *reinterpret_cast<const float(*)[8]>(x + i));
}

// One side (keys or values) of a row on its way into the cache.
template <typename T, int kKind, int kE>
__device__ __forceinline__ void write_row(const MoveArgs& p, const float (&x)[kE], void* data, float* scales, int64_t at,
                                          int64_t scale_at, int lane, bool there) {
    if constexpr (kKind == SP_CACHE_SAME) {
        if (there) store_entries(static_cast<T*>(data) + at + lane * kE, x);
    } else {
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < kE; ++i) top = max_nan(top, fabsf(x[i]));
        for (int o = 1; o < (1 << p.lg); o <<= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (!there) return;
        const float scale = row_scale<kKind>(top);
        // 1 / scale, exact as the scale is a power of two; the codes of a row with a NaN or an infinity are 0
        const bool fine = scale == scale;
        const float inv = __int_as_float(0x7f000000 - __float_as_int(scale));
        uint2 u[kE / 8];
#pragma unroll
        for (int i = 0; i < kE; i += 8)
            u[i / 8] = fine ? encode8<kKind>(*reinterpret_cast<const float(*)[8]>(x + i), inv) : make_uint2(0, 0);
        uint8_t* dst = static_cast<uint8_t*>(data) + at + lane * kE;
        if constexpr (kE == 16) *reinterpret_cast<uint4*>(dst) = make_uint4(u[0].x, u[0].y, u[1].x, u[1].y);
        else *reinterpret_cast<uint2*>(dst) = u[0];
        if (lane == 0) scales[scale_at] = scale;
    }
}

template <typename T, int kKind, int kE>
__global__ void __launch_bounds__(kCacheThreads) write_kernel(const __grid_constant__ MoveArgs p) {
    if (blockIdx.x == gridDim.x - 1) {
        check_batch(p.b, p.c, p.hdr);
        return;
    }
    __shared__ int2 places[kMaxTokens];
    const int64_t t0 = (int64_t)blockIdx.x * p.tokens;
    const int n = (int)min((int64_t)p.tokens, p.b.T - t0);
    const int lane = threadIdx.x & ((1 << p.lg) - 1), rows = n * p.c.H_kv, step = kCacheThreads >> p.lg;
    const bool act = lane * kE < p.c.d;
    bool placed = false;
    // all lanes of a warp go round together: the rows' maxima are shuffles
    for (int r0 = threadIdx.x >> p.lg; r0 - (int)(threadIdx.x >> p.lg) < rows; r0 += kAheadWrite * step) {
        float x[kAheadWrite][kE], y[kAheadWrite][kE];
        int t[kAheadWrite], h[kAheadWrite];
#pragma unroll
        for (int i = 0; i < kAheadWrite; ++i) {
            const int r = r0 + i * step;
            t[i] = r < rows ? r / p.c.H_kv : -1;
            h[i] = r - t[i] * p.c.H_kv;
#pragma unroll
            for (int e = 0; e < kE; ++e) x[i][e] = y[i][e] = 0.f;
            if (t[i] >= 0 && act) {
                load_entries(static_cast<const T*>(p.k.data) + (t0 + t[i]) * p.k.stride_row + h[i] * p.k.stride_head + lane * kE, x[i]);
                load_entries(static_cast<const T*>(p.v.data) + (t0 + t[i]) * p.v.stride_row + h[i] * p.v.stride_head + lane * kE, y[i]);
            }
        }
        if (!placed) {          // the first rows are on their way meanwhile
            for (int i = threadIdx.x; i < n; i += kCacheThreads) {
                const Place pl = place_of_row(p.b, p.c, t0 + i);
                places[i] = make_int2(pl.page, pl.slot);
            }
            __syncthreads();
            placed = true;
        }
#pragma unroll
        for (int i = 0; i < kAheadWrite; ++i) {
            const int2 pl = t[i] >= 0 ? places[t[i]] : make_int2(-1, 0);
            const bool there = pl.x >= 0 && act;
            const int64_t at = row_offset(p.c, pl.x, h[i], pl.y), sat = scale_offset(p.c, pl.x, h[i], pl.y);
            write_row<T, kKind, kE>(p, x[i], p.c.k, p.c.k_scale, at, sat, lane, there);
            write_row<T, kKind, kE>(p, y[i], p.c.v, p.c.v_scale, at, sat, lane, there);
        }
    }
}

// One side of a row in the cache, as it is loaded, and its entries.
template <typename T, int kKind, int kE>
struct Held {
    static constexpr int kWords = kKind == SP_CACHE_SAME ? kE * (int)sizeof(T) / 4 : kE / 4;
    uint32_t w[kWords];
    float scale;
    __device__ __forceinline__ void load(const void* data, const float* scales, int64_t at, int64_t scale_at, int lane) {
        const char* src = static_cast<const char*>(data) + (at + lane * kE) * (kKind == SP_CACHE_SAME ? (int)sizeof(T) : 1);
        if constexpr (kWords == 2) {
            const uint2 u = *reinterpret_cast<const uint2*>(src);
            w[0] = u.x; w[1] = u.y;
        } else {
#pragma unroll
            for (int i = 0; i < kWords; i += 4) {
                const uint4 u = reinterpret_cast<const uint4*>(src)[i / 4];
                w[i] = u.x; w[i + 1] = u.y; w[i + 2] = u.z; w[i + 3] = u.w;
            }
        }
        if constexpr (kKind != SP_CACHE_SAME) scale = scales[scale_at];
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
        scale = 1.f;
    }
    __device__ __forceinline__ void store(T* dst) const {
        if constexpr (kKind == SP_CACHE_SAME) {
#pragma unroll
            for (int i = 0; i < kWords; i += 4) reinterpret_cast<uint4*>(dst)[i / 4] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
        } else {
            float x[kE];
#pragma unroll
            for (int i = 0; i < kE; i += 8) {
                float(&v)[8] = *reinterpret_cast<float(*)[8]>(x + i);
                decode8<kKind>(make_uint2(w[i / 4], w[i / 4 + 1]), v);
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] *= scale;
            }
            store_entries(dst, x);
        }
    }
};

template <typename T, int kKind, int kE>
__global__ void __launch_bounds__(kCacheThreads) read_kernel(const __grid_constant__ MoveArgs p) {
    if (blockIdx.x == gridDim.x - 1) {
        if (blockIdx.y == 0) check_batch(p.b, p.c, p.hdr);
        return;
    }
    __shared__ int2 places[kMaxTokens];         // page (-1: zeros, -2: no token) and slot
    const int64_t t0 = (int64_t)blockIdx.x * p.tokens;
    const int n = (int)min((int64_t)p.tokens, p.b.T - t0);
    for (int t = threadIdx.x; t < n; t += kCacheThreads) {
        const Place pl = place_of_row(p.b, p.c, t0 + t);
        places[t] = make_int2(pl.token ? pl.page : -2, pl.slot);
    }
    __syncthreads();
    const int lane = threadIdx.x & ((1 << p.lg) - 1), h = blockIdx.y, step = kCacheThreads >> p.lg;
    if (lane * kE >= p.c.d) return;
    T* out_k = static_cast<T*>(p.k.data);
    T* out_v = static_cast<T*>(p.v.data);
    for (int r0 = threadIdx.x >> p.lg; r0 < n; r0 += kAheadRead * step) {
        Held<T, kKind, kE> x[kAheadRead], y[kAheadRead];
        int2 pl[kAheadRead];
#pragma unroll
        for (int i = 0; i < kAheadRead; ++i) {
            pl[i] = r0 + i * step < n ? places[r0 + i * step] : make_int2(-2, 0);
            x[i].zero();
            y[i].zero();
            if (pl[i].x < 0) continue;
            const int64_t at = row_offset(p.c, pl[i].x, h, pl[i].y), sat = scale_offset(p.c, pl[i].x, h, pl[i].y);
            if (out_k) x[i].load(p.c.k, p.c.k_scale, at, sat, lane);
            if (out_v) y[i].load(p.c.v, p.c.v_scale, at, sat, lane);
        }
#pragma unroll
        for (int i = 0; i < kAheadRead; ++i) {
            if (pl[i].x == -2) continue;
            const int64_t r = t0 + r0 + i * step;
            if (out_k) x[i].store(out_k + r * p.k.stride_row + h * p.k.stride_head + lane * kE);
            if (out_v) y[i].store(out_v + r * p.v.stride_row + h * p.v.stride_head + lane * kE);
        }
    }
}

template <typename T, int kKind, int kE>
void launch_one(bool write, MoveArgs a, cudaStream_t st) {
    while ((kE << a.lg) < a.c.d) ++a.lg;
    // about as many rows a thread as it has under way, and few enough tokens for every SM to have a block
    const int per_token = (write ? a.c.H_kv : 1) << a.lg;
    const int64_t all = write ? a.b.T : a.b.T * a.c.H_kv;
    const int64_t want = std::min<int64_t>((int64_t)(write ? kAheadWrite : kAheadRead) * kCacheThreads / per_token, (all + 2 * sm_count() - 1) / (2 * sm_count()));
    a.tokens = (int)std::max<int64_t>(1, std::min<int64_t>(want, kMaxTokens));
    const dim3 grid((unsigned)((a.b.T + a.tokens - 1) / a.tokens + 1), write ? 1u : (unsigned)a.c.H_kv);
    if (write) write_kernel<T, kKind, kE><<<grid, kCacheThreads, 0, st>>>(a);
    else read_kernel<T, kKind, kE><<<grid, kCacheThreads, 0, st>>>(a);
}

template <typename T>
void launch_kind(bool write, const MoveArgs& a, cudaStream_t st) {
    const bool wide = a.c.d % 16 == 0 &&
                      (reinterpret_cast<uintptr_t>(a.c.k) | reinterpret_cast<uintptr_t>(a.c.v) | (uintptr_t)a.c.stride_page |
                       (uintptr_t)a.c.stride_head | (uintptr_t)a.c.stride_slot) % 16 == 0;
    switch (a.c.kind) {
        case SP_CACHE_SAME: launch_one<T, SP_CACHE_SAME, 8>(write, a, st); break;
        case SP_CACHE_E4M3:
            if (wide) launch_one<T, SP_CACHE_E4M3, 16>(write, a, st);
            else launch_one<T, SP_CACHE_E4M3, 8>(write, a, st);
            break;
        case SP_CACHE_INT8:
            if (wide) launch_one<T, SP_CACHE_INT8, 16>(write, a, st);
            else launch_one<T, SP_CACHE_INT8, 8>(write, a, st);
            break;
    }
}

sp_status move_launch(bool write, const sp_cache& c, const sp_batch& b, const sp_rows& k, const sp_rows& v, void* ws,
                      cudaStream_t st) {
    const MoveArgs a{c, b, k, v, 0, 0, static_cast<WsHeader*>(ws)};
    if (c.dtype == SP_BF16) launch_kind<__nv_bfloat16>(write, a, st);
    else launch_kind<float>(write, a, st);
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
