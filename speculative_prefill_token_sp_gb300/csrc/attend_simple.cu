// Attention of new tokens over the paged cache: the general path (every type,
// head dimension and page size).
//
// One pass over a row's keys with the running maximum m and sum z of its
// softmax (base 2): x = log2(e) * scale * q.k; when x exceeds m, the sums are
// scaled by 2^(m - x).  One warp per (row, query head); a lane holds the
// entries e = 8 * lane .. 8 * lane + 7 of the query, the key and the sums.
#include "paged.cuh"

namespace sp {
namespace {

template <typename T, int kKind>
__device__ __forceinline__ bool fetch8(const sp_cache& c, const void* data, const float* scales, int page, int head,
                                       int slot, int lane, float (&x)[8]) {
    const int64_t at = row_offset(c, page, head, slot) + lane * 8;
    if constexpr (kKind == SP_CACHE_SAME) {
        load8(static_cast<const T*>(data) + at, x);
    } else {
        decode8<kKind>(*reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(data) + at), x);
        const float s = scales[scale_offset(c, page, head, slot)];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= s;
    }
    return true;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

template <typename T, int kKind>
__global__ void __launch_bounds__(128) attend_simple_kernel(const __grid_constant__ AttendProblem p, WsHeader* hdr) {
    if (blockIdx.x == gridDim.x - 1) {
        check_batch(p.batch, p.cache, p.window, hdr);
        return;
    }
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int64_t r = w / p.H;
    if (r >= p.batch.T) return;
    const int h = (int)(w - r * p.H), g = h / (p.H / p.cache.H_kv), page = p.cache.page;
    const int b = seq_of_row(p.batch, r);
    if (b < 0) return;
    const Seq s = load_seq(p.batch, page, b);
    if (r - s.row0 >= s.n) return;
    const int at = s.kv - s.n + (int)(r - s.row0);
    const int first = p.window ? max(0, at - p.window + 1) : 0;
    const bool act = lane * 8 < p.cache.d;
    float q[8] = {}, o[8] = {};
    if (act) load8(static_cast<const T*>(p.q.data) + r * p.q.stride_row + h * p.q.stride_head + lane * 8, q);
    float m = -INFINITY, z = 0.f;
    const float f = p.scale * 1.4426950408889634f;
    for (int i = first; i <= at; ++i) {
        const int pi = i / page, pg = p.batch.table[(int64_t)b * p.batch.table_stride + pi];
        if (pg < 0 || pg >= p.cache.pages) continue;
        float k[8] = {}, v[8] = {};
        if (act) {
            fetch8<T, kKind>(p.cache, p.cache.k, p.cache.k_scale, pg, g, i - pi * page, lane, k);
            fetch8<T, kKind>(p.cache, p.cache.v, p.cache.v_scale, pg, g, i - pi * page, lane, v);
        }
        float dot = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) dot += q[e] * k[e];
        const float x = warp_sum(dot) * f;
        const float mn = fmaxf(m, x), ref = mn == -INFINITY ? 0.f : mn;
        const float a = exp2f(m - ref), w2 = exp2f(x - ref);
        z = z * a + w2;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = o[e] * a + w2 * v[e];
        m = mn;
    }
    const float inv = z == 0.f ? 0.f : 1.f / z;
    if (act) {
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = z == 0.f ? 0.f : o[e] * inv;
        store8(static_cast<T*>(p.out.data) + r * p.out.stride_row + h * p.out.stride_head + lane * 8, o);
    }
    if (p.lse && lane == 0)
        p.lse[r * p.lse_stride_row + h * p.lse_stride_head] =
            z == 0.f ? -INFINITY : (m + log2f(z)) * 0.6931471805599453f;
}

}  // namespace

sp_status attend_simple_launch(const AttendProblem& p, void* ws, cudaStream_t st) {
    const int64_t blocks = (p.batch.T * p.H + 3) / 4 + 1;
    if (blocks > INT32_MAX) {
        set_error("sp_attend: %lld rows of %d heads are too many for one call", (long long)p.batch.T, p.H);
        return SP_EUNSUPPORTED;
    }
    WsHeader* hdr = static_cast<WsHeader*>(ws);
    const unsigned grid = (unsigned)blocks;
    const bool bf = p.cache.dtype == SP_BF16;
    switch (p.cache.kind) {
        case SP_CACHE_SAME:
            if (bf) attend_simple_kernel<__nv_bfloat16, SP_CACHE_SAME><<<grid, 128, 0, st>>>(p, hdr);
            else attend_simple_kernel<float, SP_CACHE_SAME><<<grid, 128, 0, st>>>(p, hdr);
            break;
        case SP_CACHE_E4M3:
            if (bf) attend_simple_kernel<__nv_bfloat16, SP_CACHE_E4M3><<<grid, 128, 0, st>>>(p, hdr);
            else attend_simple_kernel<float, SP_CACHE_E4M3><<<grid, 128, 0, st>>>(p, hdr);
            break;
        case SP_CACHE_INT8:
            if (bf) attend_simple_kernel<__nv_bfloat16, SP_CACHE_INT8><<<grid, 128, 0, st>>>(p, hdr);
            else attend_simple_kernel<float, SP_CACHE_INT8><<<grid, 128, 0, st>>>(p, hdr);
            break;
    }
    SP_LAUNCH_CHECK();
    return SP_OK;
}

}  // namespace sp
