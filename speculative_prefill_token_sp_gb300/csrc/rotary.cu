// Rotary positions of queries and keys, with one or several position axes.
//
// Pair i at position p turns by p * f_i.  The angle needs p * f_i / 2 pi only
// modulo 1, so the plan holds f_i / 2 pi as a 64-bit fraction F of a turn and
// the kernel takes p * F modulo 2^64: an integer product that is exact for
// every int32 position, where an fp32 product would be off by p * 2^-25
// radians.  The upper 32 bits, as a signed number of half turns, go to sincospi.
//
// Bound by memory: each entry is read once and written once.  A block takes a
// few tokens, works out their sines and cosines once into shared memory, and
// then runs over all the heads of q and k with 16-byte loads and stores.
// 8192 tokens of 32 + 8 heads of 128 in bf16 take 28.6 us in a graph (5.9 TB/s); 16
// tokens 2.1 us.
#include "paged.cuh"

#include <algorithm>

namespace sp {
namespace {

constexpr int kRotThreads = 256;

// What the kernel takes of a plan of at most kPairs pairs: a launch's time on the host grows with its arguments (with room for
// 128 pairs, 1.4 KB of them, a call for heads of 64 took 2 us more).
template <int kPairs>
struct RotArgs {
    int rot;
    uint64_t turns[kPairs];
    uint8_t axis[kPairs];
    const int32_t* pos;
    int64_t pos_stride, T;
    int d, H, Hk;
    int tokens;             // tokens a block takes
    float sign;             // -1: inverse
    sp_rows q, qo, k, ko;
};

// Rotates eight pairs: x0/x1 hold the pairs' entries (half layout: the two
// halves' entries; interleaved: 16 consecutive entries).  cs: cosines and sines of
// two pairs each, `stride` apart.
__device__ __forceinline__ void rotate8(float (&x0)[8], float (&x1)[8], const float4* cs, int stride, float sign, bool inter) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float4 v = cs[k * stride];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const int i = 2 * k + y;
            const float c = y ? v.z : v.x, s = (y ? v.w : v.y) * sign;
            float& a = inter ? (i < 4 ? x0[(2 * i) & 7] : x1[(2 * i) & 7]) : x0[i];
            float& b = inter ? (i < 4 ? x0[(2 * i + 1) & 7] : x1[(2 * i + 1) & 7]) : x1[i];
            const float u = a, w = b;
            a = u * c - w * s;
            b = w * c + u * s;
        }
    }
}

template <typename T, bool kInter, int kPairs>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const __grid_constant__ RotArgs<kPairs> p) {
    // [tokens][4][pairs / 8] cosine, sine of pairs 8c + 2k and 8c + 2k + 1 at (k, c): a warp's lanes have consecutive c, so
    // they read consecutive 16 bytes
    extern __shared__ float4 cs[];
    const int pairs = p.rot / 2, rc = pairs / 8;
    const int64_t t0 = (int64_t)blockIdx.x * p.tokens;
    const int nt = (int)min((int64_t)p.tokens, p.T - t0);
    for (int i = threadIdx.x; i < nt * pairs; i += kRotThreads) {
        const int t = i / pairs, j = i - t * pairs;
        const int64_t at = p.pos[p.axis[j] * p.pos_stride + t0 + t];
        const int32_t half_turns = (int32_t)(((uint64_t)at * p.turns[j]) >> 32);
        float s, c;
        sincospif((float)half_turns * 0x1p-31f, &s, &c);
        reinterpret_cast<float2*>(cs)[((t * 4 + ((j & 7) >> 1)) * rc + (j >> 3)) * 2 + (j & 1)] = make_float2(c, s);
    }
    __syncthreads();
    // a thread has one chunk, of eight pairs or of eight entries past rot, of every so many heads
    const int chunks = rc + (p.d - p.rot) / 8, heads = p.H + p.Hk, sweep = kRotThreads / chunks;
    const int c = threadIdx.x % chunks, first = threadIdx.x / chunks;
    if (first >= sweep) return;
    int h = first + blockIdx.y * sweep, t = 0;
    for (;; h += sweep * gridDim.y) {
        while (h >= heads) {
            h -= heads;
            ++t;
        }
        if (t >= nt) return;
        const bool isq = h < p.H;
        const sp_rows& in = isq ? p.q : p.k;
        const sp_rows& out = isq ? p.qo : p.ko;
        const int hh = isq ? h : h - p.H;
        const T* src = static_cast<const T*>(in.data) + (t0 + t) * in.stride_row + hh * in.stride_head;
        T* dst = static_cast<T*>(out.data) + (t0 + t) * out.stride_row + hh * out.stride_head;
        float x0[8], x1[8];
        if (c >= rc) {
            const int e = p.rot + (c - rc) * 8;
            load8(src + e, x0);
            store8(dst + e, x0);
            continue;
        }
        const int e0 = kInter ? c * 16 : c * 8, e1 = kInter ? c * 16 + 8 : pairs + c * 8;
        load8(src + e0, x0);
        load8(src + e1, x1);
        rotate8(x0, x1, cs + t * 4 * rc + c, rc, p.sign, kInter);
        store8(dst + e0, x0);
        store8(dst + e1, x1);
    }
}

template <typename T, int kPairs>
sp_status launch(const sp_rotary_plan& plan, RotArgs<kPairs> a, cudaStream_t st) {
    const int rot = plan.rot;
    a.rot = rot;
    for (int i = 0; i < rot / 2; ++i) {
        a.turns[i] = plan.turns[i];
        a.axis[i] = plan.axis[i];
    }
    a.tokens = 2;
    const int64_t blocks = (a.T + a.tokens - 1) / a.tokens;
    const int per = (a.H + a.Hk) * (rot / 16 + (a.d - rot) / 8) * a.tokens;
    // few tokens: several blocks share a token's heads, so that an SM has four
    const int64_t want = 4 * sm_count();
    const int split = blocks >= want ? 1 : (int)std::min<int64_t>((per + kRotThreads - 1) / kRotThreads, (want + blocks - 1) / blocks);
    const size_t smem = (size_t)a.tokens * (rot / 2) * sizeof(float2);
    const dim3 grid((unsigned)blocks, (unsigned)std::max(1, split));
    if (plan.interleaved) rotary_kernel<T, true, kPairs><<<grid, kRotThreads, smem, st>>>(a);
    else rotary_kernel<T, false, kPairs><<<grid, kRotThreads, smem, st>>>(a);
    SP_LAUNCH_CHECK();
    return SP_OK;
}

template <int kPairs>
sp_status fill(const sp_rotary_plan& plan, const int32_t* pos, int64_t pos_stride, int64_t T, int d, sp_dtype dtype, bool inverse,
               const sp_rows& q, const sp_rows& qo, int H, const sp_rows& k, const sp_rows& ko, int Hk, cudaStream_t st) {
    RotArgs<kPairs> a;
    a.pos = pos; a.pos_stride = pos_stride; a.T = T; a.d = d; a.H = H; a.Hk = Hk;
    a.sign = inverse ? -1.f : 1.f;
    a.q = q; a.qo = qo; a.k = k; a.ko = ko;
    return dtype == SP_BF16 ? launch<__nv_bfloat16>(plan, a, st) : launch<float>(plan, a, st);
}

}  // namespace

sp_status rotary_launch(const sp_rotary_plan& plan, const int32_t* pos, int64_t pos_stride, int64_t T, int d,
                        sp_dtype dtype, bool inverse, const sp_rows& q, const sp_rows& qo, int H, const sp_rows& k,
                        const sp_rows& ko, int Hk, cudaStream_t st) {
    if (T == 0 || H + Hk == 0) return SP_OK;
    return plan.rot <= 64    ? fill<32>(plan, pos, pos_stride, T, d, dtype, inverse, q, qo, H, k, ko, Hk, st)
           : plan.rot <= 128 ? fill<64>(plan, pos, pos_stride, T, d, dtype, inverse, q, qo, H, k, ko, Hk, st)
                             : fill<128>(plan, pos, pos_stride, T, d, dtype, inverse, q, qo, H, k, ko, Hk, st);
}

}  // namespace sp
