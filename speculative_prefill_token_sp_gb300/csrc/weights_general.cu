// The attention weight that cached tokens gather: the general path (both types, every head dimension, page size and number of rows).
//
//   w[i] = decay * w[i] + sum over the rows that see token i of 2^(f q . k_i - l),  f = scale * log2(e), l = lse * log2(e)
//
// Each row's normaliser is known, so the rows may be taken in any order and a key's sum needs no other key.  A key's row is held by a
// group of 2^g lanes, eight entries a lane (the smallest 2^g >= d / 8), and a group holds kKeys keys, so that a query row, read
// once for all of them, goes through the lanes' registers while the next one is on its way.  A CTA's warps have different
// keys; its unit is all keys that they hold at a time, and the units of all (sequence, KV head) pairs are cut into equal
// runs.  Nothing is added up across threads but the dot products, so the same call gives the same bits.
// Arithmetic is fp32 on the CUDA cores, and bounds the kernel for many rows: a chunk of 4096 tokens over 32768 (bf16, 32/8 heads of
// 128), which the tensor-core kernel takes in 0.83 ms, is 143 ms here, and a step of 16 requests of 2K to 32K tokens 165 us for 27.
#include "attend_split.cuh"

#include <type_traits>

namespace sp {
namespace {

constexpr int kThreads = 128, kWarps = 4, kKeys = 4;
constexpr int kFlush = 64;          // rows whose weights are summed before the sum goes to the total: long sums keep their low bits

template <typename T, int kKind>
__device__ __forceinline__ void load_key(const sp_cache& c, int64_t at, int64_t scale_at, float (&x)[8]) {
    if constexpr (kKind == SP_CACHE_SAME) {
        load8(static_cast<const T*>(c.k) + at, x);
    } else {
        decode8<kKind>(*reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(c.k) + at), x);
        const float scale = c.k_scale[scale_at];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= scale;
    }
}

struct GeneralArgs {
    WeightsProblem w;
    SplitArgs split;        // (of the division into runs alone: its rows and many are set so that a sequence is one item)
    int lg;
};

template <typename T, int kKind>
__global__ void __launch_bounds__(kThreads) weights_general_kernel(const __grid_constant__ GeneralArgs p) {
    const AttendProblem& a = p.w.a;
    const sp_cache& c = a.cache;
    if (blockIdx.x == gridDim.x - 1) {
        check_tokens(a.batch, c, a.window, false, p.split.hdr);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, lanes = 1 << p.lg, sub = lane & (lanes - 1), grp = lane >> p.lg;
    const int per_warp = kKeys * (32 >> p.lg), unit = kWarps * per_warp, G = p.split.G;
    const bool act = sub * 8 < c.d;
    const float f = a.scale * 1.4426950408889634f;
    bool bad = false;
    const int64_t U = total_units(p.split, unit, bad);
    const Shares shares(U, p.split.P);
    int64_t u = shares.at(blockIdx.x);
    const int64_t u_end = shares.at(blockIdx.x + 1);
    int64_t begin = 0;
    int b = u < u_end ? find_unit(p.split, unit, u, begin) : 0;
    while (u < u_end && b < a.batch.B) {
        const Seq s = load_seq(a.batch, c.page, b);
        const Span span = span_of(s, a.window, unit);
        const int64_t in_seq = u - begin, mine = (int64_t)span.units * c.H_kv * row_blocks(p.split, s);
        if (in_seq >= mine) {
            begin += mine;
            ++b;
            continue;
        }
        const int g = (int)divide(in_seq, span.units);
        if (g >= c.H_kv) {          // a second item of over 2^31 rows: all rows are taken in the first
            ++u;
            continue;
        }
        const int k0 = span.first + (int)(in_seq - (int64_t)g * span.units) * unit;
        ++u;
        const int ctx = s.kv - s.n;
        // this group's keys, and the new tokens that see any key of the unit
        float key[kKeys][8], sum[kKeys], total[kKeys];
        int64_t at[kKeys];
        int tok[kKeys];
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
            tok[i] = k0 + warp * per_warp + i * (32 >> p.lg) + grp;
            at[i] = -1;
            sum[i] = total[i] = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) key[i][e] = 0.f;
            if (tok[i] >= s.kv) continue;
            const int q = a.page_of(tok[i]), pg = a.batch.table[(int64_t)b * a.batch.table_stride + q], slot = tok[i] - q * c.page;
            if (pg < 0 || pg >= c.pages) continue;
            at[i] = scale_offset(c, pg, g, slot);
            if (act) load_key<T, kKind>(c, row_offset(c, pg, g, slot) + sub * 8, at[i], key[i]);
        }
        const int t0 = max(0, k0 - ctx);
        const int t1 = a.window ? (int)min((int64_t)s.n, (int64_t)min(k0 + unit, s.kv) - 1 + a.window - ctx) : s.n;
        float next[8] = {}, next_l = 0.f;
        auto fetch = [&](int t, int h) {
            if (act) load8(static_cast<const T*>(a.q.data) + (s.row0 + t) * a.q.stride_row + h * a.q.stride_head + sub * 8, next);
            next_l = a.lse[(s.row0 + t) * a.lse_stride_row + h * a.lse_stride_head];
        };
        if (t0 < t1) fetch(t0, g * G);
        int rows = 0;
        for (int t = t0, h = 0; t < t1;) {
            float q[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) q[e] = next[e];
            // a row that saw no token has the sum 0, whose logarithm is -inf, and gives nothing
            const float l = next_l == -INFINITY ? INFINITY : next_l * 1.4426950408889634f;
            const int place = ctx + t;
            if (++h == G) h = 0, ++t;
            if (t < t1) fetch(t, g * G + h);
            float x[kKeys];
#pragma unroll
            for (int i = 0; i < kKeys; ++i) {
                x[i] = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) x[i] += q[e] * key[i][e];
            }
            for (int w = 1; w < lanes; w <<= 1) {
#pragma unroll
                for (int i = 0; i < kKeys; ++i) x[i] += __shfl_xor_sync(0xffffffffu, x[i], w);
            }
#pragma unroll
            for (int i = 0; i < kKeys; ++i) {
                const bool seen = tok[i] <= place && (!a.window || tok[i] > place - a.window);
                const float w = ex2(x[i] * f - l);
                if (seen) sum[i] += w;
            }
            if (++rows % kFlush == 0) {
#pragma unroll
                for (int i = 0; i < kKeys; ++i) total[i] += sum[i], sum[i] = 0.f;
            }
        }
        if (sub == 0) {
#pragma unroll
            for (int i = 0; i < kKeys; ++i) {
                if (at[i] < 0) continue;
                float w = total[i] + sum[i];
                if (tok[i] < ctx && p.w.decay != 0.f) w += p.w.decay * p.w.weights[at[i]];
                p.w.weights[at[i]] = w;
            }
        }
    }
}

template <typename T>
void launch(const GeneralArgs& p, cudaStream_t st) {
    const unsigned grid = (unsigned)p.split.P + 1;
    switch (p.w.a.cache.kind) {
        case SP_CACHE_SAME: weights_general_kernel<T, SP_CACHE_SAME><<<grid, kThreads, 0, st>>>(p); break;
        case SP_CACHE_E4M3: weights_general_kernel<T, SP_CACHE_E4M3><<<grid, kThreads, 0, st>>>(p); break;
        default: weights_general_kernel<T, SP_CACHE_INT8><<<grid, kThreads, 0, st>>>(p); break;
    }
}

}  // namespace

sp_status weights_general_launch(const WeightsProblem& w, void* ws, cudaStream_t st) {
    GeneralArgs p;
    p.w = w;
    p.split.a = w.a;
    p.split.G = w.a.H / w.a.cache.H_kv;
    p.split.rows = INT32_MAX;           // a sequence with new tokens is one item a KV head
    p.split.many = 1;
    p.split.P = 4 * sm_count();
    p.split.hdr = static_cast<WsHeader*>(ws);
    p.split.err = nullptr;
    p.split.part_o = nullptr;
    p.split.part_ml = nullptr;
    p.lg = 0;
    while ((8 << p.lg) < w.a.cache.d) ++p.lg;
    if (w.a.cache.dtype == SP_BF16) launch<__nv_bfloat16>(p, st);
    else launch<float>(p, st);
    SP_LAUNCH_CHECK();
    return SP_OK;
}

}  // namespace sp
