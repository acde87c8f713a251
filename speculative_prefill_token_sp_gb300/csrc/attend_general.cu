// Attention of new tokens over the paged cache: the general path (both types,
// every head dimension, page size and number of rows).
//
// One pass over a row's keys with the running maximum m and sum z of its
// softmax (base 2): x = log2(e) * scale * q.k; when x exceeds m, the sums are
// scaled by 2^(m - x).  All arithmetic is fp32 on the CUDA cores.  A key's row is
// held by a group of 2^g lanes, eight entries a lane (the smallest 2^g >= d / 8),
// so a warp has 32 / 2^g keys in hand; each group keeps its own m, z and sums of
// four query rows of one KV head, and the groups, warps and CTAs are joined at the
// end.  A key and its value are read once for the four rows, and the next ones
// are requested before these are used.  Per key and row a lane spends 16
// multiply-adds, g shuffles and about ten other instructions, which bounds the
// kernel for many rows; for few it is bound by the latency of its loads, so the
// keys are cut over all the CTAs that the SMs hold.  One fp32 token over 512 (4 query
// heads on 2 of 64) takes 10.1 us with the joining kernel, over 8192 13 us;
// one token each of 16 requests over 32768 (16 on 4 heads of 64, fp32) 340 us (3.2 TB/s).
// Chunks are far from the tensor cores' time: 256 tokens over 4096, 32 query heads on 8, bf16, take
// 2.1 ms (d = 96) or 4.3 ms (d = 256), 30 us at d = 128 in attend_tc.cu; with d = 96, one token each of 16
// requests of 2K to 32K (16 on 4 heads) 320 us; fp32, 128 tokens over 4096 (4 on 2 heads of 64) 89 us.
#include "attend_split.cuh"

#include <algorithm>
#include <type_traits>

namespace sp {
namespace {

constexpr int kGenRows = 4, kGenWarps = 4, kGenThreads = 32 * kGenWarps;
constexpr int kUnit = 64, kWarpKeys = kUnit / kGenWarps;     // keys of a unit, and of a warp's share of it

template <typename T, int kKind>
struct Row8 {       // eight entries of a cached row as they are loaded
    static constexpr bool kSame = kKind == SP_CACHE_SAME;
    using Raw = typename std::conditional<kSame, typename std::conditional<sizeof(T) == 4, float[8], uint4>::type, uint2>::type;
    Raw raw;
    float scale;
    __device__ __forceinline__ void load(const void* data, const float* scales, int64_t at, int64_t scale_at) {
        if constexpr (!kSame) {
            raw = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(data) + at);
            scale = scales[scale_at];
        } else if constexpr (sizeof(T) == 4) {
            load8(static_cast<const float*>(data) + at, raw);
        } else {
            raw = *reinterpret_cast<const uint4*>(static_cast<const T*>(data) + at);
        }
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        if constexpr (!kSame) {
            decode8<kKind>(raw, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] *= scale;
        } else if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = raw[i];
        } else {
            unpack8(raw, x);
        }
    }
};

// Adds the sums (m2, z2, o2) to (m, z, o).
__device__ __forceinline__ void join(float& m, float& z, float (&o)[8], float m2, float z2, const float (&o2)[8]) {
    const float top = fmaxf(m, m2), ref = top == -INFINITY ? 0.f : top;
    // a side without a maximum has summed nothing, or NaN alone: its sums count as they are
    const float a = m == -INFINITY ? 1.f : ex2(m - ref), b = m2 == -INFINITY ? 1.f : ex2(m2 - ref);
    z = z * a + z2 * b;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = o[i] * a + o2[i] * b;
    m = top;
}

// Adds up the sums of a warp's groups of `lanes` lanes.
__device__ __forceinline__ void join_groups(float& m, float& z, float (&o)[8], int lanes) {
    for (int w = lanes; w < 32; w <<= 1) {
        float o2[8];
        const float m2 = __shfl_xor_sync(0xffffffffu, m, w), z2 = __shfl_xor_sync(0xffffffffu, z, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) o2[e] = __shfl_xor_sync(0xffffffffu, o[e], w);
        join(m, z, o, m2, z2, o2);
    }
}

template <typename T>
__device__ __forceinline__ void write_out(const SplitArgs& p, int64_t row, int h, int e, float m, float z, float (&o)[8]) {
    const float inv = z == 0.f ? 0.f : 1.f / z;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = z == 0.f ? 0.f : o[i] * inv;
    store8(static_cast<T*>(p.a.out.data) + row * p.a.out.stride_row + h * p.a.out.stride_head + e, o);
    if (p.a.lse && e == 0)
        p.a.lse[row * p.a.lse_stride_row + h * p.a.lse_stride_head] =
            z == 0.f ? -INFINITY : (m + log2f(z)) * 0.6931471805599453f;
}

// kTree: the new tokens are drafted ones, and p.a.seen says which of them each sees.
template <typename T, int kKind, bool kTree>
__global__ void __launch_bounds__(kGenThreads, 3) general_kernel(const __grid_constant__ SplitArgs p, int lg) {
    __shared__ float sm_o[kGenWarps][kGenRows][256];
    __shared__ float2 sm_ml[kGenWarps][kGenRows];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int lanes = 1 << lg, sub = lane & (lanes - 1), grp = lane >> lg, step = 32 >> lg;
    const sp_cache& c = p.a.cache;
    const bool act = sub * 8 < c.d;
    bool bad_seq = false, bad_page = false;
    cudaTriggerProgrammaticLaunchCompletion();
    const int64_t U = total_units(p, kUnit, bad_seq);
    const Shares shares(U, p.P);
    int64_t u = shares.at(blockIdx.x);
    const int64_t u_end = shares.at(blockIdx.x + 1);
    int64_t begin = 0;
    int b = u < u_end ? find_unit(p, kUnit, u, begin) : 0;
    const float f = p.a.scale * 1.4426950408889634f;
    while (u < u_end && b < p.a.batch.B) {         // (b: should the arrays be changed while the kernel runs)
        const Seq s = load_seq(p.a.batch, c.page, b);
        const Span span = span_of(s, p.a.window, kUnit);
        const int blocks = row_blocks(p, s);
        const int64_t in_seq = u - begin, mine = (int64_t)blocks * c.H_kv * span.units;
        if (in_seq >= mine) {
            begin += mine;
            ++b;
            continue;
        }
        const int64_t item = divide(in_seq, span.units);
        const int g = (int)divide(item, blocks), rb = (int)(item - (int64_t)g * blocks), from = (int)(in_seq - item * span.units);
        const int to = (int)min((int64_t)span.units, from + (u_end - u));
        const int64_t r0 = (int64_t)rb * kGenRows;
        const int rows = (int)min((int64_t)kGenRows, (int64_t)s.n * p.G - r0);

        float q[kGenRows][8], o[kGenRows][8], m[kGenRows], z[kGenRows];
        int last[kGenRows], drafted[kGenRows];      // drafted tokens: `last` is the row's place, which the window goes by
        int item_last = kTree ? s.kv - 1 : -1;
#pragma unroll
        for (int i = 0; i < kGenRows; ++i) {
            m[i] = -INFINITY;
            z[i] = 0.f;
            last[i] = -1;
            drafted[i] = -1;
#pragma unroll
            for (int e = 0; e < 8; ++e) q[i][e] = o[i][e] = 0.f;
            if (i >= rows) continue;
            const int t = (int)divide(r0 + i, p.G), h = g * p.G + (int)(r0 + i - (int64_t)t * p.G);
            if (act) load8(static_cast<const T*>(p.a.q.data) + (s.row0 + t) * p.a.q.stride_row + h * p.a.q.stride_head + sub * 8, q[i]);
            if constexpr (kTree) {
                drafted[i] = t;
                last[i] = p.a.window ? place_of_drafted(p.a, s, t) : 0;
            } else {
                last[i] = s.kv - s.n + t;
                item_last = max(item_last, last[i]);
            }
        }

        // this group's keys: of each unit's share of the warp, every step-th
        const int per = max(1, kWarpKeys / step), n_keys = (to - from) * per;
        const int32_t* table = p.a.batch.table + (int64_t)b * p.a.batch.table_stride;
        auto token = [&](int j) {
            const int k = j / per, off = (j - k * per) * step + grp;
            // past the share (step > kWarpKeys), past the item's last row, past the run: no token
            const int tok = span.first + (from + k) * kUnit + warp * kWarpKeys + off;
            return j < n_keys && off < kWarpKeys && tok <= item_last && tok < s.kv ? tok : -1;
        };
        auto page_of = [&](int tok) { return tok >= 0 ? table[p.a.page_of(tok)] : 0; };
        Row8<T, kKind> k0, v0, k1, v1;
        auto request = [&](int& tok, int pg, Row8<T, kKind>& k, Row8<T, kKind>& v) {
            if (tok < 0) return;
            if ((unsigned)pg >= (unsigned)c.pages) {
                bad_page = true;
                tok = -1;
                return;
            }
            if (!act) return;
            const int slot = tok - p.a.page_of(tok) * c.page;
            const int64_t at = row_offset(c, pg, g, slot) + sub * 8, sc = scale_offset(c, pg, g, slot);
            k.load(c.k, c.k_scale, at, sc);
            v.load(c.v, c.v_scale, at, sc);
        };
        // Adds a key.  The first R rows at once and without branches between them, so that their shuffles and exponentials overlap.
        auto add = [&](auto R, int tok, const float (&k)[8], const float (&v)[8]) {
            constexpr int kR = decltype(R)::value;
            float x[kR];
            bool seen[kR], grows = false;
#pragma unroll
            for (int i = 0; i < kR; ++i) {
                x[i] = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) x[i] += q[i][e] * k[e];
            }
            for (int w = 1; w < lanes; w <<= 1) {
#pragma unroll
                for (int i = 0; i < kR; ++i) x[i] += __shfl_xor_sync(0xffffffffu, x[i], w);
            }
#pragma unroll
            for (int i = 0; i < kR; ++i) {
                if constexpr (kTree) {
                    const int u = tok - (s.kv - s.n);
                    if (tok < 0 || drafted[i] < 0) seen[i] = false;
                    else if (u < 0) seen[i] = !p.a.window || tok > last[i] - p.a.window;
                    else seen[i] = seen_word(p.a, s, drafted[i], u >> 5) >> (u & 31) & 1;
                } else {
                    seen[i] = tok >= 0 && tok <= last[i] && (!p.a.window || tok > last[i] - p.a.window);
                }
                x[i] = seen[i] ? x[i] * f : -INFINITY;
                grows |= x[i] > m[i];
            }
            if (grows) {
#pragma unroll
                for (int i = 0; i < kR; ++i) {
                    const float top = fmaxf(m[i], x[i]), a = m[i] == top ? 1.f : ex2(m[i] - top);
                    m[i] = top;
                    z[i] *= a;
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[i][e] *= a;
                }
            }
#pragma unroll
            for (int i = 0; i < kR; ++i) {
                const float w2 = ex2(x[i] - (m[i] == -INFINITY ? 0.f : m[i]));
                z[i] += w2;
                if (seen[i]) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[i][e] += w2 * v[e];
                }
            }
        };
        auto use = [&](int tok, const Row8<T, kKind>& kr, const Row8<T, kKind>& vr) {
            float k[8] = {}, v[8] = {};
            if (tok >= 0 && act) {
                kr.get(k);
                vr.get(v);
            }
            if (rows > 2) add(std::integral_constant<int, 4>{}, tok, k, v);
            else if (rows == 2) add(std::integral_constant<int, 2>{}, tok, k, v);
            else add(std::integral_constant<int, 1>{}, tok, k, v);
        };
        int t0 = token(0), t1 = token(1);
        int pg0 = page_of(t0), pg1 = page_of(t1);
        request(t0, pg0, k0, v0);
        for (int j = 0; j < n_keys; j += 2) {
            const int t2 = token(j + 2);
            const int pg2 = page_of(t2);
            request(t1, pg1, k1, v1);
            use(t0, k0, v0);
            const int t3 = token(j + 3);
            const int pg3 = page_of(t3);
            t0 = t2;
            request(t0, pg2, k0, v0);
            use(t1, k1, v1);
            t1 = t3;
            pg1 = pg3;
        }

        // join the groups of the warp, then the warps
#pragma unroll
        for (int i = 0; i < kGenRows; ++i) {
            if (i >= rows) break;
            join_groups(m[i], z[i], o[i], lanes);
            if (grp == 0) {
                if (sub == 0) sm_ml[warp][i] = make_float2(m[i], z[i]);
                if (act) store8(&sm_o[warp][i][sub * 8], o[i]);
            }
        }
        __syncthreads();
        const bool whole = from == 0 && to == span.units;
        const int chunks = c.d / 8;
        for (int i = threadIdx.x; i < rows * chunks; i += kGenThreads) {
            const int r = i / chunks, e = (i - r * chunks) * 8;
            float mm = sm_ml[0][r].x, zz = sm_ml[0][r].y, v[8];
            load8(&sm_o[0][r][e], v);
#pragma unroll
            for (int w = 1; w < kGenWarps; ++w) {
                float o2[8];
                load8(&sm_o[w][r][e], o2);
                join(mm, zz, v, sm_ml[w][r].x, sm_ml[w][r].y, o2);
            }
            if (whole) {
                const int64_t t = divide(r0 + r, p.G);
                write_out<T>(p, s.row0 + t, g * p.G + (int)(r0 + r - t * p.G), e, mm, zz, v);
            } else {
                const int64_t slot = ((int64_t)blockIdx.x * 2 + (from == 0 ? 1 : 0)) * kRows + r;
                store8(p.part_o + slot * c.d + e, v);
                if (e == 0) p.part_ml[slot] = make_float2(mm, zz);
            }
        }
        __syncthreads();
        u += to - from;
    }
    const int any = (__syncthreads_or(bad_seq) ? 1 : 0) | (__syncthreads_or(bad_page) ? 2 : 0);
    if (threadIdx.x == 0) p.err[blockIdx.x] = any;
}

constexpr int kJoinWarps = 8;

// Joins the parts of the items that were cut: block (i, r) takes row r of the item whose first cut is the one before CTA i + 1.  Each
// group of 2^lg lanes has eight entries a lane of every so many parts, the next of them on the way while one is added: an
// item may be cut into hundreds (one after the other they took 0.4 us each).
template <typename T>
__global__ void __launch_bounds__(32 * kJoinWarps) general_join_kernel(const __grid_constant__ SplitArgs p, int lg) {
    __shared__ float sm_o[kJoinWarps][256];
    __shared__ float2 sm_ml[kJoinWarps];
    bool bad = false;
    const int64_t U = total_units(p, kUnit, bad);
    const Shares shares(U, p.P);
    const int c = blockIdx.x + 1, r = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t u = shares.at(c);
    int64_t begin = 0;
    const int b = u < U ? find_unit(p, kUnit, u, begin) : p.a.batch.B;
    const Seq s = b < p.a.batch.B ? load_seq(p.a.batch, p.a.cache.page, b) : Seq{0, 0, 0, true};
    cudaGridDependencySynchronize();        // the main kernel's parts
    if (blockIdx.x == 0 && r == 0) gather_status(p);
    if (b >= p.a.batch.B) return;
    const int units = span_of(s, p.a.window, kUnit).units, blocks = row_blocks(p, s);
    const int64_t item = divide(u - begin, units), first = begin + item * units;
    if (u == first || shares.at(c - 1) > first) return;       // no cut, or not the item's first
    const int g = (int)divide(item, blocks);
    const int64_t row = (item - (int64_t)g * blocks) * kGenRows + r;
    if (row >= (int64_t)s.n * p.G) return;
    const int lanes = 1 << lg, e = (lane & (lanes - 1)) * 8, groups = 32 * kJoinWarps >> lg;
    const bool act = e < p.a.cache.d;
    const int c1 = shares.of(first + units - 1);
    struct Part {
        float2 ml;
        float o[8];
    };
    auto fetch = [&](int k) {
        Part x = {make_float2(-INFINITY, 0.f), {}};
        if (k > c1) return x;
        const int64_t slot = ((int64_t)k * 2 + (k == c - 1 ? 1 : 0)) * kRows + r;
        x.ml = p.part_ml[slot];
        if (act) load8(p.part_o + slot * p.a.cache.d + e, x.o);
        return x;
    };
    float m = -INFINITY, z = 0.f, o[8] = {};
    const int k0 = c - 1 + (threadIdx.x >> lg);
    Part next = fetch(k0);
    for (int k = k0; k <= c1; k += groups) {
        const Part x = next;
        next = fetch(k + groups);
        join(m, z, o, x.ml.x, x.ml.y, x.o);
    }
    __syncwarp();
    join_groups(m, z, o, lanes);
    if (lane < lanes) {
        if (lane == 0) sm_ml[warp] = make_float2(m, z);
        if (act) store8(&sm_o[warp][e], o);
    }
    __syncthreads();
    if (warp > 0 || lane >= lanes || !act) return;
#pragma unroll
    for (int w = 1; w < kJoinWarps; ++w) {
        float o2[8];
        load8(&sm_o[w][e], o2);
        join(m, z, o, sm_ml[w].x, sm_ml[w].y, o2);
    }
    const int64_t t = divide(row, p.G);
    write_out<T>(p, s.row0 + t, g * p.G + (int)(row - t * p.G), e, m, z, o);
}

int general_ctas() { return sm_count() * 3; }

template <typename T, int kKind>
void launch_kind(const SplitArgs& p, int lg, cudaStream_t st, bool tree) {
    if (tree) general_kernel<T, kKind, true><<<p.P, kGenThreads, 0, st>>>(p, lg);
    else general_kernel<T, kKind, false><<<p.P, kGenThreads, 0, st>>>(p, lg);
}
template <typename T>
void launch_main(const SplitArgs& p, int lg, cudaStream_t st, bool tree) {
    switch (p.a.cache.kind) {
        case SP_CACHE_SAME: launch_kind<T, SP_CACHE_SAME>(p, lg, st, tree); break;
        case SP_CACHE_E4M3: launch_kind<T, SP_CACHE_E4M3>(p, lg, st, tree); break;
        default: launch_kind<T, SP_CACHE_INT8>(p, lg, st, tree); break;
    }
}

template <typename T>
sp_status launch(const SplitArgs& p, cudaStream_t st) {
    int lg = 0;
    while ((8 << lg) < p.a.cache.d) ++lg;
    launch_main<T>(p, lg, st, p.a.seen != nullptr);
    SP_LAUNCH_CHECK();
    const int64_t rows = std::min<int64_t>(kGenRows, (int64_t)p.a.batch.max_new * p.G);
    const dim3 grid((unsigned)p.P - 1, (unsigned)std::max<int64_t>(1, rows));
    return launch_early(general_join_kernel<T>, grid, 32 * kJoinWarps, (size_t)0, st, p, lg);
}

}  // namespace

size_t attend_general_ws_bytes(const sp_cache& c) { return split_ws_bytes((size_t)general_ctas(), c.d); }

sp_status attend_general_launch(const AttendProblem& a, void* ws, cudaStream_t st) {
    const SplitArgs p = split_args(a, kGenRows, true, general_ctas(), ws);
    return a.cache.dtype == SP_BF16 ? launch<__nv_bfloat16>(p, st) : launch<float>(p, st);
}

}  // namespace sp
