// Attention of few new tokens (decode and look-ahead steps) over the paged
// cache: bf16, head dimension 64 or 128, sequences of at most 16 query rows
// per KV head (a row is a new token's query head of the group).
//
// One pass over the keys with the running maximum and sum of each row's
// softmax (base 2).  The work is bound by the cache's bytes, so what counts is
// that enough of them are under way: each warp copies the rows of its next piece
// (16 tokens, 32 where a row has at most 128 bytes) into its own ring in shared
// memory with cp.async while it works on the piece before, with no barrier with
// another warp; the four warps of a CTA take consecutive pieces of a unit of 64
// (128) tokens.  Rows in the ring are 16 bytes apart from a multiple of 64, so
// that the operand reads meet no bank twice.
//
// The products are mma.sync, transposed, so that the query rows (8 a tile, few)
// are the narrow side and the accumulators are small.  Both sum over an index
// whose order does not matter (the entries of a head, the tokens), so the order
// is chosen such that a lane's operand registers are 16 consecutive bytes of a
// row.  Lane (n, q) = (lane / 4, lane % 4):
//  * S^T = K Q^T: of tokens n and n + 8 the 16-byte pieces 2q, 2q + 1 of each
//    eight; Q is laid out the same way;
//  * O^T = V^T P^T: of tokens 2q, 2q + 1, 2q + 8, 2q + 9 the entries [c * 8E +
//    n * E, + E); a byte permute pairs two tokens' entries.  P^T needs its 8 x 8
//    tiles transposed (movmatrix).  A lane's sums are runs of E consecutive
//    entries of rows 2q and 2q + 1.
// Codes of an 8-bit cache become fp16 for the first product, one instruction a pair (the query rows too, each times a
// power of two that brings its largest entry near 2^10: an entry is exact unless it is below 2^-27 of that one, and then off by at
// most 2^-35 of it).  For the second they become bf16, as its weights carry the values' scales, whose range fp16 does not have.
// The tensor cores' time at these row counts is a fraction of the loads'.
//
// The units of all (sequence, KV head) pairs are laid end to end and cut into
// equal runs, one per resident CTA, so a batch of any mixture of lengths keeps
// every SM busy to the end; a pair that is cut leaves partial sums in the
// workspace, and a second kernel, launched early, joins them in a fixed order.
//
// The weights are rounded to bf16 (2^-8 of each; z sums them unrounded), the operand type of the second product.
//
// In a graph, one token each of 16 requests of 2K to 32K (bf16, 16 query heads on 4 of
// 64) takes 49.5 us (5.3 TB/s), one over 131072 (e4m3, 32 on 8 of 128) 56.5 to 57.8 us (4.8 TB/s).  One
// over 131072, 262144, 524288 and 1048576 takes 56, 102, 193, 366 us (e4m3) and 92, 173, 333,
// 656 us (bf16): 6.25 and 6.66 TB/s along the length, 92 and 98% of the copy rate, and 12 us
// that do not grow with it, nearly all of them in this kernel (start, first loads, the last units).
// The integer pipe is 56% busy with the 8-bit kinds.  The e4m3
// case with operands loaded from global memory into registers 117 us, then with the rings 83 us.
#include "attend_split.cuh"

#include <cuda_fp16.h>

#include <algorithm>

namespace sp {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;

template <int D, int kKind>
constexpr int warp_tokens() { return kKind == SP_CACHE_SAME && D == 128 ? 16 : 32; }
template <int D, int kKind>
constexpr int unit_tokens() { return kWarps * warp_tokens<D, kKind>(); }


__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int kBytes>
struct Chunk {
    uint32_t w[kBytes / 4];
};
template <int kBytes>
__device__ __forceinline__ Chunk<kBytes> read_chunk(const uint8_t* p) {
    Chunk<kBytes> c;
    if constexpr (kBytes == 16) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        c.w[0] = v.x; c.w[1] = v.y; c.w[2] = v.z; c.w[3] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        c.w[0] = v.x; c.w[1] = v.y;
    }
    return c;
}

// Copies kBytes (16 or 4) to shared memory in the background; zeros where `there` is false.
template <int kBytes>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool there) {
    const int size = there ? kBytes : 0;
    if constexpr (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(size) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(size) : "memory");
}

// The ring of a warp: kStages pieces, each its tokens' K rows, V rows and scales.
template <int D, int kKind, int kN>
struct Ring {
    static constexpr int kTok = warp_tokens<D, kKind>();
    static constexpr int kRow = D * (kKind == SP_CACHE_SAME ? 2 : 1), kPitch = kRow + 16;
    static constexpr int kV = kTok * kPitch, kScales = 2 * kV;
    static constexpr int kStage = kScales + (kKind == SP_CACHE_SAME ? 0 : kTok * 8);
    static constexpr int kCtas = kN == 1 ? 3 : 2;                       // resident on an SM
    static constexpr int kStages = kN == 1 ? 2 : 3;
    static constexpr int kBytes = kWarps * kStages * kStage;
    static constexpr int kJoin = kWarps * 8 * kN * (D + 4) * 4;         // the warps' sums, in the ring's place at the end
    static constexpr int kSmem = kBytes > kJoin ? kBytes : kJoin;
    static_assert(kCtas * (kSmem + 1024 + kWarps * 8 * kN * 8) <= 228 * 1024, "the resident CTAs fit (1 KB of each is the system's)");
};

// The same with fp16 operands.
__device__ __forceinline__ void mma16816h(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four codes as two pairs of fp16 (their values before the scale, exactly).
template <int kKind>
__device__ __forceinline__ void half_pairs(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if constexpr (kKind == SP_CACHE_E4M3) {
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(lo), "=r"(hi) : "r"(w));
    } else {
        // 0x6400 + (8 bits) is 1024 + those bits; with the sign bit flipped they are the code + 128
        const uint32_t u = w ^ 0x80808080u;
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(__byte_perm(u, 0x64646464u, 0x4140)), "r"(0x64806480u));
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(__byte_perm(u, 0x64646464u, 0x4342)), "r"(0x64806480u));
    }
}

// A pair of bf16, times a power of two, as a pair of fp16.
__device__ __forceinline__ uint32_t half_of(uint32_t w, float scale) {
    const __half2 h = __floats2half2_rn(__uint_as_float(w << 16) * scale, __uint_as_float(w & 0xffff0000u) * scale);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Transpose of an 8 x 8 tile of 16-bit values: lane (n, q) gives row n's columns 2q, 2q + 1 and gets column n's rows 2q, 2q + 1.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// kN: tiles of 8 query rows (1 or 2).
template <int D, int kKind, int kN>
__global__ void __launch_bounds__(kThreads, kN == 1 ? 3 : 2) step_kernel(const __grid_constant__ SplitArgs p) {
    constexpr bool kSame = kKind == SP_CACHE_SAME;
    using R = Ring<D, kKind, kN>;
    constexpr int kSize = kSame ? 2 : 1;                    // bytes of an entry in the cache
    constexpr int kTok = R::kTok, kUnit = unit_tokens<D, kKind>(), kPitch = R::kPitch;
    constexpr int kT = kTok / 16;                           // tiles of 16 tokens
    constexpr int kE = 16 / kSize;                          // entries of a 16-byte piece
    constexpr int kJ = D / (4 * kE);                        // pieces of a K row that a lane reads
    constexpr int kEv = D / 8 < kE ? D / 8 : kE;            // entries of a V read
    constexpr int kC = D / (8 * kEv);                       // V reads of a token
    constexpr int kVB = kEv * kSize;                        // bytes of a V read
    constexpr int kO = kC * kEv / 2;                        // tiles of 16 entries of the sums
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float2 sm_ml[kWarps][8 * kN];
    float (*sm_o)[8 * kN][D + 4] = reinterpret_cast<float (*)[8 * kN][D + 4]>(smem);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = lane >> 2, q4 = lane & 3;
    uint8_t* ring = smem + warp * R::kStages * R::kStage;
    const uint32_t ring_at = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
    const sp_cache& c = p.a.cache;
    const sp_batch& bt = p.a.batch;
    bool bad_seq = false, bad_page = false;
    cudaTriggerProgrammaticLaunchCompletion();      // the joining kernel may line up: it waits for this one's end
    const int64_t U = total_units(p, kUnit, bad_seq);
    const Shares shares(U, p.P);
    int64_t u = shares.at(blockIdx.x);
    const int64_t u_end = shares.at(blockIdx.x + 1);
    int64_t begin = 0;
    int b = u < u_end ? find_unit(p, kUnit, u, begin) : 0;
    const float f = p.a.scale * 1.4426950408889634f;
    auto piece = [&](int j) { return kJ == 1 ? q4 : (j >> 1) * 8 + 2 * q4 + (j & 1); };

    while (u < u_end && b < p.a.batch.B) {         // (b: should the arrays be changed while the kernel runs)
        const Seq s = load_seq(bt, c.page, b);
        if (row_blocks(p, s) == 0) {
            ++b;
            continue;
        }
        const Span span = span_of(s, p.a.window, kUnit);
        const int64_t in_seq = u - begin;
        if (in_seq >= (int64_t)span.units * c.H_kv) {
            begin += (int64_t)span.units * c.H_kv;
            ++b;
            continue;
        }
        const int g = (int)divide(in_seq, span.units), from = (int)(in_seq - (int64_t)g * span.units);
        const int to = (int)min((int64_t)span.units, from + (u_end - u));
        const int rows = s.n * p.G;

        // this lane's token (lane % kTok) of a piece: its page, a piece ahead, and where its rows are
        const int32_t* table = bt.table + (int64_t)b * bt.table_stride;
        const int tok0 = span.first + warp * kTok + (lane & (kTok - 1));
        auto page_of = [&](int i) {
            const int tok = tok0 + i * kUnit;
            return i < to && tok < s.kv ? table[p.a.page_of(tok)] : 0;
        };
        // requests piece i of the run into its place in the ring
        auto request = [&](int i, int pg) {
            if (i < to) {
                const int tok = tok0 + i * kUnit;
                const uint32_t at = ring_at + ((i - from) % R::kStages) * R::kStage;
                int64_t mine = -1;
                if (tok < s.kv) {
                    if ((unsigned)pg < (unsigned)c.pages) mine = row_offset(c, pg, g, tok - p.a.page_of(tok) * c.page);
                    else bad_page = true;
                }
                if constexpr (!kSame) {
                    if (lane < kTok) {
                        const int64_t sc = mine >= 0 ? scale_offset(c, pg, g, tok - p.a.page_of(tok) * c.page) : 0;
                        copy_async<4>(at + R::kScales + lane * 8, c.k_scale + sc, mine >= 0);
                        copy_async<4>(at + R::kScales + lane * 8 + 4, c.v_scale + sc, mine >= 0);
                    }
                }
                constexpr int kLanes = R::kRow / 16, kAtOnce = 32 / kLanes;    // lanes of a row, rows of a request
#pragma unroll
                for (int t = 0; t < kTok; t += kAtOnce) {
                    const int row = t + lane / kLanes;
                    const int64_t w = __shfl_sync(0xffffffffu, mine, row);
                    const int64_t src = w * kSize + (lane % kLanes) * 16;
                    const uint32_t dst = at + row * kPitch + (lane % kLanes) * 16;
                    copy_async<16>(dst, static_cast<const char*>(c.k) + (w >= 0 ? src : 0), w >= 0);
                    copy_async<16>(dst + R::kV, static_cast<const char*>(c.v) + (w >= 0 ? src : 0), w >= 0);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        int page0 = page_of(from), page1 = page_of(from + 1);
#pragma unroll
        for (int i = 0; i < R::kStages - 1; ++i) {
            request(from + i, page0);
            page0 = page1;
            page1 = page_of(from + i + 2);
        }

        // query row n (and n + 8) as operands, and the tokens that rows 2q, 2q + 1 (+ 8) see
        uint32_t qb[kN][2 * kJ * (kE / 8)][2];
        float fq[kN][2];            // the logits' factor (8-bit caches: with the query rows' own)
        int last[kN][2], first[kN][2];
#pragma unroll
        for (int h = 0; h < kN; ++h) {
            const int r = n + 8 * h, t = r / p.G;
            const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.a.q.data) + (s.row0 + t) * p.a.q.stride_row +
                                       (g * p.G + r - t * p.G) * p.a.q.stride_head;
#pragma unroll
            for (int j = 0; j < kJ; ++j)
#pragma unroll
                for (int e = 0; e < kE / 8; ++e) {
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (r < rows) x = __ldg(reinterpret_cast<const uint4*>(src + piece(j) * kE + e * 8));
                    const int k = (j * (kE / 8) + e) * 2;
                    qb[h][k][0] = x.x; qb[h][k][1] = x.y;
                    qb[h][k + 1][0] = x.z; qb[h][k + 1][1] = x.w;
                }
            if constexpr (!kSame) {
                // the row's largest exponent; without a finite one (zeros, infinities, NaN) the row stays as it is
                uint32_t top = 0;
#pragma unroll
                for (int k = 0; k < 2 * kJ * (kE / 8); ++k)
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                        top = max(top, max(qb[h][k][y] & 0x7f80u, (qb[h][k][y] >> 16) & 0x7f80u));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int shift = top == 0 || top == 0x7f80u ? 0 : min(max(137 - (int)(top >> 7), -100), 100);
                const float up = __int_as_float((127 + shift) << 23), down = __int_as_float((127 - shift) << 23);
#pragma unroll
                for (int k = 0; k < 2 * kJ * (kE / 8); ++k)
#pragma unroll
                    for (int y = 0; y < 2; ++y) qb[h][k][y] = half_of(qb[h][k][y], up);
#pragma unroll
                for (int y = 0; y < 2; ++y) fq[h][y] = f * __shfl_sync(0xffffffffu, down, 4 * (2 * q4 + y));
            }
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int ry = 8 * h + 2 * q4 + y;
                last[h][y] = ry < rows ? s.kv - s.n + ry / p.G : -1;
                first[h][y] = p.a.window ? last[h][y] - p.a.window + 1 : 0;
            }
        }
        const int all_last = s.kv - s.n, all_first = p.a.window ? s.kv - p.a.window : 0;  // tokens that every row sees

        float o[kN][kO][4];
        float m[kN][2], z[kN][2];
#pragma unroll
        for (int h = 0; h < kN; ++h) {
            m[h][0] = m[h][1] = -INFINITY;
            z[h][0] = z[h][1] = 0.f;
#pragma unroll
            for (int i = 0; i < kO; ++i)
#pragma unroll
                for (int x = 0; x < 4; ++x) o[h][i][x] = 0.f;
        }

        for (int i = from; i < to; ++i) {
            const int base = span.first + warp * kTok + i * kUnit;
            request(i + R::kStages - 1, page0);
            page0 = page1;
            page1 = page_of(i + R::kStages + 1);
            asm volatile("cp.async.wait_group %0;" ::"n"(R::kStages - 1) : "memory");
            __syncwarp();
            const uint8_t* at = ring + ((i - from) % R::kStages) * R::kStage;
            // logits: x[h][t] holds tokens 16t + n (first two) and 16t + n + 8, rows 8h + 2q and 8h + 2q + 1
            float x[kN][kT][4];
#pragma unroll
            for (int t = 0; t < kT; ++t) {
#pragma unroll
                for (int h = 0; h < kN; ++h)
#pragma unroll
                    for (int y = 0; y < 4; ++y) x[h][t][y] = 0.f;
#pragma unroll
                for (int j = 0; j < kJ; ++j) {
                    const uint8_t* src = at + (16 * t + n) * kPitch + piece(j) * 16;
                    const Chunk<16> lo = read_chunk<16>(src), hi = read_chunk<16>(src + 8 * kPitch);
#pragma unroll
                    for (int k = 0; k < kE / 4; ++k) {
                        uint32_t a[4];
                        if constexpr (kSame) {
                            a[0] = lo.w[2 * k]; a[1] = hi.w[2 * k];
                            a[2] = lo.w[2 * k + 1]; a[3] = hi.w[2 * k + 1];
                        } else {
                            half_pairs<kKind>(lo.w[k], a[0], a[2]);
                            half_pairs<kKind>(hi.w[k], a[1], a[3]);
                        }
#pragma unroll
                        for (int h = 0; h < kN; ++h) {
                            const int kk = j * (kE / 4) + k;
                            if constexpr (kSame) mma16816(x[h][t], a, qb[h][kk][0], qb[h][kk][1]);
                            else mma16816h(x[h][t], a, qb[h][kk][0], qb[h][kk][1]);
                        }
                    }
                }
            }
            const bool masked = base + kTok - 1 > all_last || base < all_first;
            float vs[kSame ? 1 : kT][2];
            float top[kN][2];
#pragma unroll
            for (int h = 0; h < kN; ++h) top[h][0] = m[h][0], top[h][1] = m[h][1];
#pragma unroll
            for (int t = 0; t < kT; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int tl = 16 * t + 8 * e + n, tok = base + tl;
                    float2 sc = make_float2(1.f, 1.f);
                    if constexpr (!kSame) {
                        sc = *reinterpret_cast<const float2*>(at + R::kScales + tl * 8);
                        vs[t][e] = sc.y;
                    }
#pragma unroll
                    for (int h = 0; h < kN; ++h)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            float& v = x[h][t][2 * e + y];
                            v *= kSame ? f : fq[h][y] * sc.x;
                            if (masked && (tok > last[h][y] || tok < first[h][y])) v = -INFINITY;
                            top[h][y] = fmaxf(top[h][y], v);
                        }
                }
            // a NaN logit is not a maximum, but its weight is NaN and spreads to the row's sums
            bool grows = false;
#pragma unroll
            for (int h = 0; h < kN; ++h)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
#pragma unroll
                    for (int w = 4; w < 32; w <<= 1)
                        top[h][y] = fmaxf(top[h][y], __shfl_xor_sync(0xffffffffu, top[h][y], w));
                    grows |= top[h][y] > m[h][y];
                }
            if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
                for (int h = 0; h < kN; ++h)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const float a = top[h][y] == -INFINITY ? 1.f : ex2(m[h][y] - top[h][y]);
                        m[h][y] = top[h][y];
                        z[h][y] *= a;
#pragma unroll
                        for (int k = 0; k < kO; ++k) {
                            o[h][k][y] *= a;
                            o[h][k][2 + y] *= a;
                        }
                    }
            }
            uint32_t pb[kN][kT][2];
#pragma unroll
            for (int h = 0; h < kN; ++h) {
                const float r0 = m[h][0] == -INFINITY ? 0.f : m[h][0], r1 = m[h][1] == -INFINITY ? 0.f : m[h][1];
#pragma unroll
                for (int t = 0; t < kT; ++t)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float w0 = ex2(x[h][t][2 * e] - r0), w1 = ex2(x[h][t][2 * e + 1] - r1);
                        z[h][0] += w0;
                        z[h][1] += w1;
                        if constexpr (!kSame) {
                            if (masked) {       // a masked token's weight stays 0 whatever its scale is
                                w0 = w0 == 0.f ? 0.f : w0 * vs[t][e];
                                w1 = w1 == 0.f ? 0.f : w1 * vs[t][e];
                            } else {
                                w0 *= vs[t][e];
                                w1 *= vs[t][e];
                            }
                        }
                        pb[h][t][e] = transpose8(pack_bf16(w0, w1));
                    }
            }
#pragma unroll
            for (int t = 0; t < kT; ++t)
#pragma unroll
                for (int cc = 0; cc < kC; ++cc) {
                    Chunk<kVB> vr[4];           // tokens 2q, 2q + 1, 2q + 8, 2q + 9 of the tile
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        vr[y] = read_chunk<kVB>(at + R::kV + (16 * t + 8 * (y >> 1) + 2 * q4 + (y & 1)) * kPitch +
                                                (cc * 8 + n) * kVB);
#pragma unroll
                    for (int e = 0; e < kEv; e += 2) {
                        uint32_t a[4];              // entries e and e + 1 of tokens 2q, 2q + 1, then of 2q + 8, 2q + 9
#pragma unroll
                        for (int y = 0; y < 4; y += 2) {
                            const int w = e * kSize / 4;
                            const uint32_t t0 = vr[y].w[w], t1 = vr[y + 1].w[w];
                            if constexpr (kSame) {
                                a[y] = __byte_perm(t0, t1, 0x5410);
                                a[y + 1] = __byte_perm(t0, t1, 0x7632);
                            } else {
                                pairs_of<kKind, false>(__byte_perm(t0, t1, e & 2 ? 0x7632 : 0x5410), a[y], a[y + 1]);
                            }
                        }
#pragma unroll
                        for (int h = 0; h < kN; ++h) mma16816(o[h][(cc * kEv + e) / 2], a, pb[h][t][0], pb[h][t][1]);
                    }
                }
            __syncwarp();           // the piece has been read by all lanes: its place may be filled again
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();            // every warp is done with its ring, which takes the sums now

        // join the four warps: lane (n, q) holds entries cc * 8 kEv + n * kEv + e of rows 2q, 2q + 1
#pragma unroll
        for (int h = 0; h < kN; ++h)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int r = 8 * h + 2 * q4 + y;
#pragma unroll
                for (int w = 4; w < 32; w <<= 1) z[h][y] += __shfl_xor_sync(0xffffffffu, z[h][y], w);
                if (n == 0) sm_ml[warp][r] = make_float2(m[h][y], z[h][y]);
#pragma unroll
                for (int k = 0; k < kO; ++k) {
                    const int e = 2 * k, at = (e / kEv) * 8 * kEv + n * kEv + e % kEv;
                    sm_o[warp][r][at] = o[h][k][y];
                    sm_o[warp][r][at + 1] = o[h][k][2 + y];
                }
            }
        __syncthreads();
        const bool whole = from == 0 && to == span.units;
        for (int i = threadIdx.x; i < rows * (D / 8); i += kThreads) {
            const int r = i / (D / 8), e = (i % (D / 8)) * 8;
            float mm = -INFINITY, zz = 0.f, v[8] = {};
#pragma unroll
            for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sm_ml[w][r].x);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float2 ml = sm_ml[w][r];
                if (ml.x == -INFINITY && ml.y == 0.f) continue;         // saw no token of the row
                // without a maximum but with a sum: all its logits were NaN, and so is the sum
                const float a = ml.x == -INFINITY ? 1.f : ex2(ml.x - mm);
                zz += ml.y * a;
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] += sm_o[w][r][e + k] * a;
            }
            if (whole) {
                const float inv = zz == 0.f ? 0.f : 1.f / zz;
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = zz == 0.f ? 0.f : v[k] * inv;
                const int t = r / p.G, h = g * p.G + r - t * p.G;
                store8(static_cast<__nv_bfloat16*>(p.a.out.data) + (s.row0 + t) * p.a.out.stride_row +
                           h * p.a.out.stride_head + e, v);
                if (p.a.lse && e == 0)
                    p.a.lse[(s.row0 + t) * p.a.lse_stride_row + h * p.a.lse_stride_head] =
                        zz == 0.f ? -INFINITY : (mm + log2f(zz)) * 0.6931471805599453f;
            } else {
                const int64_t slot = ((int64_t)blockIdx.x * 2 + (from == 0 ? 1 : 0)) * kRows + r;
                store8(p.part_o + slot * D + e, v);
                if (e == 0) p.part_ml[slot] = make_float2(mm, zz);
            }
        }
        __syncthreads();
        u += to - from;
    }
    const int any = (__syncthreads_or(bad_seq) ? 1 : 0) | (__syncthreads_or(bad_page) ? 2 : 0);
    if (threadIdx.x == 0) p.err[blockIdx.x] = any;
}

constexpr int kJoinThreads = 256;

// Joins the parts of the pairs that were cut: block (i, r) takes row r of pair i = (sequence, KV head).  A thread
// has four entries of every kGroups-th part, several of them under way at once: a pair may be cut into hundreds.
// Block (0, 0) also gathers the status.
template <int D, int kKind>
__global__ void __launch_bounds__(kJoinThreads) step_join_kernel(const __grid_constant__ SplitArgs p) {
    constexpr int kUnit = unit_tokens<D, kKind>(), kLanes = D / 4, kGroups = kJoinThreads / kLanes;
    __shared__ float4 sm_o[kGroups][kLanes];
    __shared__ float2 sm_mz[kJoinThreads / 32];
    bool bad = false;
    cudaTriggerProgrammaticLaunchCompletion();      // of a mixed batch: the kernel of the other sequences may begin
    const int i = blockIdx.x, b = i / p.a.cache.H_kv, g = i - b * p.a.cache.H_kv, r = blockIdx.y;
    const Seq s = load_seq(p.a.batch, p.a.cache.page, b);
    const bool mine = row_blocks(p, s) > 0 && r < s.n * p.G;
    int64_t U = 0, begin = 0;
    if (mine) {
        for (int k = threadIdx.x & 31; k < p.a.batch.B; k += 32) {
            const int64_t units = seq_units(p, k, kUnit, bad);
            U += units;
            if (k < b) begin += units;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            U += __shfl_xor_sync(0xffffffffu, U, o);
            begin += __shfl_xor_sync(0xffffffffu, begin, o);
        }
    }
    U *= p.a.cache.H_kv;
    const int units = span_of(s, p.a.window, kUnit).units;
    begin = begin * p.a.cache.H_kv + (int64_t)g * units;
    const Shares shares(U, p.P);
    const int c0 = mine ? shares.of(begin) : 0, c1 = mine ? shares.of(begin + units - 1) : 0;
    cudaGridDependencySynchronize();        // the main kernel's partial sums
    if (i == 0 && r == 0) gather_status(p);
    if (c0 == c1) return;                   // not taken here, or written by the main kernel
    // the first part begins with the pair's first unit (slot 2 c0 + 1), the others do not (slot 2 k)
    const int lane = threadIdx.x % kLanes, grp = threadIdx.x / kLanes;
    float m = -INFINITY, z = 0.f;
    for (int k = c0 + threadIdx.x; k <= c1; k += kJoinThreads)
        m = fmaxf(m, p.part_ml[((int64_t)k * 2 + (k == c0)) * kRows + r].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((threadIdx.x & 31) == 0) sm_mz[threadIdx.x >> 5].x = m;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kJoinThreads / 32; ++k) m = fmaxf(m, sm_mz[k].x);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = c0 + grp; k <= c1; k += kGroups) {
        const int64_t slot = ((int64_t)k * 2 + (k == c0)) * kRows + r;
        const float2 ml = p.part_ml[slot];
        const float4 o = *reinterpret_cast<const float4*>(p.part_o + slot * D + lane * 4);
        // without a maximum the part has summed nothing, or NaN alone: it counts as it is
        const float a = ml.x == -INFINITY ? 1.f : ex2(ml.x - m);
        z += ml.y * a;
        v.x += o.x * a; v.y += o.y * a; v.z += o.z * a; v.w += o.w * a;
    }
    sm_o[grp][lane] = v;
    __shared__ float sm_z[kGroups];
    if (lane == 0) sm_z[grp] = z;
    __syncthreads();
    if (grp > 0) return;
    z = 0.f;
    v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
        const float4 o = sm_o[k][lane];
        z += sm_z[k];
        v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
    }
    const int t = r / p.G, h = g * p.G + r - t * p.G;
    const float inv = z == 0.f ? 0.f : 1.f / z;
    if (z == 0.f) v = make_float4(0.f, 0.f, 0.f, 0.f);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.a.out.data) + (s.row0 + t) * p.a.out.stride_row +
                              h * p.a.out.stride_head + lane * 4) =
        make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
    if (p.a.lse && lane == 0)
        p.a.lse[(s.row0 + t) * p.a.lse_stride_row + h * p.a.lse_stride_head] =
            z == 0.f ? -INFINITY : (m + log2f(z)) * 0.6931471805599453f;
}

int ctas(int rows) { return sm_count() * (rows <= 8 ? 3 : 2); }

template <int D, int kKind>
sp_status launch(const SplitArgs& p, cudaStream_t st) {
    const int smem = p.rows <= 8 ? Ring<D, kKind, 1>::kSmem : Ring<D, kKind, 2>::kSmem;
    void (*kern)(SplitArgs) = p.rows <= 8 ? step_kernel<D, kKind, 1> : step_kernel<D, kKind, 2>;
    SP_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
    kern<<<p.P, kThreads, smem, st>>>(p);
    SP_LAUNCH_CHECK();
    const int64_t rows = std::min<int64_t>(p.rows, (int64_t)p.a.batch.max_new * p.G);
    const dim3 grid((unsigned)p.a.batch.B * (unsigned)p.a.cache.H_kv, (unsigned)std::max<int64_t>(1, rows));
    return launch_early(step_join_kernel<D, kKind>, grid, kJoinThreads, (size_t)0, st, p);
}

template <int D>
sp_status launch_kind(const SplitArgs& p, cudaStream_t st) {
    switch (p.a.cache.kind) {
        case SP_CACHE_SAME: return launch<D, SP_CACHE_SAME>(p, st);
        case SP_CACHE_E4M3: return launch<D, SP_CACHE_E4M3>(p, st);
        default: return launch<D, SP_CACHE_INT8>(p, st);
    }
}

}  // namespace

bool attend_step_supported(const sp_cache& c) {
    if (c.dtype != SP_BF16 || (c.d != 64 && c.d != 128)) return false;
    // the 8-bit kinds are read 16 bytes at a time
    return c.kind == SP_CACHE_SAME ||
           ((reinterpret_cast<uintptr_t>(c.k) | reinterpret_cast<uintptr_t>(c.v) | (uintptr_t)c.stride_page |
             (uintptr_t)c.stride_head | (uintptr_t)c.stride_slot) % 16 == 0);
}

size_t attend_step_ws_bytes(const sp_cache& c) { return split_ws_bytes((size_t)ctas(8), c.d); }   // the larger grid's

sp_status attend_step_launch(const AttendProblem& a, void* ws, cudaStream_t st) {
    const int rows = (int64_t)a.batch.max_new * (a.H / a.cache.H_kv) <= 8 ? 8 : 16;
    const SplitArgs p = split_args(a, rows, false, ctas(rows), ws);
    return a.cache.d == 64 ? launch_kind<64>(p, st) : launch_kind<128>(p, st);
}

}  // namespace sp
