// The attention weight that cached tokens gather from few new tokens (decode steps): bf16, head dimension 64 or 128, sequences of at
// most 16 query rows per KV head.
//
//   w[i] = decay * w[i] + sum over the rows that see token i of 2^(f q . k_i - l),  f = scale * log2(e), l = lse * log2(e)
//
// The work is bound by the keys' bytes, each read once.  Each warp copies the rows of its next pieces (32 tokens), their
// scales and the weights that are there into its own ring in shared memory with cp.async while it works
// on the piece before, with no barrier with another warp.  The products are mma.sync, transposed (S^T = K Q^T): the tokens
// are the long side, the query rows (8 a tile) the narrow one, and a token's weights lie in four neighbouring lanes.  The order of
// the entries of a head is chosen such that a lane's operand registers are 16 consecutive bytes of a row.
// Codes of an 8-bit cache become fp16, one instruction a pair (the query rows too, each times a power of two that brings its
// largest entry near 2^10).
//
// A token's sum needs no other token, so the units of all (sequence, KV head) pairs are laid end to end and cut into equal runs, one
// per resident CTA, and nothing is joined.
// A step of 16 requests of 2K to 32K tokens (bf16, 4 KV heads of 64): 27.4 us, 78% of the copy rate; at heads of 128 94 us (88%), from
// e4m3 53 (83%).  The tensor-core kernel, with a tile of 128 columns for 4 rows, takes 68 us for the first of these.
#include "step_tiles.cuh"

namespace sp {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;

// The ring of a warp: kStages pieces, each its tokens' K rows, the places of their weights, what is there, and the scales.
template <int D, int kKind>
struct Ring {
    static constexpr int kRow = D * (kKind == SP_CACHE_SAME ? 2 : 1), kPitch = kRow + 16;
    static constexpr int kTok = 32, kUnit = kWarps * kTok;
    static constexpr int kAt = kTok * kPitch, kOld = kAt + 8 * kTok, kScale = kOld + 4 * kTok;
    static constexpr int kStage = kScale + (kKind == SP_CACHE_SAME ? 0 : 4 * kTok);
    static constexpr int kStages = 2;
    static constexpr int kSmem = kWarps * kStages * kStage;
    static constexpr int kMost = 227 * 1024 / (kSmem + 1024), kCtas = kMost < 4 ? kMost : 4;        // resident on an SM
};

struct StepArgs {
    WeightsProblem w;
    SplitArgs split;        // (of the division into runs alone)
};

// kN: tiles of 8 query rows (1 or 2).
template <int D, int kKind, int kN>
__global__ void __launch_bounds__(kThreads, (Ring<D, kKind>::kCtas)) weights_step_kernel(const __grid_constant__ StepArgs p) {
    constexpr bool kSame = kKind == SP_CACHE_SAME;
    using R = Ring<D, kKind>;
    constexpr int kSize = kSame ? 2 : 1;                    // bytes of an entry in the cache
    constexpr int kTok = R::kTok, kPitch = R::kPitch;
    constexpr int kE = 16 / kSize;                          // entries of a 16-byte piece
    constexpr int kJ = D / (4 * kE);                        // pieces of a K row that a lane reads
    extern __shared__ __align__(16) uint8_t smem[];
    const AttendProblem& a = p.w.a;
    const sp_cache& c = a.cache;
    const sp_batch& bt = a.batch;
    if (blockIdx.x == 0) {
        check_tokens(bt, c, a.window, false, p.split.hdr);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = lane >> 2, q4 = lane & 3, G = p.split.G;
    uint8_t* ring = smem + warp * R::kStages * R::kStage;
    const uint32_t ring_at = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
    bool bad = false;
    const int64_t U = total_units(p.split, R::kUnit, bad);
    const Shares shares(U, p.split.P);
    int64_t u = shares.at(blockIdx.x - 1);
    const int64_t u_end = shares.at(blockIdx.x);
    int64_t begin = 0;
    int b = u < u_end ? find_unit(p.split, R::kUnit, u, begin) : 0;
    const float f = a.scale * 1.4426950408889634f;
    auto piece = [&](int j) { return kJ == 1 ? q4 : (j >> 1) * 8 + 2 * q4 + (j & 1); };

    while (u < u_end && b < bt.B) {         // (b: should the arrays be changed while the kernel runs)
        const Seq s = load_seq(bt, c.page, b);
        if (row_blocks(p.split, s) == 0) {
            ++b;
            continue;
        }
        const Span span = span_of(s, a.window, R::kUnit);
        const int64_t in_seq = u - begin;
        if (in_seq >= (int64_t)span.units * c.H_kv) {
            begin += (int64_t)span.units * c.H_kv;
            ++b;
            continue;
        }
        const int g = (int)divide(in_seq, span.units), from = (int)(in_seq - (int64_t)g * span.units);
        const int to = (int)min((int64_t)span.units, from + (u_end - u)), rows = s.n * G, ctx = s.kv - s.n;

        // this lane's tokens of a piece (lane, and lane + 32 of 64): their pages, a piece ahead
        constexpr int kMine = kTok / 32;
        const int32_t* table = bt.table + (int64_t)b * bt.table_stride;
        const int tok0 = span.first + warp * kTok + lane;
        auto pages_of = [&](int i, int (&pg)[kMine]) {
#pragma unroll
            for (int y = 0; y < kMine; ++y) {
                const int tok = tok0 + i * R::kUnit + 32 * y;
                pg[y] = i < to && tok < s.kv ? __ldg(table + a.page_of(tok)) : -1;
            }
        };
        // requests piece i of the run into its place in the ring
        auto request = [&](int i, const int (&pg)[kMine]) {
            if (i < to) {
                const int st = (i - from) % R::kStages * R::kStage;
#pragma unroll
                for (int y = 0; y < kMine; ++y) {
                    const int tok = tok0 + i * R::kUnit + 32 * y, slot = tok - a.page_of(tok) * c.page;
                    const bool there = (unsigned)pg[y] < (unsigned)c.pages;
                    const int64_t mine = there ? row_offset(c, pg[y], g, slot) : -1, at = there ? scale_offset(c, pg[y], g, slot) : -1;
                    const uint32_t l = lane + 32 * y;
                    *reinterpret_cast<int64_t*>(ring + st + R::kAt + 8 * l) = at;
                    copy_async<4>(ring_at + st + R::kOld + 4 * l, p.w.weights + max(at, (int64_t)0), there && tok < ctx && p.w.decay != 0.f);
                    if constexpr (!kSame) copy_async<4>(ring_at + st + R::kScale + 4 * l, c.k_scale + max(at, (int64_t)0), there);
                    constexpr int kLanes = R::kRow / 16, kAtOnce = 32 / kLanes;    // lanes of a row, rows of a request
#pragma unroll
                    for (int t = 0; t < 32; t += kAtOnce) {
                        const int row = t + lane / kLanes;
                        const int64_t w = __shfl_sync(0xffffffffu, mine, row);
                        copy_async<16>(ring_at + st + (row + 32 * y) * kPitch + (lane % kLanes) * 16,
                                       static_cast<const char*>(c.k) + (w >= 0 ? w * kSize + (lane % kLanes) * 16 : 0), w >= 0);
                    }
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        int page0[kMine], page1[kMine];
        pages_of(from, page0);
        pages_of(from + 1, page1);
#pragma unroll
        for (int i = 0; i < R::kStages - 1; ++i) {
            request(from + i, page0);
#pragma unroll
            for (int y = 0; y < kMine; ++y) page0[y] = page1[y];
            pages_of(from + i + 2, page1);
        }

        // query row n (and n + 8) as operands; of rows 2q, 2q + 1 (+ 8) the normaliser and the tokens that they see
        uint32_t qb[kN][2 * kJ * (kE / 8)][2];
        float fq[kN][2], l[kN][2];  // the logits' factor (8-bit caches: with the query rows' own)
        int last[kN][2], first[kN][2];
#pragma unroll
        for (int h = 0; h < kN; ++h) {
            const int r = n + 8 * h, t = r / G;
            const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q.data) + (s.row0 + t) * a.q.stride_row +
                                       (g * G + r - t * G) * a.q.stride_head;
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
                    for (int y = 0; y < 2; ++y) top = max(top, max(qb[h][k][y] & 0x7f80u, (qb[h][k][y] >> 16) & 0x7f80u));
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
                const int ry = 8 * h + 2 * q4 + y, ty = ry / G;
                if constexpr (kSame) fq[h][y] = f;
                float x = -INFINITY;
                if (ry < rows) x = __ldg(a.lse + (s.row0 + ty) * a.lse_stride_row + (g * G + ry - ty * G) * a.lse_stride_head);
                // a row that saw no token has the sum 0, whose logarithm is -inf, and gives nothing
                l[h][y] = x * 1.4426950408889634f;
                last[h][y] = x != -INFINITY ? ctx + ty : -1;
                first[h][y] = a.window ? ctx + ty - a.window + 1 : 0;
            }
        }

        for (int i = from; i < to; ++i) {
            const int base = span.first + warp * kTok + i * R::kUnit;
            request(i + R::kStages - 1, page0);
#pragma unroll
            for (int y = 0; y < kMine; ++y) page0[y] = page1[y];
            pages_of(i + R::kStages + 1, page1);
            asm volatile("cp.async.wait_group %0;" ::"n"(R::kStages - 1) : "memory");
            __syncwarp();
            const uint8_t* at = ring + (i - from) % R::kStages * R::kStage;
#pragma unroll
            for (int t0 = 0; t0 < kTok; t0 += 32) {
                // logits: x[h][t] holds tokens 16t + n (first two) and 16t + n + 8, rows 8h + 2q and 8h + 2q + 1
                float sum[4];       // of tokens 8e + n
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    float x[kN][4];
#pragma unroll
                    for (int h = 0; h < kN; ++h)
#pragma unroll
                        for (int y = 0; y < 4; ++y) x[h][y] = 0.f;
#pragma unroll
                    for (int j = 0; j < kJ; ++j) {
                        const uint8_t* src = at + (t0 + 16 * t + n) * kPitch + piece(j) * 16;
                        const Chunk<16> lo = read_chunk<16>(src), hi = read_chunk<16>(src + 8 * kPitch);
#pragma unroll
                        for (int k = 0; k < kE / 4; ++k) {
                            uint32_t o[4];
                            if constexpr (kSame) {
                                o[0] = lo.w[2 * k]; o[1] = hi.w[2 * k];
                                o[2] = lo.w[2 * k + 1]; o[3] = hi.w[2 * k + 1];
                            } else {
                                half_pairs<kKind>(lo.w[k], o[0], o[2]);
                                half_pairs<kKind>(hi.w[k], o[1], o[3]);
                            }
#pragma unroll
                            for (int h = 0; h < kN; ++h) {
                                const int kk = j * (kE / 4) + k;
                                if constexpr (kSame) mma16816(x[h], o, qb[h][kk][0], qb[h][kk][1]);
                                else mma16816h(x[h], o, qb[h][kk][0], qb[h][kk][1]);
                            }
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int tl = t0 + 16 * t + 8 * e + n, tok = base + tl;
                        float sc = 1.f, w = 0.f;
                        if constexpr (!kSame) sc = *reinterpret_cast<const float*>(at + R::kScale + 4 * tl);
#pragma unroll
                        for (int h = 0; h < kN; ++h)
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const float v = ex2(x[h][2 * e + y] * (kSame ? fq[h][y] : fq[h][y] * sc) - l[h][y]);
                                w += tok <= last[h][y] && tok >= first[h][y] ? v : 0.f;
                            }
                        w += __shfl_xor_sync(0xffffffffu, w, 1);
                        sum[2 * t + e] = w + __shfl_xor_sync(0xffffffffu, w, 2);
                    }
                }
                // lane (n, q) writes token 8q + n
                const int tl = t0 + 8 * q4 + n;
                const int64_t place = *reinterpret_cast<const int64_t*>(at + R::kAt + 8 * tl);
                const float old = *reinterpret_cast<const float*>(at + R::kOld + 4 * tl);
                const float w = q4 & 2 ? (q4 & 1 ? sum[3] : sum[2]) : (q4 & 1 ? sum[1] : sum[0]);
                if (place >= 0) p.w.weights[place] = p.w.decay != 0.f ? w + p.w.decay * old : w;
            }
            __syncwarp();           // the piece has been read by all lanes: its place may be filled again
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncwarp();
        u += to - from;
    }
}

template <int D, int kKind>
sp_status launch(StepArgs& p, cudaStream_t st) {
    using R = Ring<D, kKind>;
    void (*kern)(StepArgs) = p.split.rows <= 8 ? weights_step_kernel<D, kKind, 1> : weights_step_kernel<D, kKind, 2>;
    SP_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, R::kSmem));
    p.split.P = sm_count() * R::kCtas - 1;      // and one that checks the arrays
    kern<<<p.split.P + 1, kThreads, R::kSmem, st>>>(p);
    SP_LAUNCH_CHECK();
    return SP_OK;
}

template <int D>
sp_status launch_kind(StepArgs& p, cudaStream_t st) {
    switch (p.w.a.cache.kind) {
        case SP_CACHE_SAME: return launch<D, SP_CACHE_SAME>(p, st);
        case SP_CACHE_E4M3: return launch<D, SP_CACHE_E4M3>(p, st);
        default: return launch<D, SP_CACHE_INT8>(p, st);
    }
}

}  // namespace

// (the cache as for attend_step_supported)
sp_status weights_step_launch(const WeightsProblem& w, void* ws, cudaStream_t st) {
    StepArgs p;
    p.w = w;
    p.split.a = w.a;
    p.split.G = w.a.H / w.a.cache.H_kv;
    p.split.rows = (int64_t)w.a.batch.max_new * p.split.G <= 8 ? 8 : 16;
    p.split.many = 0;
    p.split.hdr = static_cast<WsHeader*>(ws);
    p.split.err = nullptr;
    p.split.part_o = nullptr;
    p.split.part_ml = nullptr;
    return w.a.cache.d == 64 ? launch_kind<64>(p, st) : launch_kind<128>(p, st);
}

}  // namespace sp
