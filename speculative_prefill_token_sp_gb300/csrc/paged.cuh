// Device helpers shared by the operators on the paged cache (cache.cu, attend_*.cu).
#pragma once

#include "sp_common.cuh"

#include <cuda_fp8.h>
#include <math.h>

namespace sp {

// One sequence of a batch as the device arrays give it.
struct Seq {
    int64_t row0;   // first row of its new tokens
    int n;          // new tokens (0 for a sequence that is left out)
    int kv;         // tokens in the cache, the new ones included
    bool ok;        // false: the arrays say something impossible
};

__device__ __forceinline__ Seq load_seq(const sp_batch& b, int page, int i) {
    const int64_t lo = b.cu_new[i], hi = b.cu_new[i + 1], kv = b.kv_len[i];
    Seq s;
    s.ok = lo >= 0 && hi >= lo && hi <= b.T && hi - lo <= b.max_new && kv >= 0 &&
           kv <= (int64_t)b.table_width * page && kv <= (int64_t)1 << 30;
    s.row0 = lo;
    s.n = s.ok ? (int)(hi - lo) : 0;
    s.kv = s.ok ? (int)kv : 0;
    return s;
}

// The first token that a row of the sequence sees.
__device__ __forceinline__ int first_seen(const Seq& s, int window) {
    return window ? (int)max((int64_t)0, (int64_t)s.kv - s.n - window + 1) : 0;
}

// U units laid end to end, in `parts` runs whose lengths differ by one at most: run c has the units [at(c), at(c + 1)).  One
// division makes it (32 bits wide where that suffices: 64-bit divisions cost hundreds of cycles), one finds the run of a unit.
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
    return ((uint64_t)a | (uint64_t)b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}
struct Shares {
    int64_t each;       // units of a run; the first `extra` have one more
    int parts, extra;
    __device__ __forceinline__ Shares(int64_t U, int most) {
        parts = (int)max((int64_t)1, min((int64_t)most, U));        // so that every run has a unit, unless there is none at all
        each = divide(U, parts);
        extra = (int)(U - each * parts);
    }
    __device__ __forceinline__ int64_t at(int c) const { return (int64_t)min(c, parts) * each + min(c, extra); }
    __device__ __forceinline__ int of(int64_t u) const {
        const int64_t big = (each + 1) * extra;
        return (int)(u < big ? divide(u, each + 1) : extra + divide(u - big, each));
    }
};

// The sequence that row r is a new token of: the last b with cu_new[b] <= r
// (so empty sequences are passed over), or -1.
__device__ __forceinline__ int seq_of_row(const sp_batch& b, int64_t r) {
    int lo = 0, hi = b.B;       // answer + 1 is in [lo, hi]
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (b.cu_new[mid - 1] <= r) lo = mid;
        else hi = mid - 1;
    }
    return lo - 1;
}

// Place of row r of the batch in the cache: (page, slot), or page = -1 if it
// has none (not a token of the batch, a negative place, or a bad page index).
struct Place {
    int page, slot;
    bool token;     // the row is a token of a valid sequence
};

__device__ __forceinline__ Place place_of_row(const sp_batch& b, const sp_cache& c, int64_t r) {
    Place p{-1, 0, false};
    const int i = seq_of_row(b, r);
    if (i < 0) return p;
    const Seq s = load_seq(b, c.page, i);
    const int64_t t = r - s.row0;
    if (t >= s.n) return p;             // also every row of a sequence that is left out (n = 0)
    p.token = true;
    const int64_t at = (int64_t)s.kv - s.n + t;
    if (at < 0) return p;
    const unsigned q = (unsigned)at / (unsigned)c.page;
    p.slot = (int)((unsigned)at - q * (unsigned)c.page);
    const int pg = b.table[(int64_t)i * b.table_stride + q];
    if (pg >= 0 && pg < c.pages) p.page = pg;
    return p;
}

__device__ __forceinline__ int64_t row_offset(const sp_cache& c, int page, int head, int slot) {
    return page * c.stride_page + head * c.stride_head + slot * c.stride_slot;
}
__device__ __forceinline__ int64_t scale_offset(const sp_cache& c, int page, int head, int slot) {
    return ((int64_t)page * c.H_kv + head) * c.page + slot;
}

// Eight consecutive entries as fp32.
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {       // a bf16 is the upper half of an fp32
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
    unpack8(*reinterpret_cast<const uint4*>(p), x);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                                              pack_bf16(x[6], x[7]));
}

// Eight codes as the values they stand for before the scale.
template <int kKind>
__device__ __forceinline__ void decode8(uint2 u, float (&x)[8]) {
    const uint32_t w[2] = {u.x, u.y};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint8_t c = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
        if (kKind == SP_CACHE_INT8) x[i] = (float)(int8_t)c;
        else x[i] = __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
    }
}

// The four codes of a word as two pairs of bf16 (their values before the scale, exactly): codes 0, 1 and 2, 3 (kNext), or codes 0, 2
// and 1, 3.  The integer pipe bounds what uses this, so it has few masks and permutes, and the rest is left to the FMA pipe.
template <int kKind, bool kNext>
__device__ __forceinline__ void pairs_of(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if constexpr (kKind == SP_CACHE_E4M3) {
        // exponent and mantissa moved to bf16's place mean the value * 2^-120 (biases 7 and 127), also
        // for e4m3's subnormals; the product with 2^120 is exact.  0x7f is NaN in e4m3, never written, and 480 here
        if (kNext) w = __byte_perm(w, 0, 0x3120);
        const uint32_t b0 = ((w << 4) & 0x07f007f0u) | ((w << 8) & 0x80008000u), b1 = ((w >> 4) & 0x07f007f0u) | (w & 0x80008000u);
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(lo) : "r"(b0), "r"(0x7b807b80u));
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(hi) : "r"(b1), "r"(0x7b807b80u));
    } else {
        // With the sign bit flipped a code is u = code + 128, and y = 0x4300 + u as a bf16 is 128 + u below u = 128 and 2 u from
        // there on.  So the code is y - 256 below, and the half of that above: y - 256 - max(y / 2 - 128, 0).
        auto value = [](uint32_t y) {
            uint32_t t, r;
            asm("fma.rn.relu.bf16x2 %0, %1, %2, %3;" : "=r"(t) : "r"(y), "r"(0x3f003f00u), "r"(0xc300c300u));
            asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(y), "r"(0x43804380u));
            asm("sub.rn.bf16x2 %0, %0, %1;" : "+r"(r) : "r"(t));
            return r;
        };
        w ^= 0x80808080u;
        lo = value(__byte_perm(w, 0x43434343u, kNext ? 0x4140 : 0x4240));
        hi = value(__byte_perm(w, 0x43434343u, kNext ? 0x4342 : 0x4341));
    }
}

// The scale of a row whose largest magnitude is `top` (NaN or infinite if an
// entry is): 2^k with the smallest k >= -100 such that top / 2^k is at most
// the largest code.  448 = 0.875 * 2^9 and 127 = 0.9921875 * 2^7: with top = m
// * 2^e, 0.5 <= m < 1, k is e - 9 (e - 7), one more if m is above that.
template <int kKind>
__device__ __forceinline__ float row_scale(float top) {
    if (!(top < INFINITY)) return __int_as_float(0x7fffffff);
    if (top == 0.f) return 1.f;
    constexpr float kM = kKind == SP_CACHE_INT8 ? 0.9921875f : 0.875f;
    constexpr int kE = kKind == SP_CACHE_INT8 ? 7 : 9;
    int e;
    const float m = frexpf(top, &e);
    const int k = max(-100, e - kE + (m > kM ? 1 : 0));
    return __int_as_float((k + 127) << 23);
}

// max that keeps a NaN of either side
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// Eight values as codes; inv = 1 / scale, exact as the scale is a power of two.
template <int kKind>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inv) {
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        uint32_t two;
        if (kKind == SP_CACHE_INT8) {
            two = (uint32_t)(uint8_t)(int8_t)__float2int_rn(x[i] * inv) |
                  (uint32_t)(uint8_t)(int8_t)__float2int_rn(x[i + 1] * inv) << 8;
        } else {
            two = __nv_cvt_float2_to_fp8x2(make_float2(x[i] * inv, x[i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
        }
        w[i >> 2] |= two << (8 * (i & 3));
    }
    return make_uint2(w[0], w[1]);
}

// One block's check of everything the batch's device arrays say about the new
// tokens of each sequence.  Writes the status: the only writer of the call.
__device__ __forceinline__ void check_batch(const sp_batch& b, const sp_cache& c, WsHeader* hdr) {
    __shared__ int bad;
    if (threadIdx.x == 0) bad = 0;
    __syncthreads();
    int mine = 0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    for (int i = warp; i < b.B; i += warps) {
        const Seq s = load_seq(b, c.page, i);
        if (!s.ok) mine = 1;
        if (s.n == 0 || s.kv == 0) continue;
        const int first = max(0, s.kv - s.n) / c.page, last = (s.kv - 1) / c.page;
        for (int q = first + lane; q <= last; q += 32) {
            const int pg = b.table[(int64_t)i * b.table_stride + q];
            if (pg < 0 || pg >= c.pages) mine = 2;
        }
    }
    if (mine) atomicMax(&bad, mine);
    __syncthreads();
    if (threadIdx.x == 0) {
        hdr->status = bad ? SP_EDEVICE : SP_OK;
        hdr->where = bad;       // 1: impossible lengths or offsets, 2: a page index out of range
    }
}

// The same for calls that go over all tokens that a sequence's new ones see (with `idle`: of every sequence, also without new ones).
__device__ __forceinline__ void check_tokens(const sp_batch& b, const sp_cache& c, int window, bool idle, WsHeader* hdr) {
    __shared__ int bad;
    if (threadIdx.x == 0) bad = 0;
    __syncthreads();
    int mine = 0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    for (int i = warp; i < b.B; i += warps) {
        const Seq s = load_seq(b, c.page, i);
        if (!s.ok) mine = max(mine, 1);
        if (s.kv == 0 || (s.n == 0 && !idle)) continue;
        for (int q = first_seen(s, window) / c.page + lane; q <= (s.kv - 1) / c.page; q += 32) {
            const int pg = b.table[(int64_t)i * b.table_stride + q];
            if (pg < 0 || pg >= c.pages) mine = 2;
        }
    }
    if (mine) atomicMax(&bad, mine);
    __syncthreads();
    if (threadIdx.x == 0) {
        hdr->status = bad ? SP_EDEVICE : SP_OK;
        hdr->where = bad;
    }
}

// Argument checks shared by the entry points (defined in abi_paged.cu).
sp_status check_cache(const char* fn, const sp_cache* c);
sp_status check_batch_args(const char* fn, const sp_batch* b);

// SMs of the current device (defined in abi_paged.cu).
int sm_count();

// Launch that may begin while the kernel before it ends (the kernel waits for that by itself).
template <typename... A>
sp_status launch_early(void (*kern)(A...), dim3 grid, int threads, size_t smem, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    SP_CUDA_TRY(cudaLaunchKernelEx(&cfg, kern, args...));
    SP_LAUNCH_CHECK();
    return SP_OK;
}

struct AttendProblem {
    sp_rows q, out;
    sp_cache cache;
    sp_batch batch;
    int H;
    float scale;
    int window;             // 0: none
    int page_shift;         // log2 of the page, or -1: it is not a power of two
    __device__ __forceinline__ int page_of(int tok) const {
        return page_shift >= 0 ? tok >> page_shift : (int)((unsigned)tok / (unsigned)cache.page);
    }
    float* lse;             // may be null
    int64_t lse_stride_row, lse_stride_head;
    const uint32_t* seen;   // sp_attend_tree: the new tokens that a row sees, as bits; null: those up to its own
    int64_t seen_stride;
};

// The attention weight that cached tokens gather (weights_*.cu): a.q, a.lse (read), and the tokens' weights [pages, H_kv, page].
struct WeightsProblem {
    AttendProblem a;
    float decay;
    float* weights;
};

// The lowest n bits (none if n < 0).
__device__ __forceinline__ uint32_t low_bits(int n) {
    uint32_t r;
    asm("bmsk.clamp.b32 %0, 0, %1;" : "=r"(r) : "r"(max(n, 0)));
    return r;
}

// Of drafted tokens: word k of the new tokens that new token t of the sequence sees (0 behind the last one).
__device__ __forceinline__ uint32_t seen_word(const AttendProblem& a, const Seq& s, int t, int k) {
    if (k < 0 || 32 * k >= s.n) return 0;
    return __ldg(a.seen + (s.row0 + t) * a.seen_stride + k) & low_bits(s.n - 32 * k);
}

// And its place: behind the cached tokens, and as many of the new ones as it sees, itself among them.
__device__ __forceinline__ int place_of_drafted(const AttendProblem& a, const Seq& s, int t) {
    int sees = 0;
    for (int k = 0; 32 * k < s.n; ++k) sees += __popc(seen_word(a, s, t, k));
    return s.kv - s.n + max(sees, 1) - 1;
}

}  // namespace sp
