// What the attention kernels that cut the keys (attend_step.cu, attend_general.cu)
// share: an item is a block of query rows of one sequence and KV head; the items'
// units of keys are laid end to end (sequence, KV head, row block, unit) and each
// CTA takes an equal run of them.  Each CTA works this out from the
// batch's device arrays by itself.  An item that is cut leaves one part per
// CTA in the workspace: slot 2 c + 1 if the part begins with the item's first
// unit, 2 c otherwise (a CTA has at most one of each).
#pragma once

#include "paged.cuh"

namespace sp {
namespace {

constexpr int kRows = 16;          // rows of a slot of partial sums

struct SplitArgs {
    AttendProblem a;
    int G;
    int rows;               // query rows of an item
    int many;               // 0: sequences of more rows are left to another kernel; 1: they are several items
    int P;                  // CTAs of the main kernel
    WsHeader* hdr;
    int* err;               // [P] what each CTA found wrong (0: nothing)
    float* part_o;          // [P][2][kRows][d]
    float2* part_ml;        // [P][2][kRows] maximum and sum
};

inline size_t split_ws_bytes(size_t P, int d) {
    Carve w;
    w.take(P * sizeof(int));
    w.take(P * 2 * kRows * d * sizeof(float));
    w.take(P * 2 * kRows * sizeof(float2));
    return w.off;
}

inline SplitArgs split_args(const AttendProblem& a, int rows, bool many, int P, void* ws) {
    SplitArgs p;
    p.a = a;
    p.G = a.H / a.cache.H_kv;
    p.rows = rows;
    p.many = many;
    p.P = P;
    Carve w;
    char* base = static_cast<char*>(ws);
    p.hdr = reinterpret_cast<WsHeader*>(base);
    p.err = reinterpret_cast<int*>(base + w.take((size_t)P * sizeof(int)));
    p.part_o = reinterpret_cast<float*>(base + w.take((size_t)P * 2 * kRows * a.cache.d * sizeof(float)));
    p.part_ml = reinterpret_cast<float2*>(base + w.take((size_t)P * 2 * kRows * sizeof(float2)));
    return p;
}

// Tokens [first, kv) that the rows of a sequence see, and their units.
struct Span {
    int first, units;
};
__device__ __forceinline__ Span span_of(const Seq& s, int window, int unit) {
    Span r;
    r.first = first_seen(s, window);
    r.units = max(1, (s.kv - r.first + unit - 1) / unit);
    return r;
}

// Row blocks of a sequence for one KV head (0: not taken here).
__device__ __forceinline__ int row_blocks(const SplitArgs& p, const Seq& s) {
    const int64_t rows = (int64_t)s.n * p.G;
    if (!p.many) return rows > 0 && rows <= p.rows ? 1 : 0;
    return (int)((rows + p.rows - 1) / p.rows);
}

// Units of sequence i's items for one KV head.
__device__ __forceinline__ int64_t seq_units(const SplitArgs& p, int i, int unit, bool& bad) {
    const Seq s = load_seq(p.a.batch, p.a.cache.page, i);
    if (!s.ok) bad = true;
    return (int64_t)row_blocks(p, s) * span_of(s, p.a.window, unit).units;
}

// Sum over all sequences, by one warp.
__device__ __forceinline__ int64_t total_units(const SplitArgs& p, int unit, bool& bad) {
    int64_t sum = 0;
    for (int i = threadIdx.x & 31; i < p.a.batch.B; i += 32) sum += seq_units(p, i, unit, bad);
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    bad = __any_sync(0xffffffffu, bad);
    return sum * p.a.cache.H_kv;
}

// The sequence whose units hold unit u (< total), and the unit at which it
// begins, by one warp.
__device__ __forceinline__ int find_unit(const SplitArgs& p, int unit, int64_t u, int64_t& begin) {
    int64_t base = 0;
    const int lane = threadIdx.x & 31;
    bool bad = false;
    for (int i0 = 0; i0 < p.a.batch.B; i0 += 32) {
        const int64_t mine = i0 + lane < p.a.batch.B ? seq_units(p, i0 + lane, unit, bad) * p.a.cache.H_kv : 0;
        int64_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        const unsigned past = __ballot_sync(0xffffffffu, base + incl > u);
        if (past) {
            const int l = __ffs(past) - 1;
            begin = base + __shfl_sync(0xffffffffu, incl - mine, l);
            return i0 + l;
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
    }
    begin = base;
    return p.a.batch.B;
}

// Gathers what the CTAs of the main kernel found wrong into the status; every thread of one block calls it.
__device__ __forceinline__ void gather_status(const SplitArgs& p) {
    int one = 0, two = 0;
    for (int k = threadIdx.x; k < p.P; k += blockDim.x) {
        one |= p.err[k] & 1;
        two |= p.err[k] & 2;
    }
    const int code = (__syncthreads_or(one) ? 1 : 0) | (__syncthreads_or(two) ? 2 : 0);
    if (threadIdx.x == 0) {
        p.hdr->status = code ? SP_EDEVICE : SP_OK;
        p.hdr->where = code;            // 1: impossible lengths or offsets, 2: a page index out of range
    }
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace
}  // namespace sp
