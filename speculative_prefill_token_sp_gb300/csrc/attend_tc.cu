// Attention of chunks of new tokens over the paged cache on tensor cores:
// tcgen05.mma + TMA + TMEM.  bf16, head dimension 64 or 128.
//
// Query rows are packed by KV head: row r of a tile is token r / G, head r % G
// of the group, so the keys and values of a KV head are read once for all its
// query heads.  An item is 2 tiles of 128 rows (A and B) of one sequence and KV
// head against tiles of 128 keys; one pass over the keys, with a maximum m that
// stays near each row's and the sum of its softmax (base 2):
//   S = Q K^T (TMEM)  ->  P = 2^(f S - m) (registers, back to TMEM as bf16)  ->  O += P V (TMEM)
//
// The three steps of one tile depend on each other, so the two row tiles take
// turns: while the softmax of A runs, the tensor cores do P V and the next S of
// B.  Per 256 x 128 logits the MMAs take 2048 cycles (d = 128) and each
// softmax half as long for its 128 x 128 logits, from one hand-over to the next:
// one thread a row, so that maximum and sum need no exchange between threads.  (Two a row were slower, 1.55 ms
// for 1.40 ms, a chunk of 4096 over 32768: the exponentials are bound by their unit, and the registers did not suffice.)
// The first 96 weights of a row are handed over before the last 32.  O stays in TMEM.  m
// begins as the maximum of the first tile that the row sees; where a tile's weights sum to
// more than 2^8, m grows by that sum's logarithm before the next tile, and O is scaled then.  A tile
// whose weights come to more than about 2^24 is done again by its true maximum.  P is thus at
// most about 2^24, and bf16 has the same precision there.  Its rounding to bf16 (the tensor cores'
// operand type; z sums the weights unrounded) is off by 0.0016 of a weight in root mean square, and so is the
// output by as much from it, and by as much again from its own rounding: 0.0023 in all, 0.0021 to 0.0026 measured.
//
// Warp roles of a CTA (one per SM):
//  * four warps each for tiles A and B: softmax, the scaling of O, and the output;
//  * eight warps, for an 8-bit cache only: convert its rows to bf16 into the
//    shared-memory tiles;
//  * two warps issue the MMAs of A and B: a thread that issues them is held up
//    until the tensor cores are nearly done with them, so what it does in between
//    (some 1000 cycles a tile for one thread) is only hidden by the other's MMAs.
//    They hand a turn to and fro, or the tiles' MMAs would mix and both tiles'
//    softmax fall into the same time (chunk of 4096 over 32768: 1.80 ms);
//  * one makes the TMA loads of K and V tiles, page by page (boxes of the largest
//    power of two that divides the page), and of Q;
//  * one zeroes what a V tile holds of slots without a token, as 0 * NaN
//    in P V would be NaN.  (K needs none: masked logits are replaced.)
//
// The items of the call, longest part first within a sequence, are laid end to
// end, and each CTA takes an equal run of key tiles, so that the SMs end
// together whatever the lengths.  An item that is cut leaves its sums in the
// workspace and a joining kernel adds them up in a fixed order.
//
// A chunk of 4096 over 32768 (bf16, 32 query heads on 8 of 128) takes 1.13 ms,
// 1.83 PFLOP/s or 95% of the rate of a large library product; in a long loop the board's
// power limit makes it 1.29 to 1.37 ms.  Seven requests of 192 to 650 new tokens with
// a window of 4096 take 136 us from an int8 cache, 111 us from bf16: 51 key tiles a CTA
// of 1.45 us (int8: about 2, the conversion's warps share the schedulers with
// the softmax's), 10 us until the first logits, 5 us more for each of an SM's two
// or three items, 5 us of step kernels without work and as much of joining.
#include "paged.cuh"
#include "tc_ptx.cuh"

#include <string.h>

#include <algorithm>
#include <type_traits>

namespace sp {
namespace {

// Warps of a CTA by role: eight of softmax, for an 8-bit cache eight that convert, and the four single ones.  setmaxnreg shares
// out the registers that the block was launched with: 384 threads of 168, or 640 of 96.
template <int kKind>
struct Roles {
    static constexpr bool kSame = kKind == SP_CACHE_SAME;
    static constexpr int kSoftmax = 8, kMma = kSame ? 8 : 16, kTma = kMma + 2, kClean = kMma + 3;
    static constexpr int kThreads = 32 * (kMma + 4);
    static constexpr int kSoftmaxRegs = kSame ? 216 : 136, kConvertRegs = 80, kSingleRegs = kSame ? 72 : 48;
    static_assert(kSoftmax * kSoftmaxRegs + (kMma - kSoftmax) * kConvertRegs + 4 * kSingleRegs <= (kMma + 4) * (kSame ? 168 : 96),
                  "the roles' registers");
};
constexpr int kRowsItem = 256;
constexpr int kKeys = 128;              // keys of a tile
constexpr int kSmem = 227 * 1024;
// What an item costs beside its key tiles (queries, first maximum, output), in key tiles: it counts so many more in the division
// of the work.  Seven requests of 192 to 650 new tokens, 3 to 34 tiles an item, take 111, 111, 113 us with 2, 3, 4 (bf16) and
// 135, 135, 138 us (int8); before the items' ends were made faster they took 162, 142, 132, 128, 126 us with 0 to 4 (bf16).
constexpr int kExtra = 3;
constexpr int kMaxSeqs = 16384;         // their item counts are laid out in the (still empty) ring of key tiles

struct Item {
    int b, t0;              // sequence, first new token
    int lo, tiles;          // first key tile, number of key tiles (at least 1)
};

// What the joining kernel has to know of CTA c: whether its run begins inside an item that no CTA before has cut.
struct Cut {
    int first, g, t0, n;    // KV head, first new token, new tokens of the sequence
    int64_t row0;           // first row of the sequence
    int last;               // the CTA of the item's last tile
};

struct TcArgs {
    AttendProblem a;
    int G, tpt;             // query heads of a KV head; new tokens of a row tile
    int min_rows;           // sequences with at most this many rows per KV head are left to the step kernel
    int P;                  // CTAs
    int box;                // rows of a TMA box
    WsHeader* hdr;
    int* err;               // [P] what each CTA found wrong: bits 1, 2 as in SplitArgs, 4 a wait that gave up (in bits 8-15)
    Cut* cuts;              // [P]
    float* part_o;          // [P][2][d / 4][256][4]
    float2* part_ml;        // [P][2][256]
};

struct Maps {
    CUtensorMap q, k, v;
};

__device__ __forceinline__ bool is_tc(const TcArgs& p, const Seq& s) {
    return s.n > 0 && (int64_t)s.n * p.G > p.min_rows;
}

__device__ __forceinline__ int blocks_of(const TcArgs& p, const Seq& s) {
    return is_tc(p, s) ? (s.n + 2 * p.tpt - 1) / (2 * p.tpt) : 0;
}

__device__ __forceinline__ Item item_of(const TcArgs& p, const Seq& s, int b, int qt) {
    Item it;
    it.b = b;
    it.t0 = qt * 2 * p.tpt;
    const int last = min(s.n, it.t0 + 2 * p.tpt) - 1 + s.kv - s.n;      // place of the item's last token
    const int first = p.a.window ? max(0, s.kv - s.n + it.t0 - p.a.window + 1) : 0;
    it.lo = first / kKeys;
    it.tiles = last < 0 ? 1 : last / kKeys + 1 - it.lo;
    return it;
}

// Sum over the block's threads before this one's; `total` over all of them.
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t* warp_sums, int64_t& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int64_t mine = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    int64_t w = lane < warps ? warp_sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
    }
    total = __shfl_sync(0xffffffffu, w, 31);
    const int64_t before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
    __syncthreads();
    return x - mine + (warp ? before : 0);
}

// A CTA's run of key tiles, item by item: KV head, sequence, row block (from the last tokens, which see most keys, to the first),
// key tile.  Every role walks it by itself; all lanes of a warp together.
struct Segment {
    Item it;
    Seq s;
    int g, from, to;        // KV head; tiles [from, to) of the item, counted from its last keys to its first
};

struct Walk {
    int left, g, b, qt, from;       // units (tiles and kExtra an item) left; the next item and its first unit

    __device__ __forceinline__ bool next(const TcArgs& p, Segment& o) {
        while (left > 0) {
            o.s = load_seq(p.a.batch, p.a.cache.page, b);
            o.it = item_of(p, o.s, b, qt);
            o.g = g;
            o.from = from;
            const int to = min(o.it.tiles + kExtra, from + left);
            o.to = min(o.it.tiles, to);
            left -= to - from;
            from = 0;
            if (left > 0 && --qt < 0) next_seq(p);
            if (o.from < o.to) return true;         // else the run begins behind the item's last tile
        }
        return false;
    }
    // the next sequence that has rows here (there is one, as tiles are left), 32 of them at a time
    __device__ __forceinline__ void next_seq(const TcArgs& p) {
        const int lane = threadIdx.x & 31;
        for (int first = b + 1, rounds = 0;; first += 32) {
            if (first >= p.a.batch.B) {
                first = 0;
                ++g;
                if (++rounds > 1) {         // the arrays were changed while the kernel ran
                    left = 0;
                    return;
                }
            }
            int n = 0;
            if (first + lane < p.a.batch.B) n = blocks_of(p, load_seq(p.a.batch, p.a.cache.page, first + lane));
            const unsigned some = __ballot_sync(0xffffffffu, n > 0);
            if (some) {
                const int l = __ffs(some) - 1;
                b = first + l;
                qt = __shfl_sync(0xffffffffu, n, l) - 1;
                return;
            }
        }
    }
};

// Where this CTA's run begins, worked out by all its threads: the row blocks of every sequence are counted, then each thread adds
// up the key tiles of an equal share of them, and the one whose share holds the first tile finds it.  `starts` [B + 1] and `sums`
// [32] are scratch in shared memory.
__device__ __forceinline__ void plan(const TcArgs& p, int* starts, int64_t* sums, Walk* out, int* bad) {
    const int t = threadIdx.x, threads = blockDim.x, B = p.a.batch.B;
    int64_t total, base = 0;
    for (int b0 = 0; b0 < B; b0 += threads) {
        int n = 0;
        if (b0 + t < B) {
            const Seq s = load_seq(p.a.batch, p.a.cache.page, b0 + t);
            if (!s.ok) bad[0] = 1;
            n = blocks_of(p, s);
        }
        const int64_t before = block_scan(n, sums, total);
        if (b0 + t < B) starts[b0 + t] = (int)(base + before);
        base += total;
    }
    if (t == 0) {
        starts[B] = (int)base;
        *out = Walk{0, 0, 0, 0, 0};
        p.cuts[blockIdx.x].first = 0;
    }
    __syncthreads();
    const int items = (int)base, share = (items + threads - 1) / threads, j0 = min(items, t * share), j1 = min(items, j0 + share);
    int b = 0, hi = B - 1;                  // the sequence of item j0: the last one that starts at or before it
    while (b < hi) {
        const int mid = (b + hi + 1) >> 1;
        if (starts[mid] <= j0) b = mid;
        else hi = mid - 1;
    }
    // visits the share's items until `stop` of their tiles are passed; returns the tiles
    int seq = b, qt = 0;
    auto visit = [&](int64_t stop) {
        int64_t sum = 0;
        seq = b;
        for (int j = j0; j < j1; ++j) {
            while (j >= starts[seq + 1]) ++seq;
            qt = starts[seq + 1] - 1 - j;
            const int tiles = item_of(p, load_seq(p.a.batch, p.a.cache.page, seq), seq, qt).tiles + kExtra;
            if (sum + tiles > stop) break;
            sum += tiles;
        }
        return sum;
    };
    const int64_t mine = visit(INT64_MAX), before = block_scan(mine, sums, total);
    const int64_t U = total * p.a.cache.H_kv;
    const Shares shares(U, p.P);
    const int c = blockIdx.x;
    const int64_t u = shares.at(c), left = shares.at(c + 1) - u;
    if (left > 0) {
        const int g = (int)divide(u, total);
        const int64_t r = u - g * total;
        if (before <= r && r < before + mine) {
            const int from = (int)(r - before - visit(r - before));
            *out = Walk{(int)left, g, seq, qt, from};
            const Seq s = load_seq(p.a.batch, p.a.cache.page, seq);
            const Item it = item_of(p, s, seq, qt);
            if (from > 0 && from < it.tiles && shares.at(c - 1) <= u - from) {
                p.cuts[c] = Cut{1, g, it.t0, s.n, s.row0, shares.of(u - from + it.tiles - 1)};
            }
        }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");     // the scratch's place is the TMA's next
    __syncthreads();
}

struct Kept {
    Walk walk;
    Segment sg;
};

__device__ __forceinline__ int tile_of(const Segment& s, int x) { return s.it.lo + s.it.tiles - 1 - x; }
__device__ __forceinline__ bool two_tiles(const TcArgs& p, const Segment& s) { return s.it.t0 + p.tpt < s.s.n; }

// Whether the tile of keys from `base` holds slots without a token of the
// sequence, or with one that no row of the sequence sees.
__device__ __forceinline__ bool ragged(const TcArgs& p, const Segment& s, int base) {
    return base + kKeys > s.s.kv || base < first_seen(s.s, p.a.window);
}

constexpr uint32_t instr_desc(int n, bool b_mn) {
    return (1u << 4)                                // fp32 accumulator
           | (1u << 7) | (1u << 10)                 // bf16 operands
           | (b_mn ? 1u << 16 : 0u)                 // B stored with its N index contiguous (V), or its K index (K)
           | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

// V's tile as operand B: [64-entry column blocks][128 keys][64 entries], 128-byte swizzle, N contiguous:
// column blocks are 128 rows apart, groups of 8 keys 1024 bytes.
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t saddr) {
    uint64_t d = smem_desc(saddr);
    d &= ~((uint64_t)0x3FFFu << 16);
    return d | (uint64_t)((kKeys * 128) >> 4) << 16;
}

// mbar_wait in line: a call would cost the roles registers that their shares do not have.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag, int where) {
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = global_ns();
    while (!mbar_try_wait_suspend(bar, parity, 1000u)) {
        if (*abort_flag) return false;
        if (global_ns() - t0 > kTimeoutNs) {
            *abort_flag = where;
            return false;
        }
    }
    return true;
}

// For a warp whose lanes go on together.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int* abort_flag, int where) {
    return __all_sync(0xffffffffu, wait_bar(bar, parity, abort_flag, where));
}

#define TMEM_R8(r, o) "=r"(r[o]), "=r"(r[o + 1]), "=r"(r[o + 2]), "=r"(r[o + 3]), "=r"(r[o + 4]), "=r"(r[o + 5]), "=r"(r[o + 6]), "=r"(r[o + 7])
#define TMEM_W8(r, o) "r"(r[o]), "r"(r[o + 1]), "r"(r[o + 2]), "r"(r[o + 3]), "r"(r[o + 4]), "r"(r[o + 5]), "r"(r[o + 6]), "r"(r[o + 7])

// 32 columns of this thread's TMEM lane; the registers may be used after tmem_wait32 (16).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : TMEM_R8(r, 0), TMEM_R8(r, 8), TMEM_R8(r, 16), TMEM_R8(r, 24)
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : TMEM_R8(r, 0), TMEM_R8(r, 8)
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};"
        ::TMEM_W8(r, 0), TMEM_W8(r, 8), "r"(taddr)
        : "memory");
}
// Waits for this thread's TMEM loads; taking the registers as operands keeps their uses below it.
__device__ __forceinline__ void tmem_wait32(uint32_t* r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));
}

// Keeps the uses of registers that an earlier wait was for below this point.
__device__ __forceinline__ void keep32(uint32_t* r) {
#pragma unroll
    for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));
}
__device__ __forceinline__ void tmem_wait16(uint32_t* r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(r[i]));
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// (a, b) * (x, x) + (y, y), two fp32 at once
__device__ __forceinline__ void fma2(float& a, float& b, float x, float y) {
    asm("{\n\t.reg .b64 u, v, w;\n\tmov.b64 u, {%0, %1};\n\tmov.b64 v, {%2, %2};\n\tmov.b64 w, {%3, %3};\n\t"
        "fma.rn.f32x2 u, u, v, w;\n\tmov.b64 {%0, %1}, u;\n\t}"
        : "+f"(a), "+f"(b) : "f"(x), "f"(y));
}
__device__ __forceinline__ void add2(float& a, float& b, float x, float y) {
    asm("{\n\t.reg .b64 u, v;\n\tmov.b64 u, {%0, %1};\n\tmov.b64 v, {%2, %3};\n\t"
        "add.rn.f32x2 u, u, v;\n\tmov.b64 {%0, %1}, u;\n\t}"
        : "+f"(a), "+f"(b) : "f"(x), "f"(y));
}

// The largest of a thread's logits and mx, in four chains.
template <int N>
__device__ __forceinline__ void max_cols(const float* v, float (&mx)[4]) {
#pragma unroll
    for (int i = 0; i < N; i += 8)
#pragma unroll
        for (int c = 0; c < 4; ++c) mx[c] = fmax3(mx[c], v[i + 2 * c], v[i + 2 * c + 1]);
}

// The lowest n bits (none if n < 0).
__device__ __forceinline__ uint32_t low_bits(int n) {
    uint32_t r;
    asm("bmsk.clamp.b32 %0, 0, %1;" : "=r"(r) : "r"(max(n, 0)));
    return r;
}

// Takes out those of 32 columns from `first` on that the row does not see (all but lo to hi).
__device__ __forceinline__ void mask_cols(float* v, int first, int hi, int lo) {
    const uint32_t seen = low_bits(hi - first + 1) & ~low_bits(lo - first);
#pragma unroll
    for (int i = 0; i < 32; ++i)
        if (!(seen >> i & 1)) v[i] = -INFINITY;
}

// The largest logit (before the factor f) of a tile that the row sees, read once more from TMEM.
__device__ __forceinline__ float top_of_row(uint32_t s_at, uint32_t* sr, bool masked, int hi, int lo) {
    float* sv = reinterpret_cast<float*>(sr);
    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
        tmem_ld32(s_at + 32 * c, sr);
        tmem_wait32(sr);
        if (masked) mask_cols(sv, 32 * c, hi, lo);
        max_cols<32>(sv, mx);
    }
    return fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]);
}

// Weights 2^(f v - m) (nm = -m) of 32 logits as pairs of bf16, and their sums.  16 at a time and step by step: pair by pair, a warp
// alone on its scheduler took 610 to 710 cycles for 96 weights, like this 495 (384 are the exponentials').
__device__ __forceinline__ void weights32(const float* v, float f, float nm, float (&zs)[4], uint32_t* pk) {
#pragma unroll
    for (int c = 0; c < 32; c += 16) {
        float w[16];
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            w[i] = v[c + i];
            w[i + 1] = v[c + i + 1];
            fma2(w[i], w[i + 1], f, nm);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = ex2_approx(w[i]);
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            add2(zs[i & 2], zs[(i & 2) + 1], w[i], w[i + 1]);
            pk[(c + i) >> 1] = pack_bf16(w[i], w[i + 1]);
        }
    }
}

// Scales this thread's row of O.
template <int D>
__device__ __forceinline__ void scale_o(uint32_t o_at, float a) {
#pragma unroll 1
    for (int c = 0; c < D / 16; ++c) {
        uint32_t ov[16];
        tmem_ld16(o_at + 16 * c, ov);
        tmem_wait16(ov);
#pragma unroll
        for (int i = 0; i < 16; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * a);
        tmem_st16(o_at + 16 * c, ov);
    }
}

// Lane 4k + j's piece i becomes lane 4k + i's piece j.
__device__ __forceinline__ void transpose4(uint4 (&q)[4]) {
    const int lane = threadIdx.x & 31;
    auto swap = [](uint4 give, int with) {
        give.x = __shfl_xor_sync(0xffffffffu, give.x, with);
        give.y = __shfl_xor_sync(0xffffffffu, give.y, with);
        give.z = __shfl_xor_sync(0xffffffffu, give.z, with);
        give.w = __shfl_xor_sync(0xffffffffu, give.w, with);
        return give;
    };
#pragma unroll
    for (int with = 1; with <= 2; with *= 2) {
        const bool up = lane & with;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i & with) continue;
            // the lower lane gives its piece i + with for the upper lane's piece i
            const uint4 got = swap(up ? q[i] : q[i + with], with);
            if (up) q[i] = got;
            else q[i + with] = got;
        }
    }
}

// A warp's TMEM stores are done: tells the MMAs.
__device__ __forceinline__ void hand_over(uint64_t* bar) {
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(bar));
}

// The MMA warps run with all lanes and issue from one (`lead`): descriptors, addresses and loop counters are then warp-uniform for
// the compiler, which keeps them in uniform registers.  Issued from inside `if (lane == 0)`, an MMA took so many instructions
// that the softmax warps beside it on the scheduler held the tensor cores up (chunk of 4096 over 32768: 1.35 ms).
// A descriptor's upper half is constant, its lower half an address that no stage carries out of.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}\n" : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ void mma_ss(bool lead, uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %6, 0;\n\t"
        "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}\n"
        ::"r"(d), "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"((uint32_t)acc), "r"((uint32_t)lead)
        : "memory");
}
// A from TMEM.
__device__ __forceinline__ void mma_ts(bool lead, uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %6, 0;\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}\n"
        ::"r"(d), "r"(a), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"((uint32_t)acc), "r"((uint32_t)lead)
        : "memory");
}
__device__ __forceinline__ void commit_if(bool lead, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(bar), "r"((uint32_t)lead)
        : "memory");
}
__device__ __forceinline__ void arrive_if(bool lead, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}\n" ::"r"(bar), "r"((uint32_t)lead)
        : "memory");
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

template <int D>
struct Layout {
    static constexpr int kChunks = D / 64;                      // 128-byte column blocks of a row
    static constexpr int kTileBytes = kKeys * D * 2;            // a tile of Q, K or V
    static constexpr int kStages = D == 128 ? 5 : 10;
    static constexpr int kQ = 0, kRing = 2 * kTileBytes, kBars = kRing + kStages * kTileBytes;
    static constexpr int kKeep = kBars + 8 * (3 * kStages + 14), kBad = kKeep + 8 * (int)sizeof(Kept), kEnd = kBad + 8 + (int)sizeof(Walk);
    static_assert(kEnd <= kSmem, "");
    // TMEM columns
    static constexpr int kS(int w) { return w * 128; }
    static constexpr int kO(int w) { return 256 + w * D; }
};

template <int D, int kKind>
__global__ void __launch_bounds__(Roles<kKind>::kThreads, 1) attend_tc_kernel(const __grid_constant__ Maps maps,
                                                                const __grid_constant__ TcArgs p) {
    using L = Layout<D>;
    constexpr bool kSame = kKind == SP_CACHE_SAME;
    constexpr int NS = L::kStages;
    extern __shared__ __align__(1024) uint8_t raw[];
    uint8_t* smem = raw;
    if (smem_u32(smem) & 1023) {            // the swizzle goes by addresses: not met, as there is no other shared memory
        if (threadIdx.x == 0) p.err[blockIdx.x] = 4 | 9 << 8, p.cuts[blockIdx.x].first = 0;
        return;
    }
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
    uint64_t* full = bars;                  // [NS] a K or V tile is ready
    uint64_t* empty = full + NS;            // [NS] the MMAs have read it
    uint64_t* landed = empty + NS;          // [NS] a V tile has arrived and waits to be cleaned
    uint64_t* q_full = landed + NS;
    uint64_t* q_empty = q_full + 1;
    uint64_t* s_full = q_empty + 1;         // [2] S is in TMEM (and all earlier P V done)
    uint64_t* p_full = s_full + 2;          // [2][2] P's first 96 columns are in TMEM and O is scaled; all of P is
    uint64_t* o_full = p_full + 4;          // [2] O is final
    uint64_t* turn = o_full + 2;            // [2] this row tile's MMAs may be issued
    uint64_t* final_bar = turn + 2;
    volatile uint32_t* tmem_sh = reinterpret_cast<volatile uint32_t*>(final_bar + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_sh + 1);    // the wait that gave up, or 0
    int* bad = reinterpret_cast<int*>(smem + L::kBad);                          // [2] impossible lengths; a page index out of range
    Walk* start = reinterpret_cast<Walk*>(bad + 2);
    Kept* keep = reinterpret_cast<Kept*>(smem + L::kKeep);      // [8] a softmax warp's place in its run

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    using W = Roles<kKind>;
    constexpr int kMma = W::kMma, kTma = W::kTma, kClean = W::kClean;
    if (threadIdx.x == 32) {
        const CUtensorMap* m[3] = {&maps.q, &maps.k, &maps.v};
        for (int i = 0; i < (kSame ? 3 : 1); ++i) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m[i])) : "memory");
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(smem_u32(&full[i]), kSame ? 1 : W::kMma - W::kSoftmax);
            mbar_init(smem_u32(&empty[i]), 2);          // the two MMA warps
            mbar_init(smem_u32(&landed[i]), 1);
        }
        mbar_init(smem_u32(q_full), 1);
        mbar_init(smem_u32(q_empty), 2);
        for (int w = 0; w < 2; ++w) {
            mbar_init(smem_u32(&s_full[w]), 1);
            mbar_init(smem_u32(&p_full[2 * w]), 4);
            mbar_init(smem_u32(&p_full[2 * w + 1]), 4);
            mbar_init(smem_u32(&o_full[w]), 1);
            mbar_init(smem_u32(&turn[w]), 1);
        }
        mbar_init(smem_u32(final_bar), 2);
        *abort_flag = 0;
        bad[0] = bad[1] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMma) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32((const void*)tmem_sh)), "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_sh;
    cudaTriggerProgrammaticLaunchCompletion();
    plan(p, reinterpret_cast<int*>(smem + L::kRing), reinterpret_cast<int64_t*>(smem + L::kRing + 4 * (kMaxSeqs + 2)), start, bad);
    Walk walk = *start;
    Segment sg;
    const int rows_tile = p.G * p.tpt;

    if (warp < W::kSoftmax) {
        // ------------------------------ softmax and output ------------------------------
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(W::kSoftmaxRegs));
        const int w = warp >> 2, row = (warp & 3) * 32 + lane;             // row tile; row = TMEM lane
        const uint32_t lane_at = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_at = tmem + lane_at + L::kS(w), o_at = tmem + lane_at + L::kO(w);
        const float f = p.a.scale * 1.4426950408889634f;
        uint32_t ph = 0, ph_o = 0;
        bool ok = true;
        while (ok && walk.next(p, sg)) {
            if (w == 1 && !two_tiles(p, sg)) continue;
            // What the loop over the keys does not need stays in shared memory meanwhile: 128 logits take most of the registers
            if (lane == 0) keep[warp] = Kept{walk, sg};
            __syncwarp();
            // places of the tile's first and last rows, for whether a key tile needs a mask at all, and of this one
            const int p_first = sg.s.kv - sg.s.n + sg.it.t0 + w * p.tpt;
            const int p_last = sg.s.kv - sg.s.n + min(sg.s.n, sg.it.t0 + (w + 1) * p.tpt) - 1;
            const int pos = row < rows_tile ? min(p_first + row / p.G, p_last) : -1;
            // z and O are sums of 2^(logit - m).  m need not be the row's maximum, only near it: it is the maximum of the first tile
            // that the row sees, and where a tile's weights sum to more than 2^8, m grows by that sum's logarithm before the
            // next one.  So the maximum of a tile is not looked for.  A tile is done again by its true maximum if its weights
            // sum to more than 2^24, which is seen before they are handed over (of the last 32 keys by their maximum).
            float m = -INFINITY, z = 0.f, next_m = -INFINITY;
            bool follow = false, fresh = true, huge = false;
            const int n_tiles = sg.to - sg.from;
            int base = tile_of(sg, sg.from) * kKeys;
            for (int x = 0; x < n_tiles; ++x, base -= kKeys) {
                ok = wait_warp(smem_u32(&s_full[w]), ph, abort_flag, 21);
                ph ^= 1;
                if (!ok) break;
                tc_fence_after();
                const bool masked = base + kKeys - 1 > p_first || (p.a.window && base <= p_last - p.a.window);
                const int hi = pos - base, lo = p.a.window ? hi - p.a.window + 1 : -1;      // columns this row sees
                if (follow) {
                    const float a = next_m > m ? ex2_approx(m - next_m) : 1.f;
                    m = next_m;
                    z *= a;
                    scale_o<D>(o_at, a);
                }
                uint32_t sr[kSame ? 128 : 32], pk[48];
                float* sv = reinterpret_cast<float*>(sr);
                float nm, zs[4];
                // twice at most: after a pass by the true maximum nothing is lost
                for (int pass = 0; pass < 2; ++pass) {
                    if (fresh) {            // the true maximum, for rows without an m or with one left far behind
                        const float top = top_of_row(s_at, sr, masked, hi, lo) * f;         // f > 0: f times the largest product
                        // 16: a sum of 96 over 2^24 has a maximum over 2^17.  Also where there was no m
                        const bool far = top > m + (huge ? 0.f : 16.f);
                        const float a = far && m != -INFINITY ? ex2_approx(m - top) : 1.f;
                        if (__any_sync(0xffffffffu, a != 1.f)) scale_o<D>(o_at, a);
                        z *= a;
                        if (far) m = top;
                        huge = __any_sync(0xffffffffu, pos >= 0 && fabsf(m) > 1048576.f && m != -INFINITY);
                        if (huge) break;
                    }
                    nm = m == -INFINITY ? 0.f : -m;
                    zs[0] = zs[1] = zs[2] = zs[3] = 0.f;
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    float* v3 = kSame ? sv + 96 : sv;
                    tmem_ld32(s_at + 96, sr + (kSame ? 96 : 0));
                    if constexpr (kSame) tmem_ld32(s_at, sr);
                    tmem_wait32(sr + (kSame ? 96 : 0));
                    if constexpr (kSame) {
                        tmem_wait32(sr);
                        tmem_ld32(s_at + 32, sr + 32);
                        tmem_ld32(s_at + 64, sr + 64);
                    }
                    if (masked) mask_cols(v3, 96, hi, lo);
                    max_cols<32>(v3, mx);
#pragma unroll
                    for (int c = 0; c < 3; ++c) {
                        float* v = kSame ? sv + 32 * c : sv;
                        if constexpr (!kSame) tmem_ld32(s_at + 32 * c, sr);
                        if (!kSame || c == 1) tmem_wait32(reinterpret_cast<uint32_t*>(v));
                        if constexpr (kSame) {
                            if (c == 2) keep32(sr + 64);
                        }
                        if (masked) mask_cols(v, 32 * c, hi, lo);
                        weights32(v, f, nm, zs, pk + 16 * c);
                    }
                    const float top = fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]) * f;
                    const float sum = (zs[0] + zs[1]) + (zs[2] + zs[3]);
                    fresh = __any_sync(0xffffffffu, pos >= 0 && (sum > 16777216.f || top > m + 24.f));
                    if (!fresh) break;
                }
                if (huge) {
                    // Logits of more than 2^20: f v - m, rounded once, would differ from f v and m, each rounded, by more than the
                    // weights can stand (and a row's own maximum have a weight that overflows or vanishes).  Rounded first, they
                    // are off by what the products' own rounding is.
                    zs[0] = zs[1] = zs[2] = zs[3] = 0.f;
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        tmem_ld32(s_at + 32 * c, sr);
                        tmem_wait32(sr);
                        if (masked) mask_cols(sv, 32 * c, hi, lo);
#pragma unroll
                        for (int i = 0; i < 32; ++i) sv[i] = __fmul_rn(sv[i], f);
                        weights32(sv, 1.f, m == -INFINITY ? 0.f : -m, zs, pk);
                        tmem_st16(s_at + 16 * c, pk);
                    }
                    hand_over(&p_full[2 * w]);
                } else {
#pragma unroll
                    for (int c = 0; c < 3; ++c) tmem_st16(s_at + 16 * c, pk + 16 * c);
                    hand_over(&p_full[2 * w]);      // 96 keys' weights, then the last 32: the product with V begins meanwhile
                    if constexpr (!kSame) {
                        tmem_ld32(s_at + 96, sr);
                        tmem_wait32(sr);
                        if (masked) mask_cols(sv, 96, hi, lo);
                    }
                    weights32(kSame ? sv + 96 : sv, f, nm, zs, pk);
                    tmem_st16(s_at + 48, pk);
                }
                hand_over(&p_full[2 * w + 1]);
                const float sum = (zs[0] + zs[1]) + (zs[2] + zs[3]);
                z += sum;
                const bool grows = !huge && pos >= 0 && sum > 256.f && sum < INFINITY;
                next_m = grows ? m + log2f(sum) : m;
                follow = __any_sync(0xffffffffu, grows);
                fresh = huge || __any_sync(0xffffffffu, pos >= 0 && m == -INFINITY);
            }
            if (!ok) break;
            ok = wait_warp(smem_u32(&o_full[w]), ph_o, abort_flag, 22);
            ph_o ^= 1;
            if (!ok) break;
            tc_fence_after();
            walk = keep[warp].walk;
            sg = keep[warp].sg;
            const int t_row = row / p.G, t = sg.it.t0 + w * p.tpt + t_row;      // this row's new token
            const bool real = row < rows_tile && t < sg.s.n;
            const bool whole = sg.from == 0 && sg.to == sg.it.tiles;
            const float inv = z == 0.f ? 0.f : 1.f / z;
            const int64_t r = sg.s.row0 + t;
            const int h = sg.g * p.G + row - t_row * p.G;
            int64_t row_at[4];          // where the rows of this lane's group of four begin (-1: not a row)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                row_at[i] = __shfl_sync(0xffffffffu, real ? r * p.a.out.stride_row + h * p.a.out.stride_head : -1, (lane & ~3) + i);
            const int64_t slot = (int64_t)blockIdx.x * 2 + (sg.from == 0 ? 1 : 0);
            float* po = p.part_o + slot * kRowsItem * D + (w * 128 + row) * 4;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t ov[32];
                tmem_ld32(o_at + 32 * c, ov);
                tmem_wait32(ov);
                if (whole) {
                    // pieces of 16 bytes are exchanged among four lanes, so that a store writes 64 bytes of each of eight rows
                    // (16 of each of 32 took the load/store unit four times as long)
                    uint4 q[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t o4[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float a = __uint_as_float(ov[8 * i + 2 * k]) * inv, b = __uint_as_float(ov[8 * i + 2 * k + 1]) * inv;
                            o4[k] = z == 0.f ? 0u : pack_bf16(a, b);
                        }
                        q[i] = make_uint4(o4[0], o4[1], o4[2], o4[3]);
                    }
                    transpose4(q);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (row_at[i] >= 0)
                            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.a.out.data) + row_at[i] + 32 * c + 8 * (lane & 3)) = q[i];
                } else {
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        *reinterpret_cast<uint4*>(po + (int64_t)(8 * c + i / 4) * (kRowsItem * 4)) =
                            make_uint4(ov[i], ov[i + 1], ov[i + 2], ov[i + 3]);
                }
            }
            if (whole) {
                if (real && p.a.lse)
                    p.a.lse[r * p.a.lse_stride_row + h * p.a.lse_stride_head] =
                        z == 0.f ? -INFINITY : (m + log2f(z)) * 0.6931471805599453f;
            } else {
                p.part_ml[slot * kRowsItem + w * 128 + row] = make_float2(m, z);
            }
            tc_fence_before();          // O is read before this thread's next hand-off of P
            __syncwarp();               // and `keep` by all lanes
        }
    } else if (!kSame && warp < kMma) {
      if constexpr (!kSame) {
        // ------------------------------ conversion of 8-bit rows ------------------------------
        // A warp takes 16 rows of each tile, a lane 16 entries of each 64 of two rows (rl and rl + 8): eight lanes then store to eight
        // different banks, and a row is read 64 bytes at a time.  A piece is requested for the next tile as soon as it is
        // converted for this one.
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(W::kConvertRegs));
        {
            constexpr int kBlocks = D / 64;
            const sp_cache& c = p.a.cache;
            const int r0 = (warp - W::kSoftmax) * 16, sub = lane & 3, rl = lane >> 2;
            const uint32_t dst0 = (r0 + rl) * 128 + (((2 * sub) ^ rl) << 4), dst1 = (r0 + rl) * 128 + (((2 * sub + 1) ^ rl) << 4);
            int st = 0;
            uint32_t ph = 1;
            bool ok = true;
            while (ok && walk.next(p, sg)) {
                const int32_t* table = p.a.batch.table + (int64_t)sg.it.b * p.a.batch.table_stride;
                const int seen = first_seen(sg.s, p.a.window);
                // this lane's rows of a tile: where they are and their scales, which are not touched before the
                // tile's turn (waiting for them here took a third of the warps' time)
                struct Where {
                    int64_t at;
                    float ks, vs;
                };
                auto token = [&](int x, int y) { return tile_of(sg, x) * kKeys + r0 + rl + 8 * y; };
                auto page_of = [&](int tok) { return tok < sg.s.kv && tok >= seen ? table[p.a.page_of(tok)] : -1; };
                auto place = [&](int tok, int pg) {
                    Where w{sub * 16, 0.f, 0.f};        // nowhere: some row, times 0
                    if (tok >= sg.s.kv || tok < seen) return w;
                    if ((unsigned)pg >= (unsigned)c.pages) {
                        bad[1] = 1;
                        return w;
                    }
                    const int slot = tok - p.a.page_of(tok) * c.page;
                    w.at = row_offset(c, pg, sg.g, slot) + sub * 16;
                    const int64_t sc = scale_offset(c, pg, sg.g, slot);
                    w.ks = __ldg(c.k_scale + sc);
                    w.vs = __ldg(c.v_scale + sc);
                    return w;
                };
                auto fetch = [&](const void* data, int64_t at, int h) {
                    return __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(data) + at + h * 64));
                };
                Where cur[2], nxt[2];
                int next_page[2];
                uint4 codes[2][kBlocks];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    cur[y] = place(token(sg.from, y), page_of(token(sg.from, y)));
#pragma unroll
                    for (int h = 0; h < kBlocks; ++h) codes[y][h] = fetch(c.k, cur[y].at, h);
                }
                // Converts tiles [x, sg.to).  A power of two is its upper half, and so a bf16.  Scales that are none, of a cache that
                // another program has filled: the product is rounded to bf16 as sp_cache_read rounds it (kAny).  Without kAny it
                // returns at the first tile with such a scale.  Seven ragged requests take 136 us from powers of two (172 with
                // a branch for each 16 codes), 174 (int8) and 169 us (e4m3) from others.
                auto tiles = [&](auto kAny, int x) {
                    for (; x < sg.to && ok; ++x) {
                        if constexpr (!kAny) {
                            const uint32_t all = __float_as_uint(cur[0].ks) | __float_as_uint(cur[1].ks) | __float_as_uint(cur[0].vs) |
                                                 __float_as_uint(cur[1].vs);
                            if (__any_sync(0xffffffffu, all & 0xffffu)) return x;
                        }
                        const bool more = x + 1 < sg.to;
#pragma unroll
                        for (int y = 0; y < 2; ++y) next_page[y] = more ? page_of(token(x + 1, y)) : -1;
#pragma unroll
                        for (int v = 0; v < 2; ++v) {
                            if (v == 1) {
#pragma unroll
                                for (int y = 0; y < 2; ++y) {
                                    if (more) nxt[y] = place(token(x + 1, y), next_page[y]);
                                    else nxt[y].at = sub * 16;
                                }
                            }
                            ok = wait_warp(smem_u32(&empty[st]), ph, abort_flag, 61);
                            if (!ok) break;
                            uint8_t* tile = smem + L::kRing + st * L::kTileBytes;
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const float own = v ? cur[y].vs : cur[y].ks;
                                const uint32_t scale = __byte_perm(__float_as_uint(own), 0, 0x3232);     // a pair of bf16
#pragma unroll
                                for (int h = 0; h < kBlocks; ++h) {
                                    const uint32_t w4[4] = {codes[y][h].x, codes[y][h].y, codes[y][h].z, codes[y][h].w};
                                    uint32_t o[8];
#pragma unroll
                                    for (int i = 0; i < 4; ++i) {
                                        uint32_t pair[2];
                                        pairs_of<kKind, true>(w4[i], pair[0], pair[1]);
#pragma unroll
                                        for (int k = 0; k < 2; ++k)
                                            o[2 * i + k] = kAny ? pack_bf16(__uint_as_float(pair[k] << 16) * own,
                                                                            __uint_as_float(pair[k] & 0xffff0000u) * own)
                                                                : mul_bf16x2(pair[k], scale);
                                    }
                                    codes[y][h] = v ? fetch(c.k, nxt[y].at, h) : fetch(c.v, cur[y].at, h);
                                    uint8_t* at = tile + y * 1024 + h * (kKeys * 128);
                                    *reinterpret_cast<uint4*>(at + dst0) = make_uint4(o[0], o[1], o[2], o[3]);
                                    *reinterpret_cast<uint4*>(at + dst1) = make_uint4(o[4], o[5], o[6], o[7]);
                                }
                            }
                            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                            __syncwarp();
                            if (lane == 0) mbar_arrive(smem_u32(&full[st]));
                            if (++st == NS) st = 0, ph ^= 1;
                        }
                        cur[0] = nxt[0];
                        cur[1] = nxt[1];
                    }
                    return x;
                };
                tiles(std::true_type{}, tiles(std::false_type{}, sg.from));
            }
        }
      }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(W::kSingleRegs));
        if (warp == kMma || warp == kMma + 1) {
            // ------------------------------ MMAs of one row tile ------------------------------
            constexpr uint32_t kIdS = instr_desc(kKeys, false), kIdO = instr_desc(D, true);
            const int w = __shfl_sync(0xffffffffu, warp - kMma, 0);
            const bool lead = elect_one();
            const uint32_t s_at = L::kS(0) + w * 128, o_at = L::kO(0) + w * D;      // all of TMEM is this CTA's: it begins at 0
            const uint32_t ring = smem_u32(smem + L::kRing);
            const uint64_t q_desc = smem_desc(smem_u32(smem + L::kQ)), k_desc = smem_desc(ring), v_desc = smem_desc_mn(ring);
            const uint32_t q_lo = (uint32_t)q_desc + w * (L::kTileBytes >> 4), k_lo = (uint32_t)k_desc, v_lo = (uint32_t)v_desc;
            const uint32_t s_hi = (uint32_t)(k_desc >> 32), v_hi = (uint32_t)(v_desc >> 32);
            const uint32_t full_at = smem_u32(full), empty_at = smem_u32(empty), s_bar = smem_u32(s_full) + 8 * w,
                           p_bar = smem_u32(p_full) + 16 * w, o_bar = smem_u32(o_full) + 8 * w, my_turn = smem_u32(turn) + 8 * w,
                           other_turn = smem_u32(turn) + 8 * (1 - w);
            int st = 0;
            uint32_t ph = 0, ph_q = 0, ph_p = 0, ph_t = 1 - w;     // the first turn is A's
            bool ok = tmem == 0;
            auto wait = [&](uint32_t bar, uint32_t parity, int where) { return wait_warp(bar, parity, abort_flag, where); };
            auto step = [&] {
                if (++st == NS) st = 0, ph ^= 1;
            };
            auto s_mma = [&](bool hand_on) {
                const uint32_t b = k_lo + st * (L::kTileBytes >> 4);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = ((k >> 2) * (kKeys * 128) + (k & 3) * 32) >> 4;
                    mma_ss(lead, s_at, q_lo + off, b + off, s_hi, kIdS, k > 0);
                    // the other warp needs about as long to see it as the rest of these take
                    if (k == D / 16 - 3 && hand_on) arrive_if(lead, other_turn);
                }
                commit_if(lead, s_bar);
                commit_if(lead, empty_at + 8 * st);
            };
            while (ok && walk.next(p, sg)) {
                const int nt = sg.to - sg.from;
                const bool two = two_tiles(p, sg);
                ok = wait(smem_u32(q_full), ph_q, 31);
                ph_q ^= 1;
                if (!ok) break;
                if (w == 1 && !two) {
                    // no rows of this tile: the stages are handed back as they come
                    arrive_if(lead, smem_u32(q_empty));
                    for (int i = 0; i < 2 * nt && ok; ++i) {
                        ok = wait(full_at + 8 * st, ph, 37);
                        if (ok) arrive_if(lead, empty_at + 8 * st);
                        step();
                    }
                    continue;
                }
                ok = wait(full_at + 8 * st, ph, 32);
                if (!ok) break;
                tc_fence_after();
                s_mma(false);
                if (nt == 1) commit_if(lead, smem_u32(q_empty));
                step();
                for (int i = 0; i < nt; ++i) {
                    const int sk = st + 1 == NS ? 0 : st + 1;       // the next K tile's stage
                    ok = wait(full_at + 8 * st, ph, 33) && (i + 1 == nt || wait(full_at + 8 * sk, ph ^ (sk == 0), 35)) &&
                         wait(p_bar, ph_p, 34) && (!two || wait(my_turn, ph_t, 38));
                    if (two) ph_t ^= 1;
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t b = v_lo + st * (L::kTileBytes >> 4);
#pragma unroll
                    for (int k = 0; k < 6; ++k)
                        mma_ts(lead, o_at, s_at + k * 8, b + ((k * 16 * 128) >> 4), v_hi, kIdO, i > 0 || k > 0);
                    ok = wait(p_bar + 8, ph_p, 39);
                    ph_p ^= 1;
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int k = 6; k < 8; ++k) mma_ts(lead, o_at, s_at + k * 8, b + ((k * 16 * 128) >> 4), v_hi, kIdO, true);
                    commit_if(lead, empty_at + 8 * st);
                    step();
                    if (i + 1 == nt) {
                        if (two) arrive_if(lead, other_turn);
                        commit_if(lead, o_bar);
                        break;
                    }
                    s_mma(two);
                    if (i + 2 == nt) commit_if(lead, smem_u32(q_empty));
                    step();
                }
            }
            // nothing of this warp's MMAs is in flight when TMEM is freed
            commit_if(lead, smem_u32(final_bar));
            if (lead) {
                if (tmem != 0) *abort_flag = 8;
                const unsigned long long t0 = global_ns();
                while (!mbar_try_wait_suspend(smem_u32(final_bar), 0, 1000u))
                    if (global_ns() - t0 > kTimeoutNs) {
                        *abort_flag = 36;
                        break;
                    }
            }
            __syncwarp();
        } else if (warp == kTma) {
            // ------------------------------ TMA ------------------------------
            const uint32_t ring = smem_u32(smem + L::kRing), qs = smem_u32(smem + L::kQ);
            const sp_cache& c = p.a.cache;
            int st = 0, loads = 0;
            uint32_t ph = 1, ph_q = 1;          // a fresh barrier counts as completed for the odd parity
            uint32_t dirty = 0;                 // stages whose last load went to `landed`
            bool ok = true;
            const int boxes = kKeys / p.box;
            while (ok && walk.next(p, sg)) {
                const int nw = two_tiles(p, sg) ? 2 : 1;
                const int32_t* table = p.a.batch.table + (int64_t)sg.it.b * p.a.batch.table_stride;
                const int seen = first_seen(sg.s, p.a.window);
                ok = wait_warp(smem_u32(q_empty), ph_q, abort_flag, 41);
                ph_q ^= 1;
                if (!ok) break;
                if (lane == 0) {
                    mbar_expect_tx(smem_u32(q_full), (uint32_t)(nw * rows_tile * D * 2));
                    for (int w = 0; w < nw; ++w)
                        for (int ch = 0; ch < L::kChunks; ++ch)
                            tma_load_3d(qs + w * L::kTileBytes + ch * (kKeys * 128), &maps.q, ch * 64, sg.g * p.G,
                                        (int)(sg.s.row0 + sg.it.t0 + w * p.tpt), smem_u32(q_full));
                }
                if constexpr (!kSame) continue;
                // this lane's box of a tile: its page (pages: none, which loads zeros) and its first slot
                auto page_of = [&](int x, int& slot) {
                    const int tok = tile_of(sg, x) * kKeys + lane * p.box;
                    slot = 0;
                    if (lane >= boxes || tok >= sg.s.kv || tok + p.box <= seen) return (int)c.pages;
                    const int q = p.a.page_of(tok), pg = table[q];
                    if (pg < 0 || pg >= c.pages) {
                        bad[1] = 1;
                        return (int)c.pages;
                    }
                    slot = tok - q * c.page;
                    return pg;
                };
                int slot, pg = page_of(sg.from, slot);
                for (int x = sg.from; x < sg.to && ok; ++x) {
                    int slot2 = 0, pg2 = 0;
                    if (x + 1 < sg.to) pg2 = page_of(x + 1, slot2);
                    const bool clean = !ragged(p, sg, tile_of(sg, x) * kKeys);
                    for (int v = 0; v < 2; ++v) {
                        ok = wait_warp(smem_u32(&empty[st]), ph, abort_flag, 42);
                        if (!ok) break;
                        const bool wash = v == 1 && !clean;
                        const uint32_t bar = smem_u32(wash ? &landed[st] : &full[st]);
                        if (lane == 0) mbar_expect_tx(bar, L::kTileBytes);
                        __syncwarp();
                        if (lane < boxes)
#pragma unroll
                            for (int ch = 0; ch < L::kChunks; ++ch)
                                tma_load_4d(ring + st * L::kTileBytes + ch * (kKeys * 128) + lane * p.box * 128,
                                            v ? &maps.v : &maps.k, ch * 64, slot, sg.g, pg, bar);
                        if (wash) dirty |= 1u << st;
                        else dirty &= ~(1u << st);
                        ++loads;
                        if (++st == NS) st = 0, ph ^= 1;
                    }
                    pg = pg2;
                    slot = slot2;
                }
            }
            (void)dirty; (void)loads;
            // an aborted CTA's copies land before it leaves
            if (kSame && lane == 0 && *abort_flag) {
                const unsigned long long t0 = global_ns();
                for (int k = 1; k <= min(loads, NS); ++k) {
                    const int s1 = (st - k + NS) % NS;
                    const uint32_t parity = (uint32_t)(((loads - k) / NS) & 1);
                    // a load that waits to be cleaned is followed on a barrier of its own, whose phase is not known here
                    if (dirty >> s1 & 1) {
                        const unsigned long long t1 = global_ns();
                        while (global_ns() - t1 < 1000000ull) {}
                        continue;
                    }
                    while (!mbar_try_wait_suspend(smem_u32(&full[s1]), parity, 1000u) && global_ns() - t0 < kTimeoutNs) {}
                }
            }
            __syncwarp();
        } else if (warp == kClean && kSame) {
            // ------------------------------ cleaning of V ------------------------------
            int st = 0;
            uint32_t ph = 0;                    // per stage
            bool ok = true;
            while (ok && walk.next(p, sg)) {
                const int seen = first_seen(sg.s, p.a.window);
                for (int x = sg.from; x < sg.to && ok; ++x) {
                    const int base = tile_of(sg, x) * kKeys, sv = st + 1 == NS ? 0 : st + 1;
                    st = sv + 1 == NS ? 0 : sv + 1;
                    if (!ragged(p, sg, base)) continue;
                    ok = wait_warp(smem_u32(&landed[sv]), (ph >> sv) & 1, abort_flag, 51);
                    ph ^= 1u << sv;
                    if (!ok) break;
                    uint8_t* tile = smem + L::kRing + sv * L::kTileBytes;
                    // a row is 128 bytes in each column block, wherever the swizzle puts its pieces
                    for (int i = lane; i < kKeys * L::kChunks * 8; i += 32) {
                        const int rr = i >> 3, tok = base + (rr & (kKeys - 1));
                        if (tok >= sg.s.kv || tok < seen) *reinterpret_cast<uint4*>(tile + i * 16) = make_uint4(0, 0, 0, 0);
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&full[sv]));
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (threadIdx.x == 0) p.err[blockIdx.x] = (bad[0] ? 1 : 0) | (bad[1] ? 2 : 0) | (*abort_flag ? 4 | *abort_flag << 8 : 0);
    cudaGridDependencySynchronize();        // of a mixed batch: the step kernels, which ran beside this one, end before it does
    if (warp == kMma)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

// Adds up the parts of the items that were cut: block (c - 1, y) takes the item that CTA c's run begins in, and 16 of its columns;
// a thread one row.  Block (0, 0) gathers the status as well: `alone` if no other kernel of the call has one.
template <int D>
__global__ void __launch_bounds__(kRowsItem) tc_join_kernel(const __grid_constant__ TcArgs p, int alone) {
    cudaGridDependencySynchronize();
    if (blockIdx.x == 0 && blockIdx.y == 0) {
        const int e = threadIdx.x < p.P ? p.err[threadIdx.x] : 0;
        const bool bad = __syncthreads_or(e & 3), gone = __syncthreads_or(e & 4);
        if (threadIdx.x == 0 && (alone || bad)) {
            p.hdr->status = bad ? SP_EDEVICE : SP_OK;
            p.hdr->where = 0;
        }
        __syncthreads();
        if (bad && (e & 3)) p.hdr->where = e & 3;
        if (gone && (e & 4)) {
            p.hdr->status = SP_ETIMEOUT;
            p.hdr->where = e >> 8;
        }
    }
    const int c = blockIdx.x + 1, row = threadIdx.x;
    const Cut q = p.cuts[c];
    if (!q.first) return;
    const int g = q.g, c1 = q.last;
    const int w = row >> 7, r = row & 127, t_row = r / p.G, t = q.t0 + w * p.tpt + t_row;
    if (r >= p.G * p.tpt || t >= q.n) return;
    // Part after part with a running maximum; the next part is on its way while one is added.  (The first part begins with the item's
    // first tile: slot 2 k + 1, the others 2 k.)
    struct Part {
        float2 ml;
        float4 o[4];
    };
    auto fetch = [&](int k) {
        const int64_t slot = (int64_t)k * 2 + (k == c - 1);
        Part x;
        x.ml = p.part_ml[slot * kRowsItem + row];
        const float4* src = reinterpret_cast<const float4*>(p.part_o) + (slot * (D / 4) + blockIdx.y * 4) * kRowsItem + row;
#pragma unroll
        for (int i = 0; i < 4; ++i) x.o[i] = src[i * kRowsItem];
        return x;
    };
    float m = -INFINITY, z = 0.f, v[16] = {};
    Part next = fetch(c - 1);
    for (int k = c - 1; k <= c1; ++k) {
        const Part x = next;
        if (k < c1) next = fetch(k + 1);
        const float top = fmaxf(m, x.ml.x);
        // a side without a maximum has summed nothing, or NaN alone: it counts as it is
        const float a = x.ml.x == -INFINITY ? 1.f : ex2_approx(x.ml.x - top), b = m == -INFINITY ? 1.f : ex2_approx(m - top);
        m = top;
        z = z * b + x.ml.y * a;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[4 * i] = v[4 * i] * b + x.o[i].x * a;
            v[4 * i + 1] = v[4 * i + 1] * b + x.o[i].y * a;
            v[4 * i + 2] = v[4 * i + 2] * b + x.o[i].z * a;
            v[4 * i + 3] = v[4 * i + 3] * b + x.o[i].w * a;
        }
    }
    const float inv = z == 0.f ? 0.f : 1.f / z;
    const int h = g * p.G + r - t_row * p.G;
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.a.out.data) + (q.row0 + t) * p.a.out.stride_row +
                         h * p.a.out.stride_head + blockIdx.y * 16;
    float o0[8], o1[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        o0[i] = z == 0.f ? 0.f : v[i] * inv;
        o1[i] = z == 0.f ? 0.f : v[8 + i] * inv;
    }
    store8(dst, o0);
    store8(dst + 8, o1);
    if (p.a.lse && blockIdx.y == 0)
        p.a.lse[(q.row0 + t) * p.a.lse_stride_row + h * p.a.lse_stride_head] =
            z == 0.f ? -INFINITY : (m + log2f(z)) * 0.6931471805599453f;
}

struct Space {
    size_t err, cuts, part_o, part_ml, total;
};

Space carve(int d, int P) {
    Space s;
    Carve c;
    s.err = c.take((size_t)P * sizeof(int));
    s.cuts = c.take((size_t)P * sizeof(Cut));
    s.part_o = c.take((size_t)P * 2 * kRowsItem * d * sizeof(float));
    s.part_ml = c.take((size_t)P * 2 * kRowsItem * sizeof(float2));
    s.total = c.off;
    return s;
}

// A tensor map of bf16 rows; strides in entries.  An extent of 1 has no stride of its own.
sp_status encode(CUtensorMap* map, const void* data, int rank, const int64_t* extent, const int64_t* stride, const int* box) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
    if (!enc) {
        set_error("sp_attend: cuTensorMapEncodeTiled is unavailable from the driver");
        return SP_ECUDA;
    }
    cuuint64_t dim[4], step[3];
    cuuint32_t bx[4], one[4] = {1, 1, 1, 1};
    for (int i = 0; i < rank; ++i) {
        dim[i] = (cuuint64_t)extent[i];
        bx[i] = (cuuint32_t)box[i];
        if (i) step[i - 1] = extent[i] == 1 ? 16 : (cuuint64_t)stride[i] * 2;
    }
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(data), dim, step, bx, one,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        set_error("sp_attend: cuTensorMapEncodeTiled failed (%d)", (int)r);
        return SP_ECUDA;
    }
    return SP_OK;
}

template <int D, int kKind>
sp_status launch(const Maps& maps, const TcArgs& p, cudaStream_t st) {
    SP_CUDA_TRY(cudaFuncSetAttribute(attend_tc_kernel<D, kKind>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem));
    // after the step kernels of a mixed batch this one does not wait for them
    if (p.min_rows > 0) {
        const sp_status s = launch_early(attend_tc_kernel<D, kKind>, dim3((unsigned)p.P), Roles<kKind>::kThreads, (size_t)kSmem, st, maps, p);
        if (s != SP_OK) return s;
    } else {
        attend_tc_kernel<D, kKind><<<p.P, Roles<kKind>::kThreads, kSmem, st>>>(maps, p);
        SP_LAUNCH_CHECK();
    }
    return launch_early(tc_join_kernel<D>, dim3((unsigned)std::max(1, p.P - 1), D / 16), kRowsItem, (size_t)0, st, p, p.min_rows == 0 ? 1 : 0);
}

template <int D>
sp_status launch_codes(const Maps& maps, const TcArgs& p, cudaStream_t st) {
    return p.a.cache.kind == SP_CACHE_E4M3 ? launch<D, SP_CACHE_E4M3>(maps, p, st) : launch<D, SP_CACHE_INT8>(maps, p, st);
}

}  // namespace

// Whether the cache and the group of heads are within the kernel's layouts.
bool attend_tc_supported(const sp_cache& c, const sp_batch& b, int G) {
    if (b.B > kMaxSeqs || sm_count() < 2 || sm_count() > kRowsItem) return false;     // (the join looks at a CTA's status per thread)
    if (c.dtype != SP_BF16 || (c.d != 64 && c.d != 128) || G > 128) return false;
    if (c.kind != SP_CACHE_SAME)                                        // rows of codes are read 16 bytes at a time
        return (reinterpret_cast<uintptr_t>(c.k) | reinterpret_cast<uintptr_t>(c.v) | (uintptr_t)c.stride_page |
                (uintptr_t)c.stride_head | (uintptr_t)c.stride_slot) % 16 == 0;
    if (c.page % 8 != 0) return false;                                  // boxes of 8 rows at least
    const int64_t limit = (int64_t)1 << 39;                             // tensor-map strides are below 2^40 bytes
    if (c.stride_slot >= limit / 2 || c.stride_head >= limit / 2 || c.stride_page >= limit / 2) return false;
    return !(c.H_kv > 1 && c.stride_head == 0) && !(c.pages > 1 && c.stride_page == 0);
}

size_t attend_tc_ws_bytes(const sp_cache& c) { return carve(c.d, sm_count()).total; }

// min_rows: sequences of at most that many rows per KV head are taken by another kernel, whose workspace `ws` begins with; this
// one's is `offset` bytes on.
sp_status attend_tc_launch(const AttendProblem& a, int min_rows, void* ws, size_t offset, cudaStream_t st) {
    TcArgs p;
    p.a = a;
    p.G = a.H / a.cache.H_kv;
    p.tpt = 128 / p.G;
    p.min_rows = min_rows;
    p.P = sm_count();
    p.box = std::min(128, a.cache.page & -a.cache.page);
    char* base = static_cast<char*>(ws) + offset;
    const Space s = carve(a.cache.d, p.P);
    p.hdr = static_cast<WsHeader*>(ws);
    p.err = reinterpret_cast<int*>(base + s.err);
    p.cuts = reinterpret_cast<Cut*>(base + s.cuts);
    p.part_o = reinterpret_cast<float*>(base + s.part_o);
    p.part_ml = reinterpret_cast<float2*>(base + s.part_ml);
    Maps maps;
    const int64_t q_ext[3] = {a.cache.d, a.H, std::max<int64_t>(a.batch.T, 1)}, q_str[3] = {1, a.q.stride_head, a.q.stride_row};
    const int q_box[3] = {64, p.G, p.tpt};
    const int64_t c_ext[4] = {a.cache.d, a.cache.page, a.cache.H_kv, a.cache.pages};
    const int64_t c_str[4] = {1, a.cache.stride_slot, a.cache.stride_head, a.cache.stride_page};
    const int c_box[4] = {64, p.box, 1, 1};
    sp_status e;
    memset(&maps, 0, sizeof(maps));
    if ((e = encode(&maps.q, a.q.data, 3, q_ext, q_str, q_box)) != SP_OK) return e;
    if (a.cache.kind != SP_CACHE_SAME)
        return a.cache.d == 64 ? launch_codes<64>(maps, p, st) : launch_codes<128>(maps, p, st);
    if ((e = encode(&maps.k, a.cache.k, 4, c_ext, c_str, c_box)) != SP_OK ||
        (e = encode(&maps.v, a.cache.v, 4, c_ext, c_str, c_box)) != SP_OK)
        return e;
    return a.cache.d == 64 ? launch<64, SP_CACHE_SAME>(maps, p, st) : launch<128, SP_CACHE_SAME>(maps, p, st);
}

}  // namespace sp
