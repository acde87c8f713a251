// The attention weight that cached tokens gather, on tensor cores: tcgen05.mma + TMA + TMEM.  bf16, head dimension 64 or 128.
//
//   w[i] = decay * w[i] + sum over the rows that see token i of 2^(f q . k_i - l),  f = scale * log2(e), l = lse * log2(e)
//
// The keys are the rows of the product and the query rows its columns: S = K Q^T has a key in each TMEM lane, so a thread adds up its
// own key's weights and nothing is exchanged.  Query rows are packed by KV head (row r of a tile: token r / G, head r % G).
// An item is 256 keys (two tiles, A and B) of one sequence and KV head; its keys stay in shared memory while the
// tiles of 128 query rows that see any of them come by, each read for both key tiles: with one key tile an item the
// query rows' traffic would be 64 bytes a clock and SM, which L2 does not give.
//
// Per 256 x 128 logits the MMAs take 1024 cycles (d = 128; 512 at d = 64) and the exponentials as many (32 a clock and SM), so
// both units are to be busy at the same time: S has two buffers for each key tile, and the eight adding warps empty one while
// the MMAs fill the other.  What bounds it is neither unit: an adding warp issues an FMA and an ADD on pairs of weights and an
// exponential a weight, about two cycles of its scheduler each, which is 1.2 times the exponentials' own time.
// A chunk of 4096 tokens over 32768 (32/8 heads of 128): 825 us from bf16, 1.25 PFLOP/s, of which reading the normalisers from shared
// memory is some 60, and 940 from e4m3.  The last 32 of 131072 tokens (one row tile an item): 68 us from e4m3, 59 from bf16; the adding
// is 20 of them beside the rest, the conversion of codes 2, and 50 stay without either: starts, waits and the keys' way in.
//
// Warp roles of a CTA (one per SM):
//  * eight warps add up weights: of a bf16 cache each has 64 keys of both tiles and every other 32 columns, of an 8-bit one 32 keys of
//    one tile and all columns;
//  * four warps, for an 8-bit cache only: make bf16 of its codes in the shared-memory tiles (their scales are factors of
//    a thread's logits);
//  * one issues the MMAs, one makes the TMA loads of keys, page by page, and of query rows, one reads the rows' normalisers.
//
// The items of the call are laid end to end and each CTA takes an equal run of (key block, row tile) pairs.  An item that is cut
// leaves its sums in the workspace and a joining kernel adds them up in a fixed order.
#include "tc_tiles.cuh"

#include <string.h>

#include <algorithm>

namespace sp {
namespace {

constexpr int kKeys = 128;              // keys of a tile
constexpr int kBlock = 2 * kKeys;       // keys of an item
constexpr int kSmem = 227 * 1024;
constexpr int kExtra = 1;               // what an item costs beside its row tiles, in row tiles
constexpr int kMaxSeqs = 16384;         // their item counts are laid out in the (still empty) rings

// Warps of a CTA by role.  setmaxnreg shares out the registers that the block was launched with: 384 threads of 168, or 512 of 128 (eight converting
// warps left the adding ones 112 registers: 72 us for 68, the last 32 of 131072 tokens).
template <int kKind>
struct Roles {
    static constexpr bool kSame = kKind == SP_CACHE_SAME;
    static constexpr int kAdd = 8, kConvert = kSame ? 0 : 4, kMma = kAdd + kConvert, kTma = kMma + 1, kLse = kMma + 2;
    static constexpr int kThreads = 32 * (kMma + 4);
    static constexpr int kAddRegs = kSame ? 192 : 168, kConvertRegs = 80, kSingleRegs = kSame ? 120 : 96;
    static_assert(kAdd * kAddRegs + (kMma - kAdd) * kConvertRegs + 4 * kSingleRegs <= (kMma + 4) * (kSame ? 168 : 128),
                  "the roles' registers");
};

struct Cut {
    int first, b, g, k0;    // whether the CTA's run begins inside an item that no CTA before has cut; sequence, KV head, first key
    int last;               // the CTA of the item's last part
};

struct TcArgs {
    WeightsProblem w;
    int G, tpt;             // query heads of a KV head; new tokens of a row tile
    int P;                  // CTAs
    int box;                // rows of a TMA box
    int k_stages, q_stages; // of the rings
    WsHeader* hdr;
    int* err;               // [P]: 1 impossible lengths, 2 a page index out of range, 4 a wait that gave up (in bits 8-15)
    Cut* cuts;              // [P]
    float* parts;           // [P][2][256]
};

struct Maps {
    CUtensorMap q, k;
};

// Key blocks of a sequence, from the first with a token that a row sees.
__device__ __forceinline__ int blocks_of(const TcArgs& p, const Seq& s) {
    return s.n > 0 && s.kv > 0 ? (s.kv - 1) / kBlock - first_seen(s, p.w.a.window) / kBlock + 1 : 0;
}

struct Item {
    int k0;                 // first key
    int ta, tb;             // the new tokens that see any of its keys
    int tiles;              // of query rows
};
__device__ __forceinline__ Item item_of(const TcArgs& p, const Seq& s, int j) {
    Item it;
    it.k0 = (first_seen(s, p.w.a.window) / kBlock + j) * kBlock;
    const int ctx = s.kv - s.n, last = min(it.k0 + kBlock, s.kv) - 1;
    it.ta = max(0, it.k0 - ctx);
    it.tb = p.w.a.window ? (int)min((int64_t)s.n, (int64_t)last + p.w.a.window - ctx) : s.n;
    it.tiles = (it.tb - it.ta + p.tpt - 1) / p.tpt;
    return it;
}

struct Segment {
    Item it;
    Seq s;
    int b, g, from, to;     // sequence, KV head; row tiles [from, to) of the item
    bool same;              // its one row tile is the one before
};

// A CTA's run, item by item: KV head, sequence, key block, row tile.  Every role walks it by itself; all lanes of a warp together.
struct Walk {
    int left, g, b, j, from;            // units (row tiles and kExtra an item) left; the next item and its first unit
    int was_b, was_g, was_ta;           // the last item, if it had one row tile
    int have, blocks, tiles;            // the sequence that these are of: its key blocks, and the row tiles of all its new tokens
    Seq s;

    // (Nearly all items are seen by all new tokens of the sequence before: for these there is little to do, as every warp does it.)
    __device__ __forceinline__ bool next(const TcArgs& p, Segment& o) {
        while (left > 0) {
            if (have != b) {
                s = load_seq(p.w.a.batch, p.w.a.cache.page, b);
                blocks = blocks_of(p, s);
                tiles = (s.n + p.tpt - 1) / p.tpt;
                have = b;
            }
            o.s = s;
            if (j >= blocks) {          // the arrays were changed while the kernel ran
                left = 0;
                break;
            }
            if (!p.w.a.window && j * kBlock <= s.kv - s.n) o.it = Item{j * kBlock, 0, s.n, tiles};
            else o.it = item_of(p, s, j);
            o.b = b;
            o.g = g;
            o.from = from;
            const int to = min(o.it.tiles + kExtra, from + left);
            o.to = min(o.it.tiles, to);
            left -= to - from;
            from = 0;
            if (left > 0 && ++j >= blocks) next_seq(p);
            if (o.from >= o.to) continue;       // the run begins behind the item's last tile
            const bool one = o.it.tiles == 1;
            o.same = one && was_b == o.b && was_g == o.g && was_ta == o.it.ta;
            was_b = one ? o.b : -1;
            was_g = o.g;
            was_ta = o.it.ta;
            return true;
        }
        return false;
    }
    __device__ __forceinline__ void next_seq(const TcArgs& p) {
        const int lane = threadIdx.x & 31;
        j = 0;
        for (int first = b + 1, rounds = 0;; first += 32) {
            if (first >= p.w.a.batch.B) {
                first = 0;
                ++g;
                if (++rounds > 1) {
                    left = 0;
                    return;
                }
            }
            int n = 0;
            if (first + lane < p.w.a.batch.B) n = blocks_of(p, load_seq(p.w.a.batch, p.w.a.cache.page, first + lane));
            const unsigned some = __ballot_sync(0xffffffffu, n > 0);
            if (some) {
                b = first + __ffs(some) - 1;
                return;
            }
        }
    }
};

// Where this CTA's run begins, worked out by all its threads: the key blocks of every sequence are counted, then each thread adds
// up the units of an equal share of them, and the one whose share holds the first unit finds it.
__device__ __forceinline__ void plan(const TcArgs& p, int* starts, int64_t* sums, Walk* out, int* bad) {
    const int t = threadIdx.x, threads = blockDim.x, B = p.w.a.batch.B, page = p.w.a.cache.page;
    int64_t total, base = 0;
    for (int b0 = 0; b0 < B; b0 += threads) {
        int n = 0;
        if (b0 + t < B) {
            const Seq s = load_seq(p.w.a.batch, page, b0 + t);
            if (!s.ok) bad[0] = 1;
            n = blocks_of(p, s);
        }
        const int64_t before = block_scan(n, sums, total);
        if (b0 + t < B) starts[b0 + t] = (int)(base + before);
        base += total;
    }
    if (t == 0) {
        starts[B] = (int)base;
        *out = Walk{0, 0, 0, 0, 0, -1, 0, 0, -1, 0, 0, {}};
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
    // visits the share's items until `stop` of their units are passed; returns the units
    int seq = b, blk = 0;
    auto visit = [&](int64_t stop) {
        int64_t sum = 0;
        seq = b;
        Seq s = load_seq(p.w.a.batch, page, seq);
        for (int j = j0; j < j1; ++j) {
            while (j >= starts[seq + 1]) s = load_seq(p.w.a.batch, page, ++seq);
            blk = j - starts[seq];
            const int units = item_of(p, s, blk).tiles + kExtra;
            if (sum + units > stop) break;
            sum += units;
        }
        return sum;
    };
    const int64_t mine = visit(INT64_MAX), before = block_scan(mine, sums, total);
    const int64_t U = total * p.w.a.cache.H_kv;
    const Shares shares(U, p.P);
    const int c = blockIdx.x;
    const int64_t u = shares.at(c), left = shares.at(c + 1) - u;
    if (left > 0) {
        const int g = (int)divide(u, total);
        const int64_t r = u - g * total;
        if (before <= r && r < before + mine) {
            const int from = (int)(r - before - visit(r - before));
            *out = Walk{(int)left, g, seq, blk, from, -1, 0, 0, -1, 0, 0, {}};
            const Item it = item_of(p, load_seq(p.w.a.batch, page, seq), blk);
            if (from > 0 && from < it.tiles && shares.at(c - 1) <= u - from)
                p.cuts[c] = Cut{1, seq, g, it.k0, shares.of(u - from + it.tiles - 1)};
        }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");     // the scratch's place is the TMA's next
    __syncthreads();
}

// Shared memory: rings of key tiles, of row tiles and, of an 8-bit cache, of tiles of codes in what is left of 224 KB; then the
// normalisers beside S, what the halves of the adding warps exchange, and the barriers.
template <int D, int kKind>
struct Layout {
    static constexpr int kChunks = D / 64;
    static constexpr int kTileBytes = kKeys * D * 2, kCodeBytes = kKeys * D;       // a tile of K or Q; of codes
    static constexpr int kRings = 224 * 1024, kTiles = kRings / kTileBytes;
    static constexpr int kL = kRings, kHalf = kL + 2 * 128 * 4, kBars = kHalf + kBlock * 4;
    static constexpr int kMostStages = kKind == SP_CACHE_SAME ? kTiles : 2 * kTiles;        // of all rings together
    static constexpr int kBarCount = 2 * kMostStages + 4 + 4 + 1;
    static constexpr int kBad = kBars + 8 * (kBarCount + 1), kEnd = kBad + 8 + (int)sizeof(Walk);
    static_assert(kEnd <= kSmem, "");
    static_assert(kRings >= 4 * (kMaxSeqs + 2) + 8 * 32, "the plan's scratch");
    static constexpr int kS(int w, int buf) { return (2 * buf + w) * 128; }         // TMEM columns
};

// (a, b) = (x, y) * (f, f) + (n, m), two fp32 at once
__device__ __forceinline__ void fma2n(float& a, float& b, float x, float y, float f, float n, float m) {
    asm("{\n\t.reg .b64 u, v, w;\n\tmov.b64 u, {%2, %3};\n\tmov.b64 v, {%4, %4};\n\tmov.b64 w, {%5, %6};\n\t"
        "fma.rn.f32x2 u, u, v, w;\n\tmov.b64 {%0, %1}, u;\n\t}"
        : "=f"(a), "=f"(b) : "f"(x), "f"(y), "f"(f), "f"(n), "f"(m));
}

// 32 logits each of kN keys to weights 2^(f v - l) (nl = -l, of each column), those of the rows that see them added to z.
// What is hidden is taken out last: a column of no row holds anything, and l or the scale in f may be NaN.
template <bool kMasked, int kN>
__device__ __forceinline__ void add_weights(const float* v, const float (&f)[kN], const float* nl, const uint32_t (&sees)[kN], float (&z)[kN][4]) {
#pragma unroll
    for (int c = 0; c < 32; c += 16) {
        float n[16], x[kN][16];
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const float4 y = *reinterpret_cast<const float4*>(nl + c + i);
            n[i] = y.x, n[i + 1] = y.y, n[i + 2] = y.z, n[i + 3] = y.w;
        }
#pragma unroll
        for (int i = 0; i < 16; i += 2)
#pragma unroll
            for (int w = 0; w < kN; ++w) fma2n(x[w][i], x[w][i + 1], v[32 * w + c + i], v[32 * w + c + i + 1], f[w], n[i], n[i + 1]);
#pragma unroll
        for (int w = 0; w < kN; ++w)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                x[w][i] = ex2_approx(x[w][i]);
                if (kMasked && !(sees[w] >> (c + i) & 1)) x[w][i] = 0.f;
            }
#pragma unroll
        for (int i = 0; i < 16; i += 2)
#pragma unroll
            for (int w = 0; w < kN; ++w) add2(z[w][i & 2], z[w][(i & 2) + 1], x[w][i], x[w][i + 1]);
    }
}

// A wait of few instructions, as there are some twenty of them: with wait_bar's clock at each, the roles' loops fit less well into the
// instruction cache.  It gives up after 2^22 looks, of some 1.4 us each while nothing comes: 6 s.
__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity, volatile int* abort_flag, int where) {
    bool ok = true;
    for (uint32_t n = 1; !mbar_try_wait(bar, parity); ++n) {
        if (n & 1023) continue;
        if (*abort_flag == 0 && n >> 22 == 0) continue;
        if (*abort_flag == 0) *abort_flag = where;
        ok = false;
        break;
    }
    return __all_sync(0xffffffffu, ok);
}

template <int D, int kKind>
__global__ void __launch_bounds__(Roles<kKind>::kThreads, 1) weights_tc_kernel(const __grid_constant__ Maps maps,
                                                                 const __grid_constant__ TcArgs p) {
    using L = Layout<D, kKind>;
    using W = Roles<kKind>;
    constexpr bool kSame = W::kSame;
    extern __shared__ __align__(1024) uint8_t raw[];
    uint8_t* smem = raw;
    if (smem_u32(smem) & 1023) {            // the swizzle goes by addresses: not met, as there is no other shared memory
        if (threadIdx.x == 0) p.err[blockIdx.x] = 4 | 9 << 8, p.cuts[blockIdx.x].first = 0;
        return;
    }
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
    const int ks = p.k_stages, qs = p.q_stages, rs = kSame ? 0 : (L::kTiles - ks - qs) * 2;
    uint64_t* k_full = bars;                    // [ks] a key tile is ready
    uint64_t* q_full = k_full + ks;             // [qs] a row tile
    uint64_t* r_full = q_full + qs;             // [rs] a tile of codes
    uint64_t* k_empty = bars + L::kMostStages;  // the MMAs have read it
    uint64_t* q_empty = k_empty + ks;
    uint64_t* r_empty = q_empty + qs;           // it is converted
    uint64_t* s_full = bars + 2 * L::kMostStages;       // [2] S of both key tiles, and the rows' normalisers, in buffer 0 or 1
    uint64_t* s_empty = s_full + 2;
    uint64_t* x_full = s_empty + 2;             // [2] the sums of key tile A or B that the other half has are there
    uint64_t* x_empty = x_full + 2;
    uint64_t* final_bar = x_empty + 2;
    uint8_t *k_ring = smem, *q_ring = smem + ks * L::kTileBytes, *r_ring = q_ring + qs * L::kTileBytes;
    volatile uint32_t* tmem_sh = reinterpret_cast<volatile uint32_t*>(final_bar + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_sh + 1);
    int* bad = reinterpret_cast<int*>(smem + L::kBad);                          // [2] impossible lengths; a page index out of range
    Walk* start = reinterpret_cast<Walk*>(bad + 2);
    float* ls = reinterpret_cast<float*>(smem + L::kL);                         // [2][128] -l
    float* halves = reinterpret_cast<float*>(smem + L::kHalf);                  // [2][128] tile A's sums of the second half, tile B's of the first

    const AttendProblem& a = p.w.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 32) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.q)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.k)) : "memory");
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < ks + qs + rs; ++i) {
            mbar_init(smem_u32(&bars[i]), !kSame && i < ks ? W::kConvert : 1);
            mbar_init(smem_u32(&bars[L::kMostStages + i]), i < ks + qs ? 1 : W::kConvert);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&s_full[i]), 2);             // the MMAs and the normalisers
            mbar_init(smem_u32(&s_empty[i]), W::kAdd);
            mbar_init(smem_u32(&x_full[i]), 4);
            mbar_init(smem_u32(&x_empty[i]), 4);
        }
        mbar_init(smem_u32(final_bar), 1);
        *abort_flag = 0;
        bad[0] = bad[1] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == W::kMma) {
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
    plan(p, reinterpret_cast<int*>(smem), reinterpret_cast<int64_t*>(smem + 4 * (kMaxSeqs + 2)), start, bad);
    Walk walk = *start;
    Segment sg;
    auto two_of = [&](const Segment& x) { return x.it.k0 + kKeys < x.s.kv; };       // tile B has keys

    if (warp < W::kAdd) {
        // ------------------------------ weights ------------------------------
        // bf16: a warp has 32 keys of each tile, and every other block of 32 columns, since a thread's two keys share what it reads of a
        // column.  8 bits: 32 keys of one tile and all columns, with nothing to exchange (whose items are mostly short: the last 32 of
        // 131072 tokens 88 us with the exchange, 77 without)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(W::kAddRegs));
        constexpr int kN = kSame ? 2 : 1;       // keys of a thread
        const int h = warp >> 2, row = (warp & 3) * 32 + lane;      // half of the blocks, or tile; key of the tile = TMEM lane
        const uint32_t s_at = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (kSame ? 0 : h * 128);
        const float f = a.scale * 1.4426950408889634f;
        int buf = 0;
        uint32_t ph_s = 0, ph_x = 0;
        bool ok = true;
        // the key of an item whose weight this thread writes (the first half tile A's, the second tile B's): the weight's place (-1:
        // none), what is there, and the scale of its row
        struct Place {
            int64_t at;
            float old, scale;
        };
        // the page that the next item will want, if it is of the same sequence
        int then_b = -1, then_q = 0, then_pg = 0;
        auto place = [&](const Segment& x) {
            Place r{-1, 0.f, 1.f};
            const int key = x.it.k0 + h * kKeys + row;
            if (key >= x.s.kv || key < first_seen(x.s, a.window)) return r;
            const int32_t* table = a.batch.table + (int64_t)x.b * a.batch.table_stride;
            const int q = a.page_of(key), pg = x.b == then_b && q == then_q ? then_pg : __ldg(table + q);
            if (key + kBlock < x.s.kv) {
                then_b = x.b;
                then_q = a.page_of(key + kBlock);
                then_pg = __ldg(table + then_q);
            }
            if ((unsigned)pg >= (unsigned)a.cache.pages) {
                bad[1] = 1;
                return r;
            }
            r.at = scale_offset(a.cache, pg, x.g, key - q * a.cache.page);
            if constexpr (!kSame) r.scale = __ldg(a.cache.k_scale + r.at);
            if (key < x.s.kv - x.s.n && p.w.decay != 0.f && x.to == x.it.tiles && x.from == 0) r.old = p.w.weights[r.at];
            return r;
        };
        bool more = walk.next(p, sg);
        Place cur = {-1, 0.f, 1.f};
        if (more) cur = place(sg);
        while (more && ok) {
            Segment next;
            const bool then = walk.next(p, next);
            Place ahead = {-1, 0.f, 1.f};
            if (then) ahead = place(next);
            const int ctx = sg.s.kv - sg.s.n;
            float fs[kN], total[kN];
#pragma unroll
            for (int w = 0; w < kN; ++w) fs[w] = kSame ? f : f * cur.scale, total[w] = 0.f;
            int t0 = sg.it.ta + sg.from * p.tpt;
            for (int i = sg.from; i < sg.to; ++i, t0 += p.tpt) {
                const int tokens = min(p.tpt, sg.it.tb - t0), rows = tokens * p.G;
                ok = wait_all(smem_u32(&s_full[buf]), ph_s, abort_flag, 22);
                if (!ok) break;
                tc_fence_after();
                const bool masked = sg.it.k0 + kBlock - 1 > ctx + t0 || (a.window && sg.it.k0 <= ctx + t0 + tokens - 1 - a.window) || rows % 32;
                const uint32_t at = s_at + buf * 256;
                const float* nl = ls + buf * 128;
                float z[kN][4];
#pragma unroll
                for (int w = 0; w < kN; ++w)
#pragma unroll
                    for (int k = 0; k < 4; ++k) z[w][k] = 0.f;
                // (The next columns on their way meanwhile took more registers than there are: a chunk of 4096 over 32768 903 us for 812.)
#pragma unroll 1
                for (int c = kSame ? h * 32 : 0; c < rows; c += 32 * kN) {
                    uint32_t sr[32 * kN];
                    tmem_ld32(at + c, sr);
                    if constexpr (kN == 2) tmem_ld32(at + 128 + c, sr + 32);
                    tmem_wait32(sr);
                    if constexpr (kN == 2) keep32(sr + 32);
                    const float* v = reinterpret_cast<const float*>(sr);
                    uint32_t sees[kN];              // the columns that see each key
                    if (masked) {
#pragma unroll
                        for (int w = 0; w < kN; ++w) {
                            const int ahead_of = sg.it.k0 + (kSame ? w : h) * kKeys + row - ctx - t0;
                            const int hi = a.window ? min(max(ahead_of + a.window, 0), tokens) * p.G : rows, lo = min(max(ahead_of, 0), tokens) * p.G;
                            sees[w] = low_bits(hi - c) & ~low_bits(lo - c);
                        }
                        add_weights<true, kN>(v, fs, nl + c, sees, z);
                    } else {
                        add_weights<false, kN>(v, fs, nl + c, sees, z);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&s_empty[buf]));
#pragma unroll
                for (int w = 0; w < kN; ++w) total[w] += (z[w][0] + z[w][1]) + (z[w][2] + z[w][3]);
                ph_s ^= buf;
                buf ^= 1;
            }
            if (!ok) break;
            float sum = total[0];
            if constexpr (kSame) {
                // The halves exchange their sums: the first half of the warps writes tile A's keys and the second half tile B's.  (No named
                // barrier: a warp that gives up a wait would leave the others at it.)
                ok = wait_all(smem_u32(&x_empty[1 - h]), ph_x ^ 1, abort_flag, 23);
                if (!ok) break;
                halves[(1 - h) * kKeys + row] = total[1 - h];
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&x_full[1 - h]));
                ok = wait_all(smem_u32(&x_full[h]), ph_x, abort_flag, 24);
                if (!ok) break;
                sum = h ? halves[kKeys + row] + total[1] : total[0] + halves[row];
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&x_empty[h]));
                ph_x ^= 1;
            }
            if (sg.from == 0 && sg.to == sg.it.tiles) {
                if (cur.at >= 0) p.w.weights[cur.at] = p.w.decay != 0.f ? sum + p.w.decay * cur.old : sum;
            } else {
                p.parts[((int64_t)blockIdx.x * 2 + (sg.from == 0 ? 1 : 0)) * kBlock + h * kKeys + row] = sum;
            }
            __syncwarp();
            sg = next;
            cur = ahead;
            more = then;
        }
    } else if (!kSame && warp < W::kMma) {
      if constexpr (!kSame) {
        // ------------------------------ conversion of 8-bit rows ------------------------------
        // A warp takes 32 rows of each tile.  Eight lanes read 128 bytes of codes, and a lane's 16 codes become two pieces of 16 bytes of
        // the bf16 tile.
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(W::kConvertRegs));
        constexpr int kPieces = D / 16, kRounds = kPieces;        // 16-byte pieces of a row of codes; of a lane
        const int r0 = (warp - W::kAdd) * 32;
        int st = 0, rst = 0;
        uint32_t ph = 1, ph_r = 0;
        bool ok = true;
        while (ok && walk.next(p, sg)) {
            for (int w = 0; w < (two_of(sg) ? 2 : 1); ++w) {
                ok = wait_all(smem_u32(&r_full[rst]), ph_r, abort_flag, 62);
                if (!ok) break;
                ok = wait_all(smem_u32(&k_empty[st]), ph, abort_flag, 61);
                if (!ok) break;
                const uint8_t* from = r_ring + rst * L::kCodeBytes + (r0 * kPieces + lane) * 16;
                uint8_t* tile = k_ring + st * L::kTileBytes;
                // (two rounds at a time: the roles' loops together do not fit into the instruction cache as it is)
#pragma unroll 2
                for (int y = 0; y < kRounds; ++y) {
                    const int i = y * 32 + lane, rr = r0 + i / kPieces, piece = i % kPieces;
                    const uint4 codes = *reinterpret_cast<const uint4*>(from + y * 512);
                    const uint32_t w4[4] = {codes.x, codes.y, codes.z, codes.w};
                    uint32_t o[8];
#pragma unroll
                    for (int k = 0; k < 4; ++k) pairs_of<kKind, true>(w4[k], o[2 * k], o[2 * k + 1]);
                    uint8_t* at = tile + (piece >> 2) * (kKeys * 128) + rr * 128;
                    const int c0 = 2 * (piece & 3);
                    *reinterpret_cast<uint4*>(at + ((c0 ^ (rr & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                    *reinterpret_cast<uint4*>(at + (((c0 + 1) ^ (rr & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&r_empty[rst]));
                if (++rst == rs) rst = 0, ph_r ^= 1;
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&k_full[st]));
                if (++st == ks) st = 0, ph ^= 1;
            }
        }
      }
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(W::kSingleRegs));
      if (warp == W::kMma) {
        // ------------------------------ MMAs ------------------------------
        const bool lead = elect_one();
        const uint64_t k_desc = smem_desc(smem_u32(k_ring)), q_desc = smem_desc(smem_u32(q_ring));
        const uint32_t k_lo = (uint32_t)k_desc, q_lo = (uint32_t)q_desc, d_hi = (uint32_t)(k_desc >> 32);
        int kst = 0, qst = 0;
        uint32_t ph_k = 0, ph_q = 0, buf = 0, ph_s = 1;         // a fresh barrier counts as completed for the odd parity
        bool ok = tmem == 0, first = true;
        while (ok && walk.next(p, sg)) {
            const bool two = two_of(sg);
            // the last tile's place is given back now: it is used again by an item that has the same
            if (!first && !sg.same) {
                commit_if(lead, smem_u32(&q_empty[qst]));
                if (++qst == qs) qst = 0, ph_q ^= 1;
            }
            first = false;
            const int k1 = kst + 1 == ks ? 0 : kst + 1;
            ok = wait_all(smem_u32(&k_full[kst]), ph_k, abort_flag, 32) &&
                 (!two || wait_all(smem_u32(&k_full[k1]), ph_k ^ (k1 == 0), abort_flag, 32));
            if (!ok) break;
            int left = sg.it.tb - (sg.it.ta + sg.from * p.tpt);
            for (int i = sg.from; i < sg.to; ++i, left -= p.tpt) {
                const uint32_t idesc = instr_desc((min(p.tpt, left) * p.G + 15) & ~15, false);
                if (!(sg.same && i == sg.from)) ok = wait_all(smem_u32(&q_full[qst]), ph_q, abort_flag, 31);
                ok = ok && wait_all(smem_u32(&s_empty[buf]), ph_s, abort_flag, 33);
                if (!ok) break;
                tc_fence_after();
                const uint32_t qb = q_lo + qst * (L::kTileBytes >> 4);
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    if (w == 1 && !two) break;
                    const uint32_t ka = k_lo + (w ? k1 : kst) * (L::kTileBytes >> 4), d = L::kS(w, 0) + buf * 256;
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t off = ((k >> 2) * (kKeys * 128) + (k & 3) * 32) >> 4;
                        mma_ss(lead, d, ka + off, qb + off, d_hi, idesc, k > 0);
                    }
                }
                commit_if(lead, smem_u32(&s_full[buf]));
                ph_s ^= buf;
                buf ^= 1;
                if (i + 1 < sg.to) {
                    commit_if(lead, smem_u32(&q_empty[qst]));
                    if (++qst == qs) qst = 0, ph_q ^= 1;
                }
            }
            if (!ok) break;
            for (int w = 0; w < (two ? 2 : 1); ++w) {
                commit_if(lead, smem_u32(&k_empty[kst]));
                if (++kst == ks) kst = 0, ph_k ^= 1;
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
      } else if (warp == W::kTma) {
        // ------------------------------ TMA ------------------------------
        // key tiles to their ring, codes to a ring of their own
        const sp_cache& c = a.cache;
        const int rows_tile = p.G * p.tpt, boxes = kKeys / p.box, mine = lane & 15;
        static_assert(kKeys / 8 <= 16, "boxes of a tile");
        int then_b = -1, then_q = 0, then_pg = 0;       // the page that the next item will want, if it is of the same sequence
        uint64_t *t_full = kSame ? k_full : r_full, *t_empty = kSame ? k_empty : r_empty;
        uint8_t* t_ring = kSame ? k_ring : r_ring;
        constexpr int kBytes = kSame ? L::kTileBytes : L::kCodeBytes;
        const int ts = kSame ? ks : rs;
        int kst = 0, qst = 0, k_loads = 0, q_loads = 0;
        uint32_t ph_k = 1, ph_q = 1;
        bool ok = true, first = true;
        while (ok && walk.next(p, sg)) {
            const int32_t* table = a.batch.table + (int64_t)sg.b * a.batch.table_stride;
            // this lane's box (lanes 0..15: of tile A, 16..31: of tile B): its page (pages: none, which loads zeros) and its first slot
            const int tok = sg.it.k0 + (lane >> 4) * kKeys + mine * p.box;
            int slot = 0, pg = (int)c.pages;
            if (mine < boxes && tok < sg.s.kv) {
                const int q = a.page_of(tok), t = sg.b == then_b && q == then_q ? then_pg : __ldg(table + q);
                if (tok + kBlock < sg.s.kv) {
                    then_b = sg.b;
                    then_q = a.page_of(tok + kBlock);
                    then_pg = __ldg(table + then_q);
                }
                if (tok + p.box > first_seen(sg.s, a.window)) {
                    if (t >= 0 && t < c.pages) pg = t, slot = tok - q * c.page;
                    else bad[1] = 1;
                }
            }
            for (int w = 0; w < (two_of(sg) ? 2 : 1); ++w) {
                ok = wait_all(smem_u32(&t_empty[kst]), ph_k, abort_flag, 41);
                if (!ok) break;
                const uint32_t bar = smem_u32(&t_full[kst]), at = smem_u32(t_ring) + kst * kBytes;
                if (lane == 0) mbar_expect_tx(bar, kBytes);
                __syncwarp();
                if (mine < boxes && lane >> 4 == w) {
                    if constexpr (kSame) {
#pragma unroll
                        for (int ch = 0; ch < L::kChunks; ++ch)
                            tma_load_4d(at + ch * (kKeys * 128) + mine * p.box * 128, &maps.k, ch * 64, slot, sg.g, pg, bar);
                    } else {
                        tma_load_4d(at + mine * p.box * D, &maps.k, 0, slot, sg.g, pg, bar);
                    }
                }
                ++k_loads;
                if (++kst == ts) kst = 0, ph_k ^= 1;
            }
            if (!ok) break;
            if (!first && !sg.same && ++qst == qs) qst = 0, ph_q ^= 1;
            first = false;
            for (int i = sg.from; i < sg.to; ++i) {
                if (!(sg.same && i == sg.from)) {
                    ok = wait_all(smem_u32(&q_empty[qst]), ph_q, abort_flag, 42);
                    if (!ok) break;
                    if (lane == 0) {
                        const uint32_t bar = smem_u32(&q_full[qst]);
                        mbar_expect_tx(bar, (uint32_t)(rows_tile * D * 2));
                        for (int ch = 0; ch < L::kChunks; ++ch)
                            tma_load_3d(smem_u32(q_ring) + qst * L::kTileBytes + ch * (kKeys * 128), &maps.q, ch * 64, sg.g * p.G,
                                        (int)(sg.s.row0 + sg.it.ta + i * p.tpt), bar);
                    }
                    ++q_loads;
                }
                if (i + 1 < sg.to && ++qst == qs) qst = 0, ph_q ^= 1;
            }
        }
        // an aborted CTA's copies land before it leaves: the last ones of each ring, one phase of a stage's barrier each
        if (lane == 0 && *abort_flag) {
            const unsigned long long t0 = global_ns();
            for (int k = 1; k <= min(k_loads, ts); ++k) {
                const int n = k_loads - k;
                while (!mbar_try_wait_suspend(smem_u32(&t_full[n % ts]), (uint32_t)(n / ts) & 1, 1000u) && global_ns() - t0 < kTimeoutNs) {}
            }
            for (int k = 1; k <= min(q_loads, qs); ++k) {
                const int n = q_loads - k;
                while (!mbar_try_wait_suspend(smem_u32(&q_full[n % qs]), (uint32_t)(n / qs) & 1, 1000u) && global_ns() - t0 < kTimeoutNs) {}
            }
        }
        __syncwarp();
      } else if (warp == W::kLse) {
        // ------------------------------ normalisers ------------------------------
        // they lie beside S: the same barriers say when the place is free and that they are there
        uint32_t buf = 0, ph_s = 1;
        bool ok = true;
        while (ok && walk.next(p, sg)) {
            for (int i = sg.from; i < sg.to; ++i) {
                const int t0 = sg.it.ta + i * p.tpt, rows = min(p.tpt, sg.it.tb - t0) * p.G;
                float l[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int r = lane + 32 * k, t = r / p.G;
                    l[k] = 0.f;         // columns of no row are masked
                    if (r < rows) l[k] = a.lse[(sg.s.row0 + t0 + t) * a.lse_stride_row + (sg.g * p.G + r - t * p.G) * a.lse_stride_head];
                }
                ok = wait_all(smem_u32(&s_empty[buf]), ph_s, abort_flag, 51);
                if (!ok) break;
                // a row that saw no token has the sum 0, whose logarithm is -inf, and gives nothing
#pragma unroll
                for (int k = 0; k < 4; ++k) ls[buf * 128 + lane + 32 * k] = l[k] == -INFINITY ? -INFINITY : l[k] * -1.4426950408889634f;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&s_full[buf]));
                ph_s ^= buf;
                buf ^= 1;
            }
        }
      }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (threadIdx.x == 0) p.err[blockIdx.x] = (bad[0] ? 1 : 0) | (bad[1] ? 2 : 0) | (*abort_flag ? 4 | *abort_flag << 8 : 0);
    if (warp == W::kMma)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

// Adds up the parts of the items that were cut, a thread a key: block c - 1 takes the item that CTA c's run begins in.  Block 0
// gathers the status as well.
__global__ void __launch_bounds__(kBlock) weights_join_kernel(const __grid_constant__ TcArgs p) {
    cudaGridDependencySynchronize();
    if (blockIdx.x == 0) {
        const int e = threadIdx.x < p.P ? p.err[threadIdx.x] : 0;
        const bool bad = __syncthreads_or(e & 3), gone = __syncthreads_or(e & 4);
        if (threadIdx.x == 0) {
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
    const AttendProblem& a = p.w.a;
    const int c = blockIdx.x + 1;
    const Cut q = p.cuts[c];
    if (!q.first) return;
    const Seq s = load_seq(a.batch, a.cache.page, q.b);
    const int key = q.k0 + threadIdx.x;
    if (key >= s.kv || key < first_seen(s, a.window)) return;
    const int pq = a.page_of(key), pg = a.batch.table[(int64_t)q.b * a.batch.table_stride + pq];
    if ((unsigned)pg >= (unsigned)a.cache.pages) return;
    const int64_t at = scale_offset(a.cache, pg, q.g, key - pq * a.cache.page);
    float old = 0.f, total = 0.f;
    if (key < s.kv - s.n && p.w.decay != 0.f) old = p.w.weights[at];
    // the first part begins with the item's first tile: slot 2 k + 1, the others 2 k
    for (int k = c - 1; k <= q.last; ++k) total += p.parts[((int64_t)k * 2 + (k == c - 1)) * kBlock + threadIdx.x];
    p.w.weights[at] = p.w.decay != 0.f ? total + p.w.decay * old : total;
}

struct Space {
    size_t err, cuts, parts, total;
};

Space carve(int P) {
    Space s;
    Carve c;
    s.err = c.take((size_t)P * sizeof(int));
    s.cuts = c.take((size_t)P * sizeof(Cut));
    s.parts = c.take((size_t)P * 2 * kBlock * sizeof(float));
    s.total = c.off;
    return s;
}

template <int D, int kKind>
sp_status launch(const Maps& maps, const TcArgs& p, cudaStream_t st) {
    SP_CUDA_TRY(cudaFuncSetAttribute(weights_tc_kernel<D, kKind>, cudaFuncAttributeMaxDynamicSharedMemorySize, (Layout<D, kKind>::kEnd)));
    weights_tc_kernel<D, kKind><<<p.P, Roles<kKind>::kThreads, (Layout<D, kKind>::kEnd), st>>>(maps, p);
    SP_LAUNCH_CHECK();
    return launch_early(weights_join_kernel, dim3((unsigned)std::max(1, p.P - 1)), kBlock, (size_t)0, st, p);
}

template <int D>
sp_status launch_kind(const Maps& maps, const TcArgs& p, cudaStream_t st) {
    switch (p.w.a.cache.kind) {
        case SP_CACHE_SAME: return launch<D, SP_CACHE_SAME>(maps, p, st);
        case SP_CACHE_E4M3: return launch<D, SP_CACHE_E4M3>(maps, p, st);
        default: return launch<D, SP_CACHE_INT8>(maps, p, st);
    }
}

}  // namespace

// Whether the cache and the group of heads are within the kernel's layouts.
bool weights_tc_supported(const sp_cache& c, const sp_batch& b, int G) {
    // (the join looks at a CTA's status per thread; the plan counts key blocks in 32 bits)
    if (b.B > kMaxSeqs || sm_count() < 2 || sm_count() > kBlock || (int64_t)b.B * b.table_width > ((int64_t)1 << 38) / c.page) return false;
    if (c.dtype != SP_BF16 || (c.d != 64 && c.d != 128) || G > 128) return false;
    if (c.kind != SP_CACHE_SAME &&
        (reinterpret_cast<uintptr_t>(c.k) | (uintptr_t)c.stride_page | (uintptr_t)c.stride_head | (uintptr_t)c.stride_slot) % 16 != 0)
        return false;                                                   // a tensor map wants multiples of 16 bytes
    if (c.page % 8 != 0) return false;                                  // boxes of 8 rows at least
    const int64_t limit = (int64_t)1 << 39;                             // tensor-map strides are below 2^40 bytes
    if (c.stride_slot >= limit / 2 || c.stride_head >= limit / 2 || c.stride_page >= limit / 2) return false;
    return !(c.H_kv > 1 && c.stride_head == 0) && !(c.pages > 1 && c.stride_page == 0);
}

size_t weights_tc_ws_bytes() { return carve(sm_count()).total; }

sp_status weights_tc_launch(const WeightsProblem& w, void* ws, cudaStream_t st) {
    const AttendProblem& a = w.a;
    TcArgs p;
    p.w = w;
    p.G = a.H / a.cache.H_kv;
    p.tpt = 128 / p.G;
    p.P = sm_count();
    p.box = std::min(128, a.cache.page & -a.cache.page);
    const bool same = a.cache.kind == SP_CACHE_SAME;
    const int tiles = 224 * 1024 / (kKeys * a.cache.d * 2);
    p.k_stages = same ? (a.cache.d == 128 ? 4 : 8) : (a.cache.d == 128 ? 3 : 6);
    // (what is left of an 8-bit cache's 224 KB are tiles of codes, two in the place of one; a second row tile in theirs: a chunk of 4096
    // over 32768 951 us for 940.  Two key tiles instead of three: the last 32 of 131072 81 us for 68.)
    p.q_stages = same ? tiles - p.k_stages : (a.cache.d == 128 ? 1 : 2);
    const Space s = carve(p.P);
    char* base = static_cast<char*>(ws);
    p.hdr = static_cast<WsHeader*>(ws);
    p.err = reinterpret_cast<int*>(base + s.err);
    p.cuts = reinterpret_cast<Cut*>(base + s.cuts);
    p.parts = reinterpret_cast<float*>(base + s.parts);
    Maps maps;
    const int64_t q_ext[3] = {a.cache.d, a.H, std::max<int64_t>(a.batch.T, 1)}, q_str[3] = {1, a.q.stride_head, a.q.stride_row};
    const int q_box[3] = {64, p.G, p.tpt};
    const int64_t c_ext[4] = {a.cache.d, a.cache.page, a.cache.H_kv, a.cache.pages};
    const int64_t c_str[4] = {1, a.cache.stride_slot, a.cache.stride_head, a.cache.stride_page};
    const int c_box[4] = {64, p.box, 1, 1};
    sp_status e;
    memset(&maps, 0, sizeof(maps));
    if ((e = encode(&maps.q, a.q.data, 3, q_ext, q_str, q_box)) != SP_OK) return e;
    const int r_box[4] = {a.cache.d, p.box, 1, 1};          // whole rows of codes, as they lie
    if ((e = same ? encode(&maps.k, a.cache.k, 4, c_ext, c_str, c_box) : encode(&maps.k, a.cache.k, 4, c_ext, c_str, r_box, true)) != SP_OK)
        return e;
    return a.cache.d == 64 ? launch_kind<64>(maps, p, st) : launch_kind<128>(maps, p, st);
}

}  // namespace sp
