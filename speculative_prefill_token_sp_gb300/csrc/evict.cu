// Cutting a cache: which tokens to keep, by the weight they have gathered, and moving those to the front of their pages.
//
// Choosing is a selection of the k largest of a sequence's weights.  A cluster of CTAs has one (sequence, KV head), each CTA an equal
// run of the tokens, whose weights its threads hold in registers as integers of the same order.  At most four passes over 8 bits each
// find the k-th largest: a histogram in each CTA, added up over the cluster through distributed shared memory.  The tokens above it,
// and the first of those that equal it, are written in order: every warp counts its part of the run, and the counts' prefix
// sums say where it writes.  The weights are read from memory once (again in each pass by a cluster that does not hold them).
// Eight lists of 131072 tokens cut to 8192: 20.5 us, 16 requests of 1K to 32K tokens with a list for all heads 12.1.  4 MB of weights are 1 us
// of it: the rest is latency, of the loads (table, then weight), of four exchanges over the cluster, and of the writing.
//
// Moving reads each kept row once and writes it once.  In place a row's new slot may be another's old one.  The list is ascending, so
// a row never moves back, and all rows of a round may be written once the rows of that round and of the ones before it have
// been read: the cluster that has a (sequence, KV head, side) reads a round into registers, meets at its barrier and writes.
// To other pages there is nothing to wait for.
// 8192 of 131072 tokens, 8 heads of 128, bf16: 13.8 us (67 MB moved: 4.9 TB/s); 16 requests of int8 11.6; the accepted tokens of 64
// trees 7.0, of which half is the check of the lists.
#include "paged.cuh"

#include <cooperative_groups.h>

#include <algorithm>

namespace cg = cooperative_groups;

namespace sp {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32, kMostCtas = 8;

// Both kernels are launched while the one before them in the stream runs, and wait here, before they read anything, for its end, as the
// next one may for theirs.  That hides the launch: 131072 tokens cut to 8192 a head 44.6 us to 40.7, 16 requests 47.4 to 43.4.
__device__ __forceinline__ void begin_early() {
    cudaTriggerProgrammaticLaunchCompletion();
    cudaGridDependencySynchronize();
}

struct ChooseArgs {
    sp_cache c;
    sp_batch b;
    const float* weights;       // [pages, H_kv, page]
    int heads;                  // lists of a sequence: H_kv, or 1 for a list that all heads share
    int budget, first, last;
    int32_t* kept;
    int64_t stride_seq, stride_head;
    int64_t* n_kept;
    int skip_pages, skip_slots; // 32 tokens on: 32 / page and 32 % page
    WsHeader* hdr;
};

// What the choice goes by: integers in the order of the weights, 1 for NaN, which ranks below all of them, as does a token without a page
// (0 is none of the tokens).
__device__ __forceinline__ uint32_t key_of(float w) {
    const uint32_t u = __float_as_uint(w + 0.f);        // -0 is 0
    return w != w ? 1u : u >> 31 ? ~u : u | 0x80000000u;
}

// One more in a bin, if `there`: a branch for each of a thread's weights took longer than the counting.
__device__ __forceinline__ void count_if(bool there, uint32_t bin) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %0, 0;\n\t@p red.shared.add.u32 [%1], 1;\n\t}\n" ::"r"((uint32_t)there), "r"(bin)
                 : "memory");
}

// kPer: weights that a thread holds.  Token i of a piece of the run is warp i / (32 kPer)'s, so a warp's tokens are consecutive.
template <int kPer>
__global__ void __launch_bounds__(kThreads) choose_kernel(const __grid_constant__ ChooseArgs p) {
    constexpr int kPiece = kThreads * kPer;
    __shared__ uint32_t hist[2][256], totals[256];
    __shared__ uint32_t found[3];               // the digit, how many keys are above it, and how many have it
    __shared__ uint2 counts[kWarps], mine_all;  // keys above the threshold and equal to it, of each warp and of the CTA
    begin_early();
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), r = (int)cluster.block_rank();
    const int item = (int)(blockIdx.x / C) - 1;
    if (item < 0) {
        if (r == 0) check_tokens(p.b, p.c, 0, true, p.hdr);
        return;
    }
    const int b = item / p.heads, h = item - b * p.heads, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Seq s = load_seq(p.b, p.c.page, b);
    const int n = min(s.kv, p.budget);
    int32_t* kept = p.kept + b * p.stride_seq + h * p.stride_head;
    if (r == 0 && h == 0 && threadIdx.x == 0) p.n_kept[b] = n;
    const int at = r * kThreads + threadIdx.x, step = C * kThreads;
    for (int j = n + at; j < p.budget; j += step) kept[j] = -1;
    if (n == s.kv) {                            // all of them
        for (int j = at; j < n; j += step) kept[j] = j;
        return;
    }
    for (int j = at; j < p.first; j += step) kept[j] = j;
    for (int j = at; j < p.last; j += step) kept[n - p.last + j] = s.kv - p.last + j;
    int k = n - p.first - p.last;               // of the tokens between
    if (k == 0) return;

    const int all = s.kv - p.first - p.last, per = (all + C - 1) / C;
    const int lo = min(all, r * per), m = min(all, lo + per) - lo, pieces = (m + kPiece - 1) / kPiece;     // this CTA's run
    const int32_t* table = p.b.table + (int64_t)b * p.b.table_stride;
    uint32_t x[kPer];
    // The keys of this thread's tokens of a piece (0 behind the run's end).  Sixteen loads of a kind are under way at once, without
    // branches: one token after the other, a table entry and a weight each, took most of the kernel's time.
    const int64_t per_page = (int64_t)p.c.H_kv * p.c.page;
    const bool one = p.heads > 1 || p.c.H_kv == 1;
    auto load = [&](int piece) {
        constexpr int kBatch = kPer < 16 ? kPer : 16;
        int i = piece * kPiece + warp * 32 * kPer + lane;
        int q = (int)((unsigned)(p.first + lo + i) / (unsigned)p.c.page), slot = p.first + lo + i - q * p.c.page;
#pragma unroll
        for (int u0 = 0; u0 < kPer; u0 += kBatch) {
            int pg[kBatch], at[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                pg[u] = __ldg(table + (i + 32 * u < m ? q : 0));
                at[u] = slot;
                q += p.skip_pages;
                slot += p.skip_slots;
                if (slot >= p.c.page) slot -= p.c.page, ++q;
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                if (i + 32 * u >= m || (unsigned)pg[u] >= (unsigned)p.c.pages) pg[u] = 0, at[u] = -1;       // reads another's weight
                x[u0 + u] = i + 32 * u < m ? 1u : 0u;
            }
            for (int g = one ? h : 0; g < (one ? h + 1 : p.c.H_kv); ++g) {
                const float* from = p.weights + (int64_t)g * p.c.page;
                float w[kBatch];
#pragma unroll
                for (int u = 0; u < kBatch; ++u) w[u] = __ldg(from + (pg[u] * per_page + max(at[u], 0)));
#pragma unroll
                for (int u = 0; u < kBatch; ++u)
                    if (at[u] >= 0) x[u0 + u] = max(x[u0 + u], key_of(w[u]));
            }
            i += 32 * kBatch;
        }
    };
    if (pieces == 1) load(0);

    uint32_t prefix = 0;                        // of the k-th largest: its bits above `shift`
    int shift = 32;
    for (int pass = 0; pass < 4; ++pass) {
        uint32_t* bins = hist[pass & 1];
        const uint32_t at_bins = (uint32_t)__cvta_generic_to_shared(bins);
        if (threadIdx.x < 256) bins[threadIdx.x] = 0;
        __syncthreads();
        for (int q = 0; q < pieces; ++q) {
            if (pieces > 1) load(q);
#pragma unroll
            for (int u = 0; u < kPer; ++u)
                count_if(pass == 0 || x[u] >> shift == prefix, at_bins + 4 * ((x[u] >> (shift - 8)) & 255));
        }
        if (C > 1) cluster.sync();
        else __syncthreads();
        if (threadIdx.x < 256) {
            uint32_t sum = 0;
            if (C > 1) {
                uint32_t of[kMostCtas];         // all on their way at once
#pragma unroll
                for (int c = 0; c < kMostCtas; ++c) of[c] = c < C ? cluster.map_shared_rank(bins, c)[threadIdx.x] : 0;
#pragma unroll
                for (int c = 0; c < kMostCtas; ++c) sum += of[c];
            }
            totals[threadIdx.x] = C > 1 ? sum : bins[threadIdx.x];
        }
        // (the other histogram is written next, and this one again only after all have met once more)
        __syncthreads();
        if (warp == 0) {                        // lane l: digits 255 - 8 l and the seven below it
            uint32_t of[8], sub = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                of[i] = totals[255 - 8 * lane - i];
                sub += of[i];
            }
            uint32_t incl = sub;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            uint32_t above = incl - sub;
            if (above < (uint32_t)k && incl >= (uint32_t)k) {
                int i = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (i == j && above + of[j] < (uint32_t)k) {
                        above += of[j];
                        ++i;
                    }
                found[0] = 255 - 8 * lane - i;
                found[1] = above;
                found[2] = totals[255 - 8 * lane - i];
            }
        }
        __syncthreads();
        prefix = prefix << 8 | found[0];
        k -= (int)found[1];
        shift -= 8;
        if (found[2] == (uint32_t)k) break;         // all that begin like this are kept: no need to tell them apart
    }

    // keys above the threshold are kept, and the first k that equal it (all of them, if there are no more: then they count as above)
    const bool alike = found[2] == (uint32_t)k;
    const uint32_t least = alike ? prefix : prefix + 1;
    auto flags = [&](int u, unsigned& gt, unsigned& eq) {
        gt = __ballot_sync(0xffffffffu, x[u] >> shift >= least);
        eq = alike ? 0 : __ballot_sync(0xffffffffu, x[u] >> shift == prefix);
    };
    auto count = [&] {
        uint2 c = make_uint2(0, 0);
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            unsigned gt, eq;
            flags(u, gt, eq);
            c.x += __popc(gt);
            c.y += __popc(eq);
        }
        return c;
    };
    uint2 mine = make_uint2(0, 0);              // of this warp
    for (int q = 0; q < pieces; ++q) {
        if (pieces > 1) load(q);
        const uint2 c = count();
        mine.x += c.x, mine.y += c.y;
    }
    if (lane == 0) counts[warp] = mine;
    __syncthreads();
    // of the warps before this one, and of all
    auto scan = [&](uint2& before, uint2& total) {
        before = total = make_uint2(0, 0);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const uint2 c = counts[w];
            if (w < warp) before.x += c.x, before.y += c.y;
            total.x += c.x, total.y += c.y;
        }
    };
    uint2 before, total, base = make_uint2(0, 0);
    scan(before, total);
    if (C > 1) {
        if (threadIdx.x == 0) mine_all = total;
        cluster.sync();
        if (lane < r) base = *cluster.map_shared_rank(&mine_all, lane);
#pragma unroll
        for (int o = kMostCtas / 2; o; o >>= 1) {
            base.x += __shfl_xor_sync(0xffffffffu, base.x, o);
            base.y += __shfl_xor_sync(0xffffffffu, base.y, o);
        }
        base.x = __shfl_sync(0xffffffffu, base.x, 0);
        base.y = __shfl_sync(0xffffffffu, base.y, 0);
        cluster.barrier_arrive();       // (waited for at the end: no CTA leaves while another reads its counts)
    }
    for (int q = 0; q < pieces; ++q) {
        if (pieces > 1) {                       // one piece after the other
            load(q);
            const uint2 c = count();
            __syncthreads();
            if (lane == 0) counts[warp] = c;
            __syncthreads();
            scan(before, total);
        }
        uint32_t above = base.x + before.x, equal = base.y + before.y;
        const unsigned below = (1u << lane) - 1;
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            unsigned gt, eq;
            flags(u, gt, eq);
            const uint32_t rank = equal + __popc(eq & below);
            if ((gt >> lane & 1) || ((eq >> lane & 1) && rank < (uint32_t)k))
                kept[p.first + above + __popc(gt & below) + min(rank, (uint32_t)k)] = p.first + lo + q * kPiece + warp * 32 * kPer + 32 * u + lane;
            above += __popc(gt);
            equal += __popc(eq);
        }
        base.x += total.x, base.y += total.y;
    }
    if (C > 1) cluster.barrier_wait();
}

constexpr int kMoveThreads = 256, kMoveWarps = kMoveThreads / 32;
constexpr int kAhead = 8;           // pieces that a lane has under way

struct KeepArgs {
    sp_cache c;
    sp_batch b;
    const int32_t* kept;
    int heads;                  // lists of a sequence
    int64_t stride_seq, stride_head;
    const int64_t* n_kept;
    int most;                   // entries of a list
    int drafted;                // the lists count from the sequence's first new token
    const int32_t* to;          // null: in place
    int to_width;
    int64_t to_stride;
    float* weights;             // may be null
    int64_t* kv_out;
    int pairs;                  // (head, side) pairs of an item
    int ctas;                   // of an item
    int checkers;               // CTAs in front of the others that check the lists
    int page_shift;             // log2 of the page, or -1
    int lg, segs;               // log2 of the lanes of a row, and how many pieces of its a lane has (1 or 2)
    int ahead;                  // rows under way: ahead * (32 >> lg) / segs of a warp
    WsHeader* hdr;
    __device__ __forceinline__ int page_of(int tok) const {
        return page_shift >= 0 ? tok >> page_shift : (int)((unsigned)tok / (unsigned)c.page);
    }
};

// How many tokens of the sequence are kept, and the token that the list and the new places count from.
struct Kept {
    int n, base, from;          // from: tokens that the list may name
    bool ok;
};
__device__ __forceinline__ Kept kept_of(const KeepArgs& p, const Seq& s, int b) {
    Kept k;
    k.base = p.drafted ? s.kv - s.n : 0;
    k.from = s.kv - k.base;
    const int64_t n = p.n_kept[b], width = p.to ? p.to_width : p.b.table_width;
    k.ok = s.ok && k.base >= 0 && n >= 0 && n <= p.most && n <= k.from && k.base + n <= width * p.c.page;
    k.n = k.ok ? (int)n : 0;
    return k;
}

__device__ __forceinline__ int page_at(const KeepArgs& p, const int32_t* table, int tok, int& slot) {
    const int q = p.page_of(tok), pg = __ldg(table + q);
    slot = tok - q * p.c.page;
    return (unsigned)pg < (unsigned)p.c.pages ? pg : -1;
}

// The check of everything that the device arrays say, by the first CTAs, each of which records what it found: threads take the entries
// of all lists in turn, several of them under way at once.  (One CTA took 20 us for 64 lists of 1024 to 8192 entries, longer than the moving.)
constexpr int kMostCheckers = 48;
__device__ __forceinline__ void check_kept(const KeepArgs& p) {
    int mine = 0;
    const int64_t lists = (int64_t)p.b.B * p.heads, step = (int64_t)p.checkers * kMoveThreads;
    const int64_t me = (int64_t)blockIdx.x * kMoveThreads + threadIdx.x;
    for (int64_t b = me; b < p.b.B; b += step)
        if (!kept_of(p, load_seq(p.b, p.c.page, (int)b), (int)b).ok) mine = 1;
    constexpr int kBatch = 4;
    for (int64_t i0 = me; i0 < lists * p.most; i0 += kBatch * step) {
        int e[kBatch], before[kBatch], from[kBatch], pg[kBatch], pg2[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int64_t i = i0 + u * step, l = divide(i, p.most);
            const int b = (int)divide(l, p.heads), h = (int)(l - (int64_t)b * p.heads), j = (int)(i - l * p.most);
            from[u] = -1;
            if (i >= lists * p.most) continue;
            const Seq s = load_seq(p.b, p.c.page, b);
            const Kept k = kept_of(p, s, b);
            if (j >= k.n) continue;
            const int32_t* list = p.kept + b * p.stride_seq + h * p.stride_head;
            from[u] = k.from;
            e[u] = __ldg(list + j);
            before[u] = j ? __ldg(list + j - 1) : -1;
            const int32_t *table = p.b.table + b * p.b.table_stride, *to = p.to ? p.to + b * p.to_stride : table;
            pg2[u] = __ldg(to + p.page_of(k.base + j));
            pg[u] = e[u] >= 0 && e[u] < k.from ? __ldg(table + p.page_of(k.base + e[u])) : 0;
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (from[u] < 0) continue;
            if (e[u] <= before[u] || e[u] >= from[u]) mine = max(mine, 3);
            else if ((unsigned)pg[u] >= (unsigned)p.c.pages || (unsigned)pg2[u] >= (unsigned)p.c.pages) mine = max(mine, 2);
        }
    }
    // 1: impossible lengths or counts, 2: a page index out of range, 3: a list that is not ascending
    const bool three = __syncthreads_or(mine == 3), two = __syncthreads_or(mine == 2), one = __syncthreads_or(mine == 1);
    if (threadIdx.x == 0) {
        p.hdr->aux[blockIdx.x] = three ? 3 : two ? 2 : one ? 1 : 0;
        if (blockIdx.x == 0) p.hdr->status = kSpread + p.checkers;
    }
}

template <typename Piece, bool kInPlace>
__global__ void __launch_bounds__(kMoveThreads) keep_kernel(const __grid_constant__ KeepArgs p) {
    begin_early();
    if (blockIdx.x < p.checkers) {
        check_kept(p);
        return;
    }
    const int cta = blockIdx.x - p.checkers, item = cta / p.ctas, r = cta - item * p.ctas;
    const int per_seq = (2 * p.c.H_kv + p.pairs - 1) / p.pairs, b = item / per_seq, first = (item - b * per_seq) * p.pairs;
    const Seq s = load_seq(p.b, p.c.page, b);
    const Kept k = kept_of(p, s, b);
    if (first == 0 && r == 0 && threadIdx.x == 0) p.kv_out[b] = k.ok ? k.base + k.n : p.b.kv_len[b];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane & ((1 << p.lg) - 1), grp = lane >> p.lg;
    const int rows_at_once = 32 >> p.lg, rows_w = rows_at_once * p.ahead / p.segs, rows_cta = kMoveWarps * rows_w;
    const int esize = p.c.kind == SP_CACHE_SAME ? (p.c.dtype == SP_BF16 ? 2 : 4) : 1, pieces = p.c.d * esize / (int)sizeof(Piece);
    const int32_t *table = p.b.table + b * p.b.table_stride, *to = p.to ? p.to + b * p.to_stride : table;
    // the item's rows, pair after pair (more than one pair only where their rows are few)
    const int rows = min(p.pairs, 2 * p.c.H_kv - first) * k.n;
    for (int j0 = 0; j0 < rows; j0 += p.ctas * rows_cta) {
        // this lane's row of the warp's: where it is and where it goes
        const int row = j0 + (r * kMoveWarps + warp) * rows_w + lane;
        char *src = nullptr, *dst = nullptr;
        float *scales = nullptr, *weights = nullptr;
        int64_t src_s = 0, dst_s = 0;
        if (lane < rows_w && row < rows) {
            const int pair = p.pairs > 1 ? row / k.n : 0, j = row - pair * k.n, side = (first + pair) & 1, h = (first + pair) >> 1;
            const int e = __ldg(p.kept + b * p.stride_seq + (p.heads > 1 ? h : 0) * p.stride_head + j);
            if (e >= 0 && e < k.from && (!kInPlace || e > j)) {
                int slot, slot2;
                const int pg = page_at(p, table, k.base + e, slot), pg2 = page_at(p, to, k.base + j, slot2);
                if (pg >= 0 && pg2 >= 0) {
                    char* data = static_cast<char*>(side ? p.c.v : p.c.k);
                    src = data + row_offset(p.c, pg, h, slot) * esize;
                    dst = data + row_offset(p.c, pg2, h, slot2) * esize;
                    src_s = scale_offset(p.c, pg, h, slot);
                    dst_s = scale_offset(p.c, pg2, h, slot2);
                    if (p.c.kind != SP_CACHE_SAME) scales = side ? p.c.v_scale : p.c.k_scale;
                    if (!side) weights = p.weights;
                }
            }
        }
        Piece x[kAhead];
        float scale = 0.f, weight = 0.f;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (u < p.ahead) {
                const int q = u * rows_at_once + grp, of = p.segs == 2 ? q >> 1 : q, piece = sub + (p.segs == 2 ? (q & 1) << p.lg : 0);
                const char* at = reinterpret_cast<const char*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), of));
                if (at && piece < pieces) x[u] = *reinterpret_cast<const Piece*>(at + piece * sizeof(Piece));
            }
        }
        if (scales) scale = scales[src_s];
        if (weights) weight = weights[src_s];
        if (kInPlace) cg::this_cluster().sync();
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (u < p.ahead) {
                const int q = u * rows_at_once + grp, of = p.segs == 2 ? q >> 1 : q, piece = sub + (p.segs == 2 ? (q & 1) << p.lg : 0);
                char* at = reinterpret_cast<char*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), of));
                if (at && piece < pieces) *reinterpret_cast<Piece*>(at + piece * sizeof(Piece)) = x[u];
            }
        }
        if (scales) scales[dst_s] = scale;
        if (weights) weights[dst_s] = weight;
    }
}

template <typename... A>
sp_status launch_cluster(void (*kern)(A...), unsigned grid, int threads, int cluster, size_t smem, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    SP_CUDA_TRY(cudaLaunchKernelEx(&cfg, kern, args...));
    SP_LAUNCH_CHECK();
    return SP_OK;
}

int page_shift_of(int page) {
    for (int i = 0; i < 31; ++i)
        if (page == 1 << i) return i;
    return -1;
}

// Largest power of two that is at most x (1 .. most).
int power_below(int64_t x, int most) {
    int c = 1;
    while (c * 2 <= x && c * 2 <= most) c *= 2;
    return c;
}

}  // namespace

sp_status cache_choose_launch(const sp_cache& c, const sp_batch& b, const float* weights, bool shared, int64_t budget, int64_t first,
                              int64_t last, int32_t* kept, int64_t stride_seq, int64_t stride_head, int64_t* n_kept, void* ws,
                              cudaStream_t st) {
    ChooseArgs a{c, b, weights, shared ? 1 : c.H_kv, (int)budget, (int)first, (int)last, kept, stride_seq, stride_head, n_kept,
                 32 / c.page, 32 % c.page, static_cast<WsHeader*>(ws)};
    const int64_t items = (int64_t)b.B * a.heads, tokens = std::min<int64_t>((int64_t)b.table_width * c.page, (int64_t)1 << 30);
    // (clusters of 16, of which the GPU does not hold eight at a time: 30 us for 20.5, eight lists of 131072)
    const int cluster = power_below(std::min<int64_t>((tokens + 2047) / 2048, std::max<int64_t>(1, 2 * sm_count() / items)), kMostCtas);
    void (*kern)(ChooseArgs) = tokens <= (int64_t)cluster * kThreads * 8 ? choose_kernel<8>
                               : tokens <= (int64_t)cluster * kThreads * 16 ? choose_kernel<16> : choose_kernel<32>;
    return launch_cluster(kern, (unsigned)((items + 1) * cluster), kThreads, cluster, 0, st, a);
}

sp_status cache_keep_launch(const sp_cache& c, const sp_batch& b, const int32_t* kept, int heads, int64_t stride_seq,
                            int64_t stride_head, const int64_t* n_kept, int64_t most, bool drafted, const int32_t* to, int to_width,
                            int64_t to_stride, float* weights, int64_t* kv_out, void* ws, cudaStream_t st) {
    KeepArgs a{c, b, kept, heads, stride_seq, stride_head, n_kept, (int)most, drafted, to, to_width, to_stride, weights, kv_out,
               1, 1, 1, page_shift_of(c.page), 0, 1, kAhead, static_cast<WsHeader*>(ws)};
    const int bytes = c.d * (c.kind != SP_CACHE_SAME ? 1 : c.dtype == SP_BF16 ? 2 : 4);
    // the kinds of 8 bits may have rows at multiples of 8 bytes only
    const bool wide = bytes % 16 == 0 && (reinterpret_cast<uintptr_t>(c.k) | reinterpret_cast<uintptr_t>(c.v)) % 16 == 0 &&
                      (c.kind == SP_CACHE_SAME || ((uintptr_t)c.stride_page | (uintptr_t)c.stride_head | (uintptr_t)c.stride_slot) % 16 == 0);
    const int pieces = bytes / (wide ? 16 : 8);
    while ((1 << a.lg) < std::min(pieces, 32)) ++a.lg;
    a.segs = pieces > 32 ? 2 : 1;
    a.ahead = std::min(kAhead, a.segs << a.lg);         // a lane has the places of one row
    const int rows_cta = kMoveWarps * (32 >> a.lg) * a.ahead / a.segs;
    // short lists share a CTA, as long as the rows of all fit into a round
    a.pairs = (int)std::min<int64_t>(2 * c.H_kv, std::max<int64_t>(1, rows_cta / std::max<int64_t>(1, most)));
    const int64_t items = (int64_t)b.B * ((2 * c.H_kv + a.pairs - 1) / a.pairs), useful = std::max<int64_t>(1, (most + rows_cta - 1) / rows_cta);
    // In place one cluster an item.  To other pages as many CTAs as there are rounds: the rows of a round are read at once, but one
    // round follows the other.
    const int cluster = to ? 1 : power_below(std::min<int64_t>(useful, std::max<int64_t>(1, 4 * sm_count() / items)), 8);
    a.ctas = to ? (int)std::min<int64_t>(useful, std::max<int64_t>(1, (1 << 28) / items)) : cluster;
    const int64_t entries = (int64_t)b.B * heads * most;
    a.checkers = (int)std::min<int64_t>(kMostCheckers, (entries + 4 * kMoveThreads - 1) / (4 * kMoveThreads) + cluster) / cluster * cluster;
    void (*kern)(KeepArgs) = to ? (wide ? keep_kernel<uint4, false> : keep_kernel<uint2, false>)
                                : (wide ? keep_kernel<uint4, true> : keep_kernel<uint2, true>);
    return launch_cluster(kern, (unsigned)(items * a.ctas + a.checkers), kMoveThreads, cluster, 0, st, a);
}

}  // namespace sp
