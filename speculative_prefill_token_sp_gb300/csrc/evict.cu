// Cutting a cache: which tokens to keep, by the weight they have gathered, and moving those to the front of their pages.
//
// Choosing is a selection of the k largest of a sequence's weights.  A cluster of CTAs has one (sequence, KV head), each CTA an equal
// run of the tokens, in shared memory as integers of the same order.  Four passes over 8 bits each find the k-th largest: a histogram
// in each CTA, added up over the cluster through distributed shared memory.  The tokens above it, and the first of
// those that equal it, are written in order: every warp counts its run, and the counts' prefix sums say where it writes.
// The weights are read from memory once.
//
// Moving reads each kept row once and writes it once.  In place a row's new slot may be another's old one.  The list is ascending, so
// a row never moves back, and all rows of a round may be written once the rows of that round and of the ones before it have
// been read: the cluster that has a (sequence, KV head, side) reads a round into registers, meets at its barrier and writes.
// To other pages there is nothing to wait for.
#include "paged.cuh"

#include <cooperative_groups.h>

#include <algorithm>

namespace cg = cooperative_groups;

namespace sp {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBatch = 8;                   // tokens whose weights a thread has under way
constexpr int kMostHeld = 48 * 1024;        // tokens that a CTA holds in shared memory; more are read again in each pass

struct ChooseArgs {
    sp_cache c;
    sp_batch b;
    const float* weights;       // [pages, H_kv, page]
    int heads;                  // lists of a sequence: H_kv, or 1 for a list that all heads share
    int budget, first, last;
    int32_t* kept;
    int64_t stride_seq, stride_head;
    int64_t* n_kept;
    int held;                   // keys of shared memory
    int page_shift;             // log2 of the page, or -1
    WsHeader* hdr;
};

// What the choice goes by: integers in the order of the weights, 0 for NaN, which ranks below all of them.
__device__ __forceinline__ uint32_t key_of(float w) {
    const uint32_t u = __float_as_uint(w + 0.f);        // -0 is 0
    if (w != w) return 0;
    return u >> 31 ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kThreads) choose_kernel(const __grid_constant__ ChooseArgs p) {
    extern __shared__ uint32_t held[];
    __shared__ uint32_t hist[2][256];
    __shared__ uint32_t found[2];               // the digit, and how many keys are above it
    __shared__ uint32_t found_equal;
    __shared__ uint2 counts[kWarps], mine_all;  // keys above the threshold and equal to it, of each warp and of the CTA
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), r = (int)cluster.block_rank();
    const int item = blockIdx.x / C;
    if (item == p.b.B * p.heads) {
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
    const int lo = min(all, r * per), m = min(all, lo + per) - lo;          // this CTA's run
    const int32_t* table = p.b.table + (int64_t)b * p.b.table_stride;
    // The keys of tokens i, i + kThreads, ... (kBatch of them) of the run, their loads under way together: one after the other, a table
    // entry and a weight each, they took most of the kernel's time.
    auto load = [&](int i, uint32_t (&x)[kBatch]) {
        int pg[kBatch], slot[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int tok = p.first + lo + i + u * kThreads;
            const int q = p.page_shift >= 0 ? tok >> p.page_shift : (int)((unsigned)tok / (unsigned)p.c.page);
            pg[u] = i + u * kThreads < m ? __ldg(table + q) : -1;
            slot[u] = tok - q * p.c.page;
            x[u] = 0;
        }
        const bool one = p.heads > 1 || p.c.H_kv == 1;
        for (int g = one ? h : 0; g < (one ? h + 1 : p.c.H_kv); ++g) {
            float w[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                w[u] = (unsigned)pg[u] < (unsigned)p.c.pages ? __ldg(p.weights + scale_offset(p.c, pg[u], g, slot[u])) : __int_as_float(0x7fffffff);
#pragma unroll
            for (int u = 0; u < kBatch; ++u) x[u] = max(x[u], key_of(w[u]));
        }
    };
    const bool in_shared = m <= p.held;
    if (in_shared) {
        for (int i = threadIdx.x; i < m; i += kBatch * kThreads) {
            uint32_t x[kBatch];
            load(i, x);
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                if (i + u * kThreads < m) held[i + u * kThreads] = x[u];
        }
    }
    auto key = [&](int i) {
        if (in_shared) return held[i];
        const int tok = p.first + lo + i, q = (int)((unsigned)tok / (unsigned)p.c.page), pg = __ldg(table + q), slot = tok - q * p.c.page;
        if ((unsigned)pg >= (unsigned)p.c.pages) return 0u;
        if (p.heads > 1 || p.c.H_kv == 1) return key_of(__ldg(p.weights + scale_offset(p.c, pg, h, slot)));
        uint32_t top = 0;
        for (int g = 0; g < p.c.H_kv; ++g) top = max(top, key_of(__ldg(p.weights + scale_offset(p.c, pg, g, slot))));
        return top;
    };

    uint32_t prefix = 0;                        // of the k-th largest: its bits above `shift`
    int shift = 32;
    for (int pass = 0; pass < 4; ++pass) {
        uint32_t* mine = hist[pass & 1];
        if (threadIdx.x < 256) mine[threadIdx.x] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < m; i += kThreads) {
            const uint32_t x = key(i);
            if (pass == 0 || x >> shift == prefix) atomicAdd(&mine[(x >> (shift - 8)) & 255], 1u);
        }
        cluster.sync();
        uint32_t sum = 0;
        if (threadIdx.x < 256)
            for (int c = 0; c < C; ++c) sum += cluster.map_shared_rank(mine, c)[threadIdx.x];
        // (the other histogram is written next, and this one again only after all have met once more)
        __shared__ uint32_t totals[256];
        if (threadIdx.x < 256) totals[threadIdx.x] = sum;
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
                found_equal = totals[255 - 8 * lane - i];
            }
        }
        __syncthreads();
        prefix = prefix << 8 | found[0];
        k -= (int)found[1];
        shift -= 8;
        if (found_equal == (uint32_t)k) break;      // all that begin like this are kept: no need to tell them apart
    }

    // keys above the threshold are kept, and the first k that equal it; a warp has a run of its own
    const int seg = (((m + kWarps - 1) / kWarps) + 31) & ~31, from = min(m, warp * seg), to = min(m, from + seg);
    uint2 cnt = make_uint2(0, 0);
    for (int i = from + lane; i - lane < to; i += 32) {
        const uint32_t x = i < to ? key(i) >> shift : 0;
        cnt.x += __popc(__ballot_sync(0xffffffffu, i < to && x > prefix));
        cnt.y += __popc(__ballot_sync(0xffffffffu, i < to && x == prefix));
    }
    if (lane == 0) counts[warp] = cnt;
    __syncthreads();
    uint2 before = make_uint2(0, 0), total = make_uint2(0, 0);
    for (int w = 0; w < kWarps; ++w) {
        const uint2 c = counts[w];
        if (w < warp) before.x += c.x, before.y += c.y;
        total.x += c.x, total.y += c.y;
    }
    if (threadIdx.x == 0) mine_all = total;
    cluster.sync();
    for (int c = 0; c < r; ++c) {
        const uint2 o = *cluster.map_shared_rank(&mine_all, c);
        before.x += o.x, before.y += o.y;
    }
    for (int i = from + lane; i - lane < to; i += 32) {
        const uint32_t x = i < to ? key(i) >> shift : 0;
        const unsigned gt = __ballot_sync(0xffffffffu, i < to && x > prefix), eq = __ballot_sync(0xffffffffu, i < to && x == prefix);
        const unsigned below = (1u << lane) - 1;
        const uint32_t eq_rank = before.y + __popc(eq & below);
        if ((gt >> lane & 1) || ((eq >> lane & 1) && eq_rank < (uint32_t)k))
            kept[p.first + before.x + __popc(gt & below) + min(eq_rank, (uint32_t)k)] = p.first + lo + i;
        before.x += __popc(gt);
        before.y += __popc(eq);
    }
    cluster.sync();             // no CTA leaves while another reads its counts
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
    int ctas;                   // of an item
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

// A cluster's check of everything that the device arrays say: its threads take the entries of all lists in turn, several of them
// under way at once (one warp a list, an entry after the other, it took ten times as long as the moving).
__device__ __forceinline__ void check_kept(const KeepArgs& p) {
    __shared__ int bad;
    cg::cluster_group cluster = cg::this_cluster();
    if (threadIdx.x == 0) bad = 0;
    cluster.sync();
    int mine = 0;
    const int64_t lists = (int64_t)p.b.B * p.heads, step = (int64_t)cluster.num_blocks() * kMoveThreads;
    const int64_t me = (int64_t)cluster.block_rank() * kMoveThreads + threadIdx.x;
    for (int64_t b = me; b < p.b.B; b += step)
        if (!kept_of(p, load_seq(p.b, p.c.page, (int)b), (int)b).ok) mine = 1;
    constexpr int kBatch = 8;
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
    if (mine) atomicMax(cluster.map_shared_rank(&bad, 0), mine);
    cluster.sync();
    if (me == 0) {
        p.hdr->status = bad ? SP_EDEVICE : SP_OK;
        p.hdr->where = bad;     // 1: impossible lengths or counts, 2: a page index out of range, 3: a list that is not ascending
    }
}

template <typename Piece, bool kInPlace>
__global__ void __launch_bounds__(kMoveThreads) keep_kernel(const __grid_constant__ KeepArgs p) {
    const unsigned clusters = gridDim.x / cg::this_cluster().num_blocks();
    if (blockIdx.x / cg::this_cluster().num_blocks() == clusters - 1) {
        check_kept(p);
        return;
    }
    const int item = blockIdx.x / p.ctas, r = blockIdx.x - item * p.ctas;
    const int side = item & 1, bh = item >> 1, b = bh / p.c.H_kv, h = bh - b * p.c.H_kv;
    const Seq s = load_seq(p.b, p.c.page, b);
    const Kept k = kept_of(p, s, b);
    if (h == 0 && side == 0 && r == 0 && threadIdx.x == 0) p.kv_out[b] = k.ok ? k.base + k.n : p.b.kv_len[b];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane & ((1 << p.lg) - 1), grp = lane >> p.lg;
    const int rows_at_once = 32 >> p.lg, rows_w = rows_at_once * p.ahead / p.segs, rows_cta = kMoveWarps * rows_w;
    const int esize = p.c.kind == SP_CACHE_SAME ? (p.c.dtype == SP_BF16 ? 2 : 4) : 1, pieces = p.c.d * esize / (int)sizeof(Piece);
    char* data = static_cast<char*>(side ? p.c.v : p.c.k);
    float* scales = p.c.kind == SP_CACHE_SAME ? nullptr : side ? p.c.v_scale : p.c.k_scale;
    float* weights = side ? nullptr : p.weights;
    const int32_t* list = p.kept + b * p.stride_seq + (p.heads > 1 ? h : 0) * p.stride_head;
    const int32_t *table = p.b.table + b * p.b.table_stride, *to = p.to ? p.to + b * p.to_stride : table;

    for (int j0 = 0; j0 < k.n; j0 += p.ctas * rows_cta) {
        // this lane's row of the warp's: where it is and where it goes
        const int j = j0 + (r * kMoveWarps + warp) * rows_w + lane;
        int64_t src = -1, dst = -1, src_s = 0, dst_s = 0;
        if (lane < rows_w && j < k.n) {
            const int e = list[j];
            if (e >= 0 && e < k.from && (!kInPlace || e > j)) {
                int slot, slot2;
                const int pg = page_at(p, table, k.base + e, slot), pg2 = page_at(p, to, k.base + j, slot2);
                if (pg >= 0 && pg2 >= 0) {
                    src = row_offset(p.c, pg, h, slot) * esize;
                    dst = row_offset(p.c, pg2, h, slot2) * esize;
                    src_s = scale_offset(p.c, pg, h, slot);
                    dst_s = scale_offset(p.c, pg2, h, slot2);
                }
            }
        }
        Piece x[kAhead];
        float scale = 0.f, weight = 0.f;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (u < p.ahead) {
                const int q = u * rows_at_once + grp, row = p.segs == 2 ? q >> 1 : q, piece = sub + (p.segs == 2 ? (q & 1) << p.lg : 0);
                const int64_t at = __shfl_sync(0xffffffffu, src, row);
                if (at >= 0 && piece < pieces) x[u] = *reinterpret_cast<const Piece*>(data + at + piece * sizeof(Piece));
            }
        }
        if (src >= 0) {
            if (scales) scale = scales[src_s];
            if (weights) weight = weights[src_s];
        }
        if (kInPlace) cg::this_cluster().sync();
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (u < p.ahead) {
                const int q = u * rows_at_once + grp, row = p.segs == 2 ? q >> 1 : q, piece = sub + (p.segs == 2 ? (q & 1) << p.lg : 0);
                const int64_t at = __shfl_sync(0xffffffffu, dst, row);
                if (at >= 0 && piece < pieces) *reinterpret_cast<Piece*>(data + at + piece * sizeof(Piece)) = x[u];
            }
        }
        if (src >= 0) {
            if (scales) scales[dst_s] = scale;
            if (weights) weights[dst_s] = weight;
        }
    }
}

template <typename... A>
sp_status launch_cluster(void (*kern)(A...), unsigned grid, int threads, int cluster, size_t smem, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
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
    ChooseArgs a{c, b, weights, shared ? 1 : c.H_kv, (int)budget, (int)first, (int)last, kept, stride_seq, stride_head, n_kept, 0,
                 page_shift_of(c.page), static_cast<WsHeader*>(ws)};
    const int64_t items = (int64_t)b.B * a.heads, tokens = std::min<int64_t>((int64_t)b.table_width * c.page, (int64_t)1 << 30);
    const int cluster = power_below(std::min<int64_t>((tokens + 2047) / 2048, std::max<int64_t>(1, 2 * sm_count() / items)), 8);
    a.held = (int)std::min<int64_t>(kMostHeld, (tokens + cluster - 1) / cluster);
    const size_t smem = (size_t)a.held * 4;
    SP_CUDA_TRY(cudaFuncSetAttribute(choose_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostHeld * 4));
    return launch_cluster(choose_kernel, (unsigned)((items + 1) * cluster), kThreads, cluster, smem, st, a);
}

sp_status cache_keep_launch(const sp_cache& c, const sp_batch& b, const int32_t* kept, int heads, int64_t stride_seq,
                            int64_t stride_head, const int64_t* n_kept, int64_t most, bool drafted, const int32_t* to, int to_width,
                            int64_t to_stride, float* weights, int64_t* kv_out, void* ws, cudaStream_t st) {
    KeepArgs a{c, b, kept, heads, stride_seq, stride_head, n_kept, (int)most, drafted, to, to_width, to_stride, weights, kv_out,
               1, page_shift_of(c.page), 0, 1, kAhead, static_cast<WsHeader*>(ws)};
    const int bytes = c.d * (c.kind != SP_CACHE_SAME ? 1 : c.dtype == SP_BF16 ? 2 : 4);
    // the kinds of 8 bits may have rows at multiples of 8 bytes only
    const bool wide = bytes % 16 == 0 && (reinterpret_cast<uintptr_t>(c.k) | reinterpret_cast<uintptr_t>(c.v)) % 16 == 0 &&
                      (c.kind == SP_CACHE_SAME || ((uintptr_t)c.stride_page | (uintptr_t)c.stride_head | (uintptr_t)c.stride_slot) % 16 == 0);
    const int pieces = bytes / (wide ? 16 : 8);
    while ((1 << a.lg) < std::min(pieces, 32)) ++a.lg;
    a.segs = pieces > 32 ? 2 : 1;
    a.ahead = std::min(kAhead, a.segs << a.lg);         // a lane has the places of one row
    const int rows_cta = kMoveWarps * (32 >> a.lg) * a.ahead / a.segs;
    const int64_t items = 2 * (int64_t)b.B * c.H_kv;
    const int64_t useful = std::max<int64_t>(1, (most + rows_cta - 1) / rows_cta);
    // In place one cluster an item.  To other pages as many CTAs as there are rounds: the rows of a round are read at once, but one
    // round follows the other.
    const int cluster = power_below(to && (int64_t)b.B * heads * most > 4096 ? 8 : std::min<int64_t>(useful, std::max<int64_t>(1, 4 * sm_count() / items)), 8);
    a.ctas = to ? (int)std::min<int64_t>((useful + cluster - 1) / cluster, std::max<int64_t>(1, (1 << 24) / items)) * cluster : cluster;
    const unsigned grid = (unsigned)(items * a.ctas + cluster);
    void (*kern)(KeepArgs) = to ? (wide ? keep_kernel<uint4, false> : keep_kernel<uint2, false>)
                                : (wide ? keep_kernel<uint4, true> : keep_kernel<uint2, true>);
    return launch_cluster(kern, grid, kMoveThreads, cluster, 0, st, a);
}

}  // namespace sp
