// Trees of drafted tokens: which tokens a drafted token sees, its position, and the walk along those that the target agrees with.
//
// A tree is a parent per new token, before it in the sequence; a token sees its ancestors and itself, and its position is behind the
// cached tokens by its depth.  Both kernels touch a few KB, so their time is a launch and the latency of a few dependent loads.
// 64 sequences of up to 64 new tokens: 2.8 and 3.7 us (16 of 24: 2.2 and 2.0).
#include "paged.cuh"

#include <algorithm>

namespace sp {
namespace {

constexpr int kThreads = 256;

// The sequence as its arrays give it; there is no page to go by, so any length up to 2^30 will do.
__device__ __forceinline__ Seq load_drafted(const sp_batch& b, int i) { return load_seq(b, 1 << 30, i); }

// The parent of a new token: -1 for a root, which one that is none of the tokens before it is taken for.
__device__ __forceinline__ int parent_of(const int32_t* parent, int t) {
    const int u = __ldg(parent + t);
    return u >= 0 && u < t ? u : -1;
}

// One block's check of what the arrays say; the only writer of the status.
__device__ __forceinline__ void check_tree(const sp_batch& b, const int32_t* parent, int most, WsHeader* hdr) {
    __shared__ int bad;
    if (threadIdx.x == 0) bad = 0;
    __syncthreads();
    int mine = 0;
    // eight lanes a sequence: the sequences' loads depend on each other, so many of them are under way
    for (int i = threadIdx.x >> 3; i < b.B; i += kThreads / 8) {
        const Seq s = load_drafted(b, i);
        if (!s.ok || s.n > most) mine = max(mine, 1);
#pragma unroll 4
        for (int t = threadIdx.x & 7; t < s.n; t += 8) {
            const int u = __ldg(parent + s.row0 + t);
            if (u < -1 || u >= t) mine = 3;
        }
    }
    if (mine) atomicMax(&bad, mine);
    __syncthreads();
    if (threadIdx.x == 0) {
        hdr->status = bad ? SP_EDEVICE : SP_OK;
        hdr->where = bad;       // 1: impossible lengths or offsets, 3: a parent that is not before its child
    }
}

struct SeenArgs {
    sp_batch b;
    const int32_t* parent;
    uint32_t* seen;         // may be null
    int64_t stride;
    int words;
    int32_t* positions;     // may be null
    int per;                // blocks of a sequence
    WsHeader* hdr;
};

// A chain of n tokens takes n^3 / 64 steps up in all: 5 ms for 4096, but minutes for a prompt's length.
constexpr int kMostSeen = 4096;

// A thread has one word of a token's bits, and walks up from the token as far as that word goes; the first word's thread, which
// goes all the way, knows the depth.
__global__ void __launch_bounds__(kThreads) seen_kernel(const __grid_constant__ SeenArgs p) {
    if (blockIdx.x == gridDim.x - 1) {
        check_tree(p.b, p.parent, kMostSeen, p.hdr);
        return;
    }
    const int b = blockIdx.x / p.per;
    const Seq s = load_drafted(p.b, b);
    if (s.n > kMostSeen) return;
    const int32_t* parent = p.parent + s.row0;
    for (int64_t i = (int64_t)(blockIdx.x - b * p.per) * kThreads + threadIdx.x; i < (int64_t)s.n * p.words; i += (int64_t)p.per * kThreads) {
        const int t = (int)(i / p.words), k = (int)(i - (int64_t)t * p.words);
        uint32_t bits = 0;
        int depth = 0;
        for (int u = t; u >= 32 * k; u = parent_of(parent, u), ++depth)
            if (u >> 5 == k) bits |= 1u << (u & 31);
        if (p.seen) p.seen[(s.row0 + t) * p.stride + k] = bits;
        if (k == 0 && p.positions) p.positions[s.row0 + t] = s.kv - s.n + depth - 1;
    }
}

struct AcceptArgs {
    sp_batch b;
    const int32_t *parent, *draft, *target;
    int32_t* path;
    int64_t stride;
    int64_t* n_path;
    int32_t* next;          // may be null
    WsHeader* hdr;
};

constexpr int kWalkWarps = kThreads / 32;

// A warp has a sequence.  Children come after their parent, so one sweep over the tokens finds each next one: 32 at a time, those
// that hang on the last accepted token and are what the target says after it; the first of them is taken and the sweep
// goes on behind it.
__global__ void __launch_bounds__(kThreads) accept_kernel(const __grid_constant__ AcceptArgs p) {
    if (blockIdx.x == gridDim.x - 1) {
        check_tree(p.b, p.parent, INT32_MAX, p.hdr);
        return;
    }
    const int b = blockIdx.x * kWalkWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (b >= p.b.B) return;
    const Seq s = load_drafted(p.b, b);
    int32_t* path = p.path + (int64_t)b * p.stride;
    int cur = 0, n = 0, says = -1;
    if (s.n > 0) {
        says = p.target[s.row0];
        if (lane == 0) path[0] = 0;
        n = 1;
    }
    for (int t0 = 0; t0 < s.n; t0 += 32) {
        const int t = t0 + lane;
        const int up = t < s.n ? p.parent[s.row0 + t] : -2, is = t < s.n ? p.draft[s.row0 + t] : 0;
        const int then = t < s.n ? p.target[s.row0 + t] : 0;
        for (;;) {          // at most 32 times: each token found is behind the one before
            const unsigned found = __ballot_sync(0xffffffffu, up == cur && t > cur && is == says);
            if (!found) break;
            const int l = __ffs(found) - 1;
            cur = t0 + l;
            says = __shfl_sync(0xffffffffu, then, l);
            if (lane == 0) path[n] = cur;
            ++n;
        }
    }
    __syncwarp();
    for (int i = n + lane; i < p.b.max_new; i += 32) path[i] = -1;
    if (lane == 0) {
        p.n_path[b] = n;
        if (p.next) p.next[b] = says;
    }
}

}  // namespace

sp_status tree_seen_launch(const sp_batch& b, const int32_t* parent, uint32_t* seen, int64_t stride, int words, int32_t* positions,
                           void* ws, cudaStream_t st) {
    // enough blocks that a thread has few words, but not so many that a large batch of short sequences drowns in them
    const int64_t want = ((int64_t)b.max_new * words + kThreads - 1) / kThreads;
    const int per = (int)std::max<int64_t>(1, std::min<int64_t>(want, std::max(1, 8 * sm_count() / b.B)));
    const SeenArgs a{b, parent, seen, stride, words, positions, per, static_cast<WsHeader*>(ws)};
    seen_kernel<<<(unsigned)((int64_t)b.B * per + 1), kThreads, 0, st>>>(a);
    SP_LAUNCH_CHECK();
    return SP_OK;
}

sp_status tree_accept_launch(const sp_batch& b, const int32_t* parent, const int32_t* draft, const int32_t* target, int32_t* path,
                             int64_t stride, int64_t* n_path, int32_t* next, void* ws, cudaStream_t st) {
    const AcceptArgs a{b, parent, draft, target, path, stride, n_path, next, static_cast<WsHeader*>(ws)};
    accept_kernel<<<(unsigned)((b.B + kWalkWarps - 1) / kWalkWarps + 1), kThreads, 0, st>>>(a);
    SP_LAUNCH_CHECK();
    return SP_OK;
}

}  // namespace sp
