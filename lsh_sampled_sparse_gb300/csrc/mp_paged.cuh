// What the kernels of attention over a paged cache share: how its work is laid over the GPU.
#pragma once

#include "mp_internal.cuh"

namespace mp {

__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// ------------------------------------------------------------------------------------------------
// Attention of one query token per sequence.
//
// A unit is (sequence, KV head, chunk of up to NH query heads of its group); its keys come in tiles.
// The tiles of all units, laid end to end, are shared out evenly over as many CTAs as the GPU holds at
// once, by the lengths themselves: each CTA takes a run of tiles, whatever units they belong to. A
// unit that one CTA has to itself is written out by that CTA; the others' partial softmax states (at
// most two a CTA: the rest of a unit that began before, the beginning of one that ends after) go to
// the workspace and are joined by a second kernel in a fixed order. Few tiles (a.cluster) are shared
// out unit by unit instead, each to a cluster of up to eight CTAs, which joins its states itself.
// ------------------------------------------------------------------------------------------------
struct PArgs {
    const void* q;
    const void* keys;
    const void* values;
    PageRef pages;
    float* part;                                 // [CTA][2][NH][kPart]: o, m, l
    long long* before;                           // [B + 1] tiles of the sequences before (lengths only)
    float* out;
    int q_bf16, q_wide, B, Hq, Hkv, G, chunks, nh, n, ctas, tile;
    int cluster;                                 // CTAs a unit is shared out to, a cluster; 0: all
    int page_shift;                              // log2 of page_size, -1: no power of two
    float scale;                                 // of q.k, times log2 e
    int* status;                                 // index checks of the MP_CHECKS build
};
constexpr int kPart = kD + 4;

__device__ __forceinline__ int length_of(const PArgs& a, int b) {
    return a.pages.lengths ? max(0, min(a.n, a.pages.lengths[b])) : a.n;
}
__device__ __forceinline__ int tiles_of(const PArgs& a, int len) { return (len + a.tile - 1) / a.tile; }
// a / b of numbers that mostly fit 32 bits, where a division takes a fifth of the time
__device__ __forceinline__ long long quotient(long long a, int b) {
    if ((a >> 32) == 0) return static_cast<long long>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b));
    return a / b;
}
// `total` tiles shared out to CTAs: the first `more` of them take each + 1, the others `each`
struct Shares {
    long long each, more;
    int n;                                       // CTAs that have any
    __device__ __forceinline__ Shares(const PArgs& a, long long total) {
        n = static_cast<int>(min(static_cast<long long>(a.ctas), total));
        each = n > 0 ? quotient(total, n) : 0;
        more = total - each * n;
    }
    __device__ __forceinline__ long long first(int c) const {            // tile of CTA c
        return each * c + min(static_cast<long long>(c), more);
    }
    __device__ __forceinline__ int of(long long t) const {               // the CTA that has tile t
        const long long in_more = more * (each + 1);
        if (each >= 0x7fffffffll) return static_cast<int>(t < in_more ? t / (each + 1)
                                                                      : more + (t - in_more) / each);
        return static_cast<int>(t < in_more ? quotient(t, static_cast<int>(each) + 1)
                                            : more + quotient(t - in_more, static_cast<int>(each)));
    }
};
__device__ __forceinline__ int slot_of(const PArgs& a, int token) {
    return a.page_shift >= 0 ? token >> a.page_shift : token / a.pages.page_size;
}
// KV head of a unit of a sequence, and the first query head of its group that it takes
__device__ __forceinline__ int kv_head(const PArgs& a, int unit) {
    return a.chunks == 1 ? unit : unit / a.chunks;
}

// Where a CTA's run of tiles begins, and how many there are; walked through by next().
struct Walk {
    long long left;                              // tiles of the run from here on
    int b, unit, t, tiles, len;                  // unit of the sequence, its next tile, all its tiles
    __device__ __forceinline__ int here() const {
        return static_cast<int>(min(left, static_cast<long long>(tiles - t)));
    }
    // past `here` tiles: the next unit, if the run goes on
    __device__ __forceinline__ void next(const PArgs& a, int here) {
        left -= here;
        t = 0;
        if (left <= 0 || ++unit < a.Hkv * a.chunks) return;
        unit = 0;
        do {
            len = length_of(a, ++b);
            tiles = tiles_of(a, len);
        } while (tiles == 0);
    }
};

struct PlanSmem {
    long long warp_sum[32];
    Walk walk;
};
// The run of this CTA; every thread of the CTA calls it. CTA 0 leaves the sums for the join.
__device__ inline Walk plan_run(const PArgs& a, PlanSmem& s) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per_tile = a.Hkv * a.chunks;       // tiles of a sequence for each tile of its length
    Walk w;
    if (a.cluster) {                             // rank r of n takes tiles [r tiles / n, (r + 1) tiles / n)
        const int id = blockIdx.x / a.cluster, rank = blockIdx.x - id * a.cluster;
        w.b = id / per_tile;
        w.unit = id - w.b * per_tile;
        w.len = length_of(a, w.b);
        w.tiles = tiles_of(a, w.len);
        w.t = static_cast<int>(static_cast<uint32_t>(rank * w.tiles) / a.cluster);
        w.left = static_cast<int>(static_cast<uint32_t>((rank + 1) * w.tiles) / a.cluster) - w.t;
        return w;
    }
    const int c = blockIdx.x;
    if (!a.pages.lengths) {
        w.len = a.n;
        w.tiles = tiles_of(a, a.n);
        const long long unit_tiles = static_cast<long long>(per_tile) * a.B;
        const Shares share(a, unit_tiles * w.tiles);
        const long long lo = share.first(c), unit = quotient(lo, w.tiles);
        w.left = c < share.n ? share.first(c + 1) - lo : 0;
        w.t = static_cast<int>(lo - unit * w.tiles);
        w.b = static_cast<int>(quotient(unit, per_tile));
        w.unit = static_cast<int>(unit - static_cast<long long>(w.b) * per_tile);
        return w;
    }
    // a stretch of sequences a thread, their sums added up over the CTA
    const int each = (a.B + static_cast<int>(blockDim.x) - 1) / static_cast<int>(blockDim.x);
    const int b0 = min(a.B, tid * each), b1 = min(a.B, b0 + each);
    long long sum = 0;
    for (int b = b0; b < b1; ++b) sum += static_cast<long long>(per_tile) * tiles_of(a, length_of(a, b));
    long long incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) s.warp_sum[warp] = incl;
    if (tid == 0) s.walk.left = 0;
    __syncthreads();
    long long before = incl - sum, total = 0;
    for (int i = 0; i < static_cast<int>(blockDim.x) / 32; ++i) {
        if (i < warp) before += s.warp_sum[i];
        total += s.warp_sum[i];
    }
    const Shares share(a, total);
    const long long lo = share.first(c);
    const bool mine = c < share.n && lo >= before && lo < before + sum;
    if (c == 0 || mine) {
        for (int b = b0; b < b1; ++b) {
            if (c == 0) a.before[b] = before;
            const int len = length_of(a, b), tiles = tiles_of(a, len);
            const long long here = static_cast<long long>(per_tile) * tiles;
            if (mine && lo >= before && lo < before + here) {
                w.left = share.first(c + 1) - lo;
                w.b = b;
                w.unit = static_cast<int>(quotient(lo - before, tiles));
                w.t = static_cast<int>(lo - before - static_cast<long long>(w.unit) * tiles);
                w.tiles = tiles;
                w.len = len;
                s.walk = w;
            }
            before += here;
        }
        if (c == 0 && tid == static_cast<int>(blockDim.x) - 1) a.before[a.B] = total;
    }
    __syncthreads();
    return s.walk;
}

// Where a unit's state goes: out, where the CTA has all its tiles, else one of its two places
__device__ __forceinline__ float* part_of(const PArgs& a, bool from_start, int h) {
    return a.part + ((static_cast<size_t>(blockIdx.x) * 2 + (from_start ? 1 : 0)) * a.nh + h) * kPart;
}

// The states of a cluster's CTAs ([a.nh][kPart] each, in shared memory), joined in order by kD threads,
// each CTA some of the heads. Every thread of the cluster calls it after a barrier of its CTA; a state
// that holds nothing has m = -inf and zeros.
constexpr int kPagedMaxCluster = 8;
__device__ inline void join_cluster(const PArgs& a, const float* share, int b, int unit) {
    if (a.cluster > 1) cluster_barrier();
    const int g = kv_head(a, unit), h0 = (unit - g * a.chunks) * a.nh;
    const int tid = threadIdx.x, rank = static_cast<int>(blockIdx.x % a.cluster);
    if (tid < kD) {
        for (int h = rank; h < min(a.nh, a.G - h0); h += a.cluster) {
            const uint32_t at = smem_u32(share + h * kPart);
            float ms[kPagedMaxCluster], ls[kPagedMaxCluster], os[kPagedMaxCluster], M = -INFINITY;
#pragma unroll
            for (int r = 0; r < kPagedMaxCluster; ++r) {
                ms[r] = -INFINITY;
                ls[r] = os[r] = 0.0f;
                if (r < a.cluster) {
                    const uint32_t there = peer_address(at, r);
                    ms[r] = load_peer(there + 4 * kD);
                    ls[r] = load_peer(there + 4 * (kD + 1));
                    os[r] = load_peer(there + 4 * tid);
                }
                M = fmaxf(M, ms[r]);
            }
            const float from = M == -INFINITY ? 0.0f : M;
            float sum = 0.0f, out = 0.0f;
#pragma unroll
            for (int r = 0; r < kPagedMaxCluster; ++r) {
                const float c = exp2_fast(ms[r] - from);
                sum = fmaf(c, ls[r], sum);
                out = fmaf(c, os[r], out);
            }
            const size_t row = static_cast<size_t>(b) * a.Hq + g * a.G + h0 + h;
            if (mp_check(a.status, static_cast<long long>(row), static_cast<long long>(a.B) * a.Hq,
                         kSitePagedOut))
                a.out[row * kD + tid] = sum == 0.0f ? 0.0f : out * __frcp_rn(sum);
        }
    }
    if (a.cluster > 1) cluster_barrier();        // no CTA leaves while another reads from it
}

// Over a bf16 cache, on the tensor cores (mp_paged_tc.cu): query heads a unit takes for a group of G,
// its CTAs, the tokens of its tiles, and the launch.
int paged_tc_heads(int G);
constexpr int kPagedTcCtas = 152, kPagedTcTile = 128;
cudaError_t launch_paged_attention_tc(const PArgs& a, const mp_paged& cache, unsigned grid,
                                      cudaStream_t st);
cudaError_t prepare_paged_tc();

}  // namespace mp
