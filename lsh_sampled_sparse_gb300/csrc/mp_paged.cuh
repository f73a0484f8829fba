// What the kernels of attention over a paged cache share: how its work is laid over the GPU.
#pragma once

#include "mp_internal.cuh"

namespace mp {

// Weights, and factors of states: 2^x within 2^-22 of itself, the bound of exp2f too, but 0 below 2^-126, which
// is nothing beside the largest weight of a row, 1 (7 x 12/12 float32 heads x up to 3001 tokens: outputs off 64 bits
// by 3.3e-7, by 3.0e-7 where elementary operations in float32 make them)
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// A sum of values over the sum of their weights, which is 1 at least, or 0 where there are none (or NaN): by the
// reciprocal, within 2^-23 of itself, once an output
__device__ __forceinline__ float over_sum(float o, float sum) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(sum));
    return sum == 0.0f ? 0.0f : o * r;
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
    float* part;                                 // [CTA][2][nh][kPart]: o, m, l
    int4* begin;                                 // [CTA] where its run begins: b, unit, t, tiles; then the
                                                 // number of all tiles
    float* out;
    int q_bf16, q_wide, B, Hq, Hkv, G, chunks, nh, n, ctas;
    int tile_shift;                              // log2 of a tile's tokens
    int cluster;                                 // CTAs a unit is shared out to, a cluster; 0: all
    int page_shift;                              // log2 of page_size, -1: no power of two
    float scale;                                 // of q.k, times log2 e
    int* status;                                 // index checks of the MP_CHECKS build,
    long long ws_floats;                         // and what the workspace has for them
};
constexpr int kPart = kD + 4;

// Index checks of the MP_CHECKS build: a state of the workspace, an entry of begin, a slot of the table
__device__ __forceinline__ bool part_there(const PArgs& a, int cta, int half, int h) {
    return mp_check(a.status, ((2ll * cta + half) * a.nh + h + 1) * kPart - 1, a.ws_floats, kSitePagedOut);
}
__device__ __forceinline__ bool begin_there(const PArgs& a, int c) {
    return mp_check(a.status, 2ll * a.ctas * a.nh * kPart + 4 * (c + 1ll) - 1, a.ws_floats, kSitePagedOut);
}
__device__ __forceinline__ int page_in(const PArgs& a, const int32_t* slots, int slot) {
    return mp_check(a.status, slot, a.pages.n_slots, kSitePagedRow) ? slots[slot] : -1;
}

__host__ __device__ __forceinline__ int length_of(const PArgs& a, int b) {
    return a.pages.lengths ? max(0, min(a.n, a.pages.lengths[b])) : a.n;
}
__host__ __device__ __forceinline__ int tiles_of(const PArgs& a, int len) {
    return (len + (1 << a.tile_shift) - 1) >> a.tile_shift;
}
// `total` tiles (less than 2^31: a call's sizes see to that) shared out to CTAs: the first `more` of
// them take each + 1, the others `each`
struct Shares {
    int each, more, n;                           // n: CTAs that have any
    __host__ __device__ __forceinline__ Shares(const PArgs& a, int total) {
        n = min(a.ctas, total);
        each = n > 0 ? total / n : 0;
        more = total - each * n;
    }
    __host__ __device__ __forceinline__ int first(int c) const { return each * c + min(c, more); }  // tile of CTA c
    __host__ __device__ __forceinline__ int of(int t) const {                     // the CTA that has tile t
        const int in_more = more * (each + 1);
        return t < in_more ? t / (each + 1) : more + (t - in_more) / each;
    }
};
__device__ __forceinline__ int slot_of(const PArgs& a, int token) {
    return a.page_shift >= 0 ? token >> a.page_shift : token / a.pages.page_size;
}
// KV head of a unit of a sequence
__device__ __forceinline__ int kv_head(const PArgs& a, int unit) {
    return a.chunks == 1 ? unit : unit / a.chunks;
}

// Where a CTA's run of tiles begins, and how many there are; walked through by next().
struct Walk {
    int left;                                    // tiles of the run from here on
    int b, unit, t, tiles, len;                  // unit of the sequence, its next tile, all its tiles
    __host__ __device__ __forceinline__ int here() const { return min(left, tiles - t); }
    // past `here` tiles: the next unit, if the run goes on
    __host__ __device__ __forceinline__ void next(const PArgs& a, int here) {
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
    int warp_sum[32];
    Walk walk;
};
// The run of this CTA; every thread of the CTA calls it. Where it begins is left for the join.
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
        w.t = rank * w.tiles / a.cluster;
        w.left = (rank + 1) * w.tiles / a.cluster - w.t;
        return w;
    }
    const int c = blockIdx.x;
    if (!a.pages.lengths) {
        w.len = a.n;
        w.tiles = tiles_of(a, a.n);
        const Shares share(a, per_tile * a.B * w.tiles);
        const int lo = share.first(c), unit = lo / w.tiles;
        w.left = c < share.n ? share.first(c + 1) - lo : 0;
        w.t = lo - unit * w.tiles;
        w.b = unit / per_tile;
        w.unit = unit - w.b * per_tile;
        if (tid == 0 && begin_there(a, c)) {
            a.begin[c] = make_int4(w.b, w.unit, w.t, w.tiles);
            if (c == 0 && begin_there(a, a.ctas)) a.begin[a.ctas].x = per_tile * a.B * w.tiles;
        }
        return w;
    }
    // a stretch of sequences a thread, their sums added up over the CTA
    const int threads = static_cast<int>(blockDim.x);
    const int each = a.B <= threads ? 1 : (a.B + threads - 1) / threads;
    const int b0 = min(a.B, tid * each), b1 = min(a.B, b0 + each);
    const int len0 = b0 < b1 ? length_of(a, b0) : 0;             // mostly the only one
    int sum = per_tile * tiles_of(a, len0);
    for (int b = b0 + 1; b < b1; ++b) sum += per_tile * tiles_of(a, length_of(a, b));
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) s.warp_sum[warp] = incl;
    if (tid == 0) s.walk.left = 0;
    __syncthreads();
    int before = incl - sum, total = 0;
    for (int i = 0; i < threads / 32; ++i) {
        const int x = s.warp_sum[i];
        if (i < warp) before += x;
        total += x;
    }
    const Shares share(a, total);
    const int lo = share.first(c);
    const bool mine = c < share.n && lo >= before && lo < before + sum;
    if (mine) {
        int b = b0, len = len0, tiles = tiles_of(a, len0);
        for (; lo >= before + per_tile * tiles; tiles = tiles_of(a, len)) {
            before += per_tile * tiles;
            len = length_of(a, ++b);
        }
        w.left = share.first(c + 1) - lo;
        w.b = b;
        w.unit = (lo - before) / tiles;
        w.t = lo - before - w.unit * tiles;
        w.tiles = tiles;
        w.len = len;
        s.walk = w;
        if (begin_there(a, c)) a.begin[c] = make_int4(w.b, w.unit, w.t, w.tiles);
    }
    if (c == 0 && tid == 0 && begin_there(a, a.ctas)) a.begin[a.ctas].x = total;
    __syncthreads();
    return s.walk;
}

// Four query elements from element i on (a multiple of four), as floats
__device__ __forceinline__ void load_query4(const PArgs& a, size_t i, float (&x)[4]) {
    if (!a.q_wide) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = load_elem(a.q, a.q_bf16, i + e);
    } else if (a.q_bf16) {
        const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(a.q) + i);
        x[0] = __uint_as_float(v.x << 16);
        x[1] = __uint_as_float(v.x & 0xffff0000u);
        x[2] = __uint_as_float(v.y << 16);
        x[3] = __uint_as_float(v.y & 0xffff0000u);
    } else {
        const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + i);
        x[0] = v.x;
        x[1] = v.y;
        x[2] = v.z;
        x[3] = v.w;
    }
}

// Sequences of length 0 have no tiles: their rows, shared out to the CTAs, are zeroed by `threads` threads
__device__ inline void zero_empty(const PArgs& a, int thread, int threads) {
    if (a.cluster || !a.pages.lengths) return;
    for (int b = blockIdx.x; b < a.B; b += gridDim.x)
        if (length_of(a, b) == 0)
            for (int i = thread; i < a.Hq * kD / 4; i += threads)
                reinterpret_cast<float4*>(a.out + static_cast<size_t>(b) * a.Hq * kD)[i] =
                    make_float4(0.0f, 0.0f, 0.0f, 0.0f);
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
                a.out[row * kD + tid] = over_sum(out, sum);
        }
    }
    if (a.cluster > 1) cluster_barrier();        // no CTA leaves while another reads from it
}

// Over a bf16 cache, on the tensor cores (mp_paged_tc.cu): query heads a unit takes for a group of G,
// its CTAs, the tokens of its tiles, and the launch.
int paged_tc_heads(int G);
constexpr int kPagedTcCtas = 152;                // one an SM of a GB300: a constant, as a workspace's size
                                                 // is asked for on hosts without one
constexpr int kPagedTcShift = 7;
cudaError_t launch_paged_attention_tc(const PArgs& a, const mp_paged& cache, unsigned grid,
                                      cudaStream_t st);
cudaError_t prepare_paged_tc();
// Over a float32 cache, for more than four heads a KV head (mp_paged_mma.cu), with the same CTAs and tiles.
cudaError_t launch_paged_attention_mma(const PArgs& a, unsigned grid, cudaStream_t st);
cudaError_t prepare_paged_mma();
cudaError_t paged_tc_clusters(int size, int* n);     // clusters of that size that the GPU holds at once
template <typename Fn>
cudaError_t max_clusters(Fn fn, int threads, size_t smem, int size, int* n) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(size);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = size;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(n, fn, &cfg);
}

}  // namespace mp
