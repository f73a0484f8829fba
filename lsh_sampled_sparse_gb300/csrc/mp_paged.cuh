// What the kernels of attention over a paged cache share: how its work is laid over the GPU.
#pragma once

#include "mp_internal.cuh"

namespace mp {

// ------------------------------------------------------------------------------------------------
// Attention of one query token per sequence.
//
// A unit is (sequence, KV head, chunk of up to NH query heads of its group); its keys come in tiles.
// The tiles of all units, laid end to end, are shared out evenly over as many CTAs as the GPU holds at
// once, by the lengths themselves: each CTA takes a run of tiles, whatever units they belong to. A
// unit that one CTA has to itself is written out by that CTA; the others' partial softmax states (at
// most two a CTA: the rest of a unit that began before, the beginning of one that ends after) go to
// the workspace and are joined by a second kernel in a fixed order.
// ------------------------------------------------------------------------------------------------
struct PArgs {
    const void* q;
    const void* keys;
    const void* values;
    PageRef pages;
    float* part;                                 // [CTA][2][NH][kPart]: o, m, l
    long long* before;                           // [B + 1] tiles of the sequences before (lengths only)
    float* out;
    int q_bf16, B, Hq, Hkv, G, chunks, nh, n, ctas, tile;
    float scale;                                 // of q.k, times log2 e
    int* status;                                 // index checks of the MP_CHECKS build
};
constexpr int kPart = kD + 4;

__device__ __forceinline__ int length_of(const PArgs& a, int b) {
    return a.pages.lengths ? max(0, min(a.n, a.pages.lengths[b])) : a.n;
}
__device__ __forceinline__ int tiles_of(const PArgs& a, int len) { return (len + a.tile - 1) / a.tile; }
// How many CTAs share `total` tiles, the first tile of CTA c, the CTA that has tile t
__device__ __forceinline__ int shares_of(const PArgs& a, long long total) {
    return static_cast<int>(min(static_cast<long long>(a.ctas), total));
}
__device__ __forceinline__ long long first_tile(long long total, int shares, int c) {
    return total * c / shares;
}
__device__ __forceinline__ int share_with(long long total, int shares, long long t) {
    return static_cast<int>(((t + 1) * shares - 1) / total);
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
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = blockIdx.x;
    const int per_tile = a.Hkv * a.chunks;       // tiles of a sequence for each tile of its length
    if (!a.pages.lengths) {
        Walk w;
        w.len = a.n;
        w.tiles = tiles_of(a, a.n);
        const long long each = static_cast<long long>(per_tile) * w.tiles, total = each * a.B;
        const int shares = shares_of(a, total);
        const long long lo = first_tile(total, shares, c);
        w.left = c < shares ? first_tile(total, shares, c + 1) - lo : 0;
        w.b = static_cast<int>(lo / each);
        const long long in_b = lo - w.b * each;
        w.unit = static_cast<int>(in_b / w.tiles);
        w.t = static_cast<int>(in_b - static_cast<long long>(w.unit) * w.tiles);
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
    for (int w = 0; w < static_cast<int>(blockDim.x) / 32; ++w) {
        if (w < warp) before += s.warp_sum[w];
        total += s.warp_sum[w];
    }
    const int shares = shares_of(a, total);
    const long long lo = shares > 0 ? first_tile(total, shares, c) : 0;
    const bool mine = c < shares && lo >= before && lo < before + sum;
    if (c == 0 || mine) {
        for (int b = b0; b < b1; ++b) {
            if (c == 0) a.before[b] = before;
            const int len = length_of(a, b), tiles = tiles_of(a, len);
            const long long here = static_cast<long long>(per_tile) * tiles;
            if (mine && lo >= before && lo < before + here) {
                Walk w;
                w.left = first_tile(total, shares, c + 1) - lo;
                w.b = b;
                w.unit = static_cast<int>((lo - before) / tiles);
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

__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Over a bf16 cache, on the tensor cores (mp_paged_tc.cu): query heads a unit takes for a group of G,
// its CTAs, the tokens of its tiles, and the launch.
int paged_tc_heads(int G);
constexpr int kPagedTcCtas = 152, kPagedTcTile = 128;
cudaError_t launch_paged_attention_tc(PArgs a, const mp_paged& cache, cudaStream_t st);
cudaError_t prepare_paged_tc();

}  // namespace mp
