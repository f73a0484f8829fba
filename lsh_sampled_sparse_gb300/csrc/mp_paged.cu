// A paged K/V cache at full precision: tokens appended with their rotary positions applied on the
// way, and exact attention of single query tokens over the pages (of float32; those of bf16:
// mp_paged_tc.cu). The paper keeps K and V of one sequence in one piece: pages have no counterpart
// there. The layout is the one magicpig.h describes.
//
// The kernels are launched as dependents of what precedes them in the stream: their lives begin
// before it has written what they read. So no load here is a non-coherent one, which would promise
// that nobody writes its memory meanwhile; ordinary loads stay behind the wait.
#include <algorithm>

#include "mp_paged.cuh"

namespace mp {
namespace {

using Bf16 = __nv_bfloat16;

// ------------------------------------------------------------------------------------------------
// Append. Pair j of a row at position p turns by a = p inv_freq[j]; in half turns a / pi = 2 frac(p t)
// with t = inv_freq[j] / (2 pi). t mod 1 is taken to 64 fractional bits, p t mod 1 is then one
// wrapping 64-bit product, exact, and cos and sin are those of a number in [-1, 1] half turns: no loss
// at far positions, where p inv_freq in float32 is off by whole fractions of a turn.
// ------------------------------------------------------------------------------------------------
struct AppendArgs {
    mp_rows k, v, q;                             // strides in elements
    void* q_out;
    void* k_out;
    void* keys;
    void* values;
    const int32_t* positions;
    const int32_t* counts;
    const float* inv_freq;
    PageRef pages;
    int pairs, interleaved, B, Hq, Hkv, m, n_begin, tok_shift, tok_blocks;
    int* status;                                 // index checks of the MP_CHECKS build
};

constexpr int kAppThreads = 256;
constexpr int kRowLanes = 8;                     // lanes a row, 2 x 8 dims each
constexpr int kAppRows = kAppThreads / kRowLanes;
constexpr int kAppCtas = 6;                      // an SM: 40 registers a thread (4, 5 and 8 take as long)
// tokens a block has: of up to eight heads, whatever their number (5 sequences x 333 tokens of 12 + 3 + 3 heads: a
// quarter of the rows of 1260 CTAs stay empty, and 912 fit at once)
constexpr int kMaxToks = 4;
static_assert(kMaxToks * (kD / 2) == kAppThreads, "a thread an angle");

// 8 elements as they are in memory, two of them as floats
template <typename T>
struct Eight {
    uint4 v[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
    }
    __device__ __forceinline__ float2 two(int e) const {                 // elements 2 e, 2 e + 1
        const uint4& q = v[sizeof(T) == 2 ? 0 : e >> 1];
        if constexpr (sizeof(T) == 2) {
            const uint32_t w = e == 0 ? q.x : (e == 1 ? q.y : (e == 2 ? q.z : q.w));
            return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
        } else {
            return e & 1 ? make_float2(__uint_as_float(q.z), __uint_as_float(q.w))
                         : make_float2(__uint_as_float(q.x), __uint_as_float(q.y));
        }
    }
};
__device__ __forceinline__ uint32_t two_bf16(float2 x) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// x cos - y sin, y cos + x sin
__device__ __forceinline__ void turn_pair(float& x, float& y, float2 t) {
    const float x0 = x;
    x = fmaf(x0, t.x, -(y * t.y));
    y = fmaf(y, t.x, x0 * t.y);
}
// A lane's two pieces of a row, turned (cs: cos and sin of its eight pairs, two of them kRowLanes apart
// from the next two; NULL: as they are) and rounded to D, to dst and, unless it is NULL, to dst2 too.
template <typename T, typename D>
__device__ __forceinline__ void turn_and_store(const Eight<T>& a, const Eight<T>& b, const float4* cs,
                                               bool interleaved, D* dst, D* dst2, int da, int db) {
    auto turned = [&](int e, float2& x, float2& y) {
        x = a.two(e);
        y = b.two(e);
        if (!cs) return;
        if (interleaved) {
            const float4 t = cs[kRowLanes * (e >> 1)], u = cs[kRowLanes * (2 + (e >> 1))];
            turn_pair(x.x, x.y, e & 1 ? make_float2(t.z, t.w) : make_float2(t.x, t.y));
            turn_pair(y.x, y.y, e & 1 ? make_float2(u.z, u.w) : make_float2(u.x, u.y));
        } else {
            const float4 t = cs[kRowLanes * e];
            turn_pair(x.x, y.x, make_float2(t.x, t.y));
            turn_pair(x.y, y.y, make_float2(t.z, t.w));
        }
    };
    if constexpr (sizeof(D) == 2) {
        uint32_t wa[4], wb[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float2 x, y;
            turned(e, x, y);
            wa[e] = two_bf16(x);
            wb[e] = two_bf16(y);
        }
        const uint4 va = make_uint4(wa[0], wa[1], wa[2], wa[3]), vb = make_uint4(wb[0], wb[1], wb[2], wb[3]);
        if (dst) {
            *reinterpret_cast<uint4*>(dst + da) = va;
            *reinterpret_cast<uint4*>(dst + db) = vb;
        }
        if (dst2) {
            *reinterpret_cast<uint4*>(dst2 + da) = va;
            *reinterpret_cast<uint4*>(dst2 + db) = vb;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
            float2 x0, y0, x1, y1;
            turned(e, x0, y0);
            turned(e + 1, x1, y1);
            const float4 va = make_float4(x0.x, x0.y, x1.x, x1.y), vb = make_float4(y0.x, y0.y, y1.x, y1.y);
            if (dst) {
                *reinterpret_cast<float4*>(dst + da + 2 * e) = va;
                *reinterpret_cast<float4*>(dst + db + 2 * e) = vb;
            }
            if (dst2) {
                *reinterpret_cast<float4*>(dst2 + da + 2 * e) = va;
                *reinterpret_cast<float4*>(dst2 + db + 2 * e) = vb;
            }
        }
    }
}

// 2^64 (f / (2 pi) mod 1), toward zero, of a float f: its 24 bits times 2^64 / (2 pi), shifted by its
// exponent. Off by less than 1 + |f| (in units of 2^-64).
__device__ __forceinline__ uint64_t turn_of(float f) {
    constexpr uint64_t kPerTurn = 0x28be60db9391054aull;                 // 2^64 / (2 pi)
    const uint32_t bits = __float_as_uint(f), ex = (bits >> 23) & 255u;
    const uint64_t mant = (bits & 0x7fffffu) | (ex ? 0x800000u : 0u);
    const int down = 150 - static_cast<int>(ex ? ex : 1u);               // f = mant 2^-down
    const uint64_t lo = mant * kPerTurn, hi = __umul64hi(mant, kPerTurn);
    uint64_t t;
    if (down >= 64) t = down < 128 ? hi >> (down - 64) : 0ull;
    else if (down > 0) t = (lo >> down) | (hi << (64 - down));
    else t = down > -64 ? lo << -down : 0ull;
    return bits >> 31 ? 0ull - t : t;
}

// cos and sin of `part` 2^-64 turns. Rounded to 24 bits as a whole it is off by 2^-26 turns, 9.4e-8 radians, which
// a float32 row would show. kFine: the nearest quarter turn is taken off before the rest, an eighth of a turn at
// most, is rounded, off by 2^-28 turns. Rows that are bf16 in and out have 2^-9 of their own, and the few
// instructions cost 0.8 us of 40 (8192 tokens of 32 + 8 + 8 heads).
template <bool kFine>
__device__ __forceinline__ float2 cos_sin(long long part) {
    float s, c;
    if constexpr (!kFine) {
        sincospif(static_cast<float>(part) * 0x1p-63f, &s, &c);
        return make_float2(c, s);
    }
    const uint32_t hi = static_cast<uint32_t>(static_cast<uint64_t>(part) >> 32);
    const uint32_t quarters = (hi + 0x20000000u) >> 30;
    const uint64_t rest = static_cast<uint64_t>(part) - (static_cast<uint64_t>(quarters) << 62);
    sincospif(static_cast<float>(static_cast<long long>(rest)) * 0x1p-63f, &s, &c);
    const float x = quarters & 1 ? -s : c, y = quarters & 1 ? c : s;
    return quarters & 2 ? make_float2(-x, -y) : make_float2(x, y);
}

// A CTA takes 32 rows of up to 2^tok_shift tokens of one sequence (blockIdx.y: of which heads; the query
// heads come first, then the key heads, then the value heads), a row to eight lanes, all on their way
// before anything is known of the tokens. No CTA takes more than that: a loop over rows had less in flight
// than the rows of the CTAs that fit an SM (8192 tokens of 32 + 8 + 8 heads: 45 us, so 40, 5.5 TB/s).
template <typename T, typename C>
__global__ void __launch_bounds__(kAppThreads, kAppCtas) paged_append_kernel(const AppendArgs a) {
    // cos and sin of a token's pairs: pair 8 l + 2 j + i is half i of turn[token][j][l], so that the lanes of a
    // row read side by side
    __shared__ float4 turn[kMaxToks][4][kRowLanes];
    __shared__ long long place[kMaxToks];        // a token's row of the pool for KV head 0, or -1
    const int tid = threadIdx.x, lane = tid & (kRowLanes - 1), row = tid / kRowLanes;
    const int b = blockIdx.x / a.tok_blocks;
    const int i0 = static_cast<int>(blockIdx.x - static_cast<unsigned>(b) * a.tok_blocks) << a.tok_shift;
    const int i = row & ((1 << a.tok_shift) - 1), tok = i0 + i;
    const int h = (row >> a.tok_shift) + blockIdx.y * (kAppRows >> a.tok_shift);
    const int hk = h - a.Hq, hv = hk - a.Hkv;    // < 0: a query's row, a key's
    // this lane's two pieces of 8 dims: a pair's two halves, or whole pairs, or dims that stay
    const int turned = a.pairs / 8;              // lanes whose pieces turn
    const bool halves = !a.interleaved && lane < turned;
    const int da = halves ? 8 * lane : 16 * lane, db = halves ? a.pairs + 8 * lane : 16 * lane + 8;
    wait_for_predecessor();
    allow_dependents();
    // (behind the sequence's last token; of a step's few tokens the rows do not wait for the count)
    if (a.counts && a.tok_blocks > 1 && i0 >= a.counts[b]) return;
    Eight<T> xa, xb;
    const bool mine = tok < a.m && hv < a.Hkv;
    if (mine) {
        const mp_rows& from = hk < 0 ? a.q : (hv < 0 ? a.k : a.v);
        const T* src = static_cast<const T*>(from.data) + b * from.stride_b + tok * from.stride_m +
                       (hk < 0 ? h : (hv < 0 ? hk : hv)) * from.stride_h;
        xa.load(src + da);
        xb.load(src + db);
    }
    const int live = a.counts ? min(a.m, a.counts[b]) : a.m;
    const long long p0 = (a.positions ? static_cast<long long>(a.positions[b]) : a.n_begin) + i0;
    if (tid < 1 << a.tok_shift) {
        const long long p = p0 + tid;
        place[tid] = p >= 0 && p < static_cast<long long>(a.pages.n_slots) * a.pages.page_size
                         ? paged_row(a.pages, a.pages.table + static_cast<long long>(b) * a.pages.stride,
                                     static_cast<int>(p), a.Hkv, 0)
                         : -1;
    }
    if ((tid & 63) < a.pairs && tid >> 6 < 1 << a.tok_shift) {
        const long long part = static_cast<long long>(turn_of(a.inv_freq[tid & 63]) *
                                                      static_cast<uint64_t>(p0 + (tid >> 6)));
        reinterpret_cast<float2*>(&turn[tid >> 6][tid >> 1 & 3][tid >> 3 & 7])[tid & 1] =
            cos_sin<sizeof(T) == 4 || sizeof(C) == 4>(part);
    }
    __syncthreads();
    if (!mine || tok >= live) return;
    const float4* cs = hv < 0 && lane < turned ? &turn[i][0][lane] : nullptr;
    if (hk < 0) {
        const long long r = (static_cast<long long>(b) * a.Hq + h) * a.m + tok;
        if (mp_check(a.status, r, static_cast<long long>(a.B) * a.Hq * a.m, kSitePagedOut))
            turn_and_store<T, T>(xa, xb, cs, a.interleaved, static_cast<T*>(a.q_out) + r * kD, nullptr, da,
                                 db);
        return;
    }
    const long long in_pool = place[i] + static_cast<long long>(hv < 0 ? hk : hv) * a.pages.page_size;
    const long long in_rows = (static_cast<long long>(b) * a.Hkv + hk) * a.m + tok;
    C* dst = place[i] >= 0 && mp_check(a.status, in_pool, static_cast<long long>(a.pages.n_pages) * a.Hkv *
                                                              a.pages.page_size, kSitePagedRow)
                 ? static_cast<C*>(hv < 0 ? a.keys : a.values) + in_pool * kD : nullptr;
    C* dst2 = hv < 0 && a.k_out && mp_check(a.status, in_rows, static_cast<long long>(a.B) * a.Hkv * a.m,
                                            kSitePagedOut)
                  ? static_cast<C*>(a.k_out) + in_rows * kD : nullptr;
    turn_and_store<T, C>(xa, xb, cs, a.interleaved, dst, dst2, da, db);
}

// A float32 cache, on CUDA cores: a warp takes groups of four tokens of one page (pages hold multiples
// of eight), a lane four dims of each. Groups come through a ring of three in the warp's own piece of
// shared memory (cp.async: 12 KB in flight a warp), across the units of the run; a lane copies what it
// reads itself. The NH scores of four tokens are summed over the lanes by a reduce-scatter, which leaves
// a score to 8 / NH lanes, the softmax steps are lane-parallel, weights come back through
// shared memory. Bound by memory: 8 sequences x 8 heads x 8K tokens with 1, 2 and 4 query heads a KV head 85, 86
// and 87 us, 6.2 TB/s. Eight heads would hold 32 sums and 32 queries' dims a lane in 128 registers (113 us):
// more than four are mp_paged_mma.cu's.
constexpr int kSimtWarps = 8;
constexpr int kSimtThreads = 32 * kSimtWarps;
constexpr int kSimtShift = 5;                    // log2 of a tile's tokens: four a warp
constexpr int kSimtTile = 1 << kSimtShift;
static_assert(kSimtTile == 4 * kSimtWarps, "a group a warp");
constexpr int kRing = 3;
constexpr int kGroupBytes = 2 * 4 * kD * 4;      // four rows of K, four of V

template <int NH>
struct SimtSmem {
    // [warp][kRing] groups (a warp's state in the place of a group it is done with), weights and
    // factors of a group, m and l of the warps, a cluster's states, the plan
    static constexpr int kOffWeights = kSimtWarps * kRing * kGroupBytes;
    static constexpr int kOffMl = kOffWeights + kSimtWarps * 5 * NH * 4;
    static constexpr int kOffShare = kOffMl + kSimtWarps * NH * 8;
    static constexpr int kOffPlan = (kOffShare + NH * kPart * 4 + 15) / 16 * 16;
    static constexpr int kBytes = kOffPlan + static_cast<int>(sizeof(PlanSmem));
    static_assert(NH * kD * 4 <= kGroupBytes, "a warp's state takes the place of a group");
    static_assert(2 * (kBytes + 1024) <= 233472, "two CTAs an SM");
};

__device__ __forceinline__ void copy16_or_zero(uint32_t dst, const void* src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(live ? 16 : 0)
                 : "memory");
}

// A lane's four dims of a row or of a head's sums, in pairs, whose packed instructions halve the issue
// slots of the sums (8 sequences x 8 heads x 8K tokens, four query heads each: 92 -> 88 us).
struct Four {
    unsigned long long v[2];
    __device__ __forceinline__ void set(float4 x) {
        asm("mov.b64 %0, {%1, %2};" : "=l"(v[0]) : "f"(x.x), "f"(x.y));
        asm("mov.b64 %0, {%1, %2};" : "=l"(v[1]) : "f"(x.z), "f"(x.w));
    }
    __device__ __forceinline__ float4 get() const {
        float4 x;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(x.x), "=f"(x.y) : "l"(v[0]));
        asm("mov.b64 {%0, %1}, %2;" : "=f"(x.z), "=f"(x.w) : "l"(v[1]));
        return x;
    }
    static __device__ __forceinline__ unsigned long long twice(float f) {
        unsigned long long r;
        asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(f));
        return r;
    }
    __device__ __forceinline__ float dot(const Four& q) const {
        unsigned long long r;
        asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(v[0]), "l"(q.v[0]));
        asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(r) : "l"(v[1]), "l"(q.v[1]));
        float lo, hi;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(r));
        return lo + hi;
    }
    __device__ __forceinline__ void scale(float f) {
        const unsigned long long t = twice(f);
#pragma unroll
        for (int i = 0; i < 2; ++i) asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(v[i]) : "l"(t));
    }
    __device__ __forceinline__ void add(float f, const Four& x) {
        const unsigned long long t = twice(f);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(v[i]) : "l"(t), "l"(x.v[i]));
    }
};

template <int NH>
__global__ void __launch_bounds__(kSimtThreads, 2) paged_attention_simt_kernel(const PArgs a) {
    using S = SimtSmem<NH>;
    constexpr int kLanes = 8 / NH;               // lanes that hold a score
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    float* weights = reinterpret_cast<float*>(smem + S::kOffWeights) + warp * 5 * NH;
    float2* ml = reinterpret_cast<float2*>(smem + S::kOffMl);            // [warp][NH]
    float* share = reinterpret_cast<float*>(smem + S::kOffShare);
    const uint8_t* ring = smem + warp * kRing * kGroupBytes + 16 * lane;
    wait_for_predecessor();
    allow_dependents();
    Walk w = plan_run(a, *reinterpret_cast<PlanSmem*>(smem + S::kOffPlan));
    const int unit_b = w.b, unit = w.unit;       // of a cluster: its only ones
    if (a.cluster && w.left == 0) {              // fewer tiles than CTAs
        for (int i = tid; i < NH * kPart; i += kSimtThreads)
            share[i] = i % kPart == kD ? -INFINITY : 0.0f;
    }
    // ---- the group to copy next: its unit, its tile there, its slot's entry of the table, looked up
    // one group ahead; bits 4 i .. of `live`: how many tokens the group in place i of the ring holds
    Walk ahead = w;
    int ahead_here = w.left > 0 ? w.here() : 0, ahead_k = 0;
    uint32_t live = 0u;
    auto entry = [&]() {
        const int tok = (ahead.t + ahead_k) * kSimtTile + 4 * warp;
        return ahead.left > 0 && tok < ahead.len
                   ? page_in(a, a.pages.table + static_cast<long long>(ahead.b) * a.pages.stride, slot_of(a, tok))
                   : -1;
    };
    int page = entry();
    auto issue = [&](int place) {
        if (ahead.left > 0) {
            const int tok = (ahead.t + ahead_k) * kSimtTile + 4 * warp;
            const bool there = page >= 0 && page < a.pages.n_pages;
            const long long row = there ? (static_cast<long long>(page) * a.Hkv +
                                           kv_head(a, ahead.unit)) * a.pages.page_size +
                                              (tok - slot_of(a, tok) * a.pages.page_size)
                                        : 0;
            const int now = there && mp_check(a.status, row + 3,
                                              static_cast<long long>(a.pages.n_pages) * a.Hkv *
                                                  a.pages.page_size, kSitePagedRow)
                                ? min(4, ahead.len - tok) : 0;
            live = (live & ~(15u << (4 * place))) | (static_cast<uint32_t>(now) << (4 * place));
            const float* kp = static_cast<const float*>(a.keys) + row * kD + 4 * lane;
            const float* vp = static_cast<const float*>(a.values) + row * kD + 4 * lane;
            const uint32_t dst = smem_u32(ring) + place * kGroupBytes;
            if (now > 0) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    copy16_or_zero(dst + i * kD * 4, kp + (i < now ? i * kD : 0), i < now);
                    copy16_or_zero(dst + (4 + i) * kD * 4, vp + (i < now ? i * kD : 0), i < now);
                }
            }
            if (++ahead_k == ahead_here) {
                ahead.next(a, ahead_here);
                ahead_k = 0;
                if (ahead.left > 0) ahead_here = ahead.here();
            }
            page = entry();
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kRing; ++i) issue(i);
    int place = 0;
    while (w.left > 0) {
        const int here = w.here(), g = kv_head(a, w.unit), h0 = (w.unit - g * a.chunks) * NH;
        const int heads = min(NH, a.G - h0);
        const size_t row0 = static_cast<size_t>(w.b) * a.Hq + g * a.G + h0;
        Four q[NH], o[NH];
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            float x[4];
            load_query4(a, (row0 + min(h, heads - 1)) * kD + 4 * lane, x);
            q[h].set(make_float4(x[0], x[1], x[2], x[3]));
            o[h].set(make_float4(0.0f, 0.0f, 0.0f, 0.0f));
        }
        float m = -INFINITY, l = 0.0f;
        for (int k = 0; k < here; ++k) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
            const float4* group = reinterpret_cast<const float4*>(ring + place * kGroupBytes);
            const int now = (live >> (4 * place)) & 15u;
            if (now > 0) {
                float s[4 * NH];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    Four x;
                    x.set(group[i * (kD / 4)]);
#pragma unroll
                    for (int h = 0; h < NH; ++h) s[i * NH + h] = x.dot(q[h]);
                }
#pragma unroll
                for (int lv = 0; ((2 * NH) >> lv) >= 1; ++lv) {
                    const int off = 16 >> lv, keep = (2 * NH) >> lv;
                    const bool up = (lane & off) != 0;
#pragma unroll
                    for (int i = 0; i < keep; ++i) {
                        const float send = up ? s[i] : s[i + keep];
                        s[i] = (up ? s[i + keep] : s[i]) + __shfl_xor_sync(0xffffffffu, send, off);
                    }
                }
                float logit = s[0];
#pragma unroll
                for (int off = kLanes / 2; off >= 1; off >>= 1)
                    logit += __shfl_xor_sync(0xffffffffu, logit, off);
                logit = lane / (kLanes * NH) < now ? logit * a.scale : -INFINITY;
                float mt = logit;
#pragma unroll
                for (int off = 16; off >= kLanes * NH; off >>= 1)
                    mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, off));
                mt = fmaxf(m, mt);
                const float from = mt == -INFINITY ? 0.0f : mt;
                const float corr = exp2_fast(m - from), p = exp2_fast(logit - from);
                const bool moved = __any_sync(0xffffffffu, corr != 1.0f);
                m = mt;
                l = fmaf(l, corr, p);
                weights[lane / kLanes] = p;                              // token NH + head
                if (lane < kLanes * NH) weights[4 * NH + lane / kLanes] = corr;
                __syncwarp();
                // NH numbers, four a load where there are (a load costs what it returns to the lanes)
                auto factors = [&](const float* from, float (&f)[NH]) {
                    if constexpr (NH >= 4) {
#pragma unroll
                        for (int h = 0; h < NH; h += 4) {
                            const float4 x = *reinterpret_cast<const float4*>(from + h);
                            f[h] = x.x;
                            f[h + 1] = x.y;
                            f[h + 2] = x.z;
                            f[h + 3] = x.w;
                        }
                    } else {
#pragma unroll
                        for (int h = 0; h < NH; ++h) f[h] = from[h];
                    }
                };
                float f[NH];
                if (moved) {
                    factors(weights + 4 * NH, f);
#pragma unroll
                    for (int h = 0; h < NH; ++h) o[h].scale(f[h]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    Four x;
                    x.set(group[(4 + i) * (kD / 4)]);
                    factors(weights + i * NH, f);
#pragma unroll
                    for (int h = 0; h < NH; ++h) o[h].add(f[h], x);
                }
                __syncwarp();
            }
            if (k + 1 < here) {
                issue(place);
                place = place == kRing - 1 ? 0 : place + 1;
            }
        }
        // ---- the warps' states, each in the place of the group it took last, joined in order
#pragma unroll
        for (int off = 16; off >= kLanes * NH; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
        float4* state = reinterpret_cast<float4*>(smem + (warp * kRing + place) * kGroupBytes);
#pragma unroll
        for (int h = 0; h < NH; ++h)
            state[h * (kD / 4) + lane] = o[h].get();
        if (lane < kLanes * NH) ml[warp * NH + lane / kLanes] = make_float2(m, l);
        __syncthreads();
        const int e = tid & (kD - 1);
        for (int h = tid / kD; h < heads; h += kSimtThreads / kD) {
            float M = -INFINITY, L = 0.0f, O = 0.0f;
#pragma unroll
            for (int i = 0; i < kSimtWarps; ++i) M = fmaxf(M, ml[i * NH + h].x);
            const float from = M == -INFINITY ? 0.0f : M;
#pragma unroll
            for (int i = 0; i < kSimtWarps; ++i) {
                const float2 x = ml[i * NH + h];
                const float c = exp2_fast(x.x - from);
                L = fmaf(c, x.y, L);
                O = fmaf(c, reinterpret_cast<const float*>(smem + (i * kRing + place) *
                                                                      kGroupBytes)[h * kD + e], O);
            }
            if (a.cluster) {
                share[h * kPart + e] = O;
                if (e == 0) {
                    share[h * kPart + kD] = M;
                    share[h * kPart + kD + 1] = L;
                }
            } else if (here == w.tiles) {
                if (mp_check(a.status, static_cast<long long>(row0 + h),
                             static_cast<long long>(a.B) * a.Hq, kSitePagedOut))
                    a.out[(row0 + h) * kD + e] = over_sum(O, L);
            } else if (part_there(a, blockIdx.x, w.t == 0, h)) {
                float* p = part_of(a, w.t == 0, h);
                p[e] = O;
                if (e == 0) {
                    p[kD] = M;
                    p[kD + 1] = L;
                }
            }
        }
        __syncthreads();                         // the states are read: their places may be filled
        issue(place);
        place = place == kRing - 1 ? 0 : place + 1;
        w.next(a, here);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    zero_empty(a, tid, kSimtThreads);
    if (a.cluster) {
        __syncthreads();
        join_cluster(a, share, unit_b, unit);
    }
}

// The parts of the units that several CTAs have, joined in a fixed order, a query row a CTA: blockIdx.x + 1
// is the first of the CTAs whose run begins within the unit. Warp w folds parts w, w + kJoinWarps, ...,
// kJoinAhead of them loaded at once, four dims a lane; then the warps in order. A part that holds nothing
// has m = -inf and zeros; NaN passes through its zero factor. Bound by its latencies: 5.8 us by itself, 2 to
// 3 behind the attention, whose end its launch overlaps.
constexpr int kJoinWarps = 8, kJoinAhead = 4;
__global__ void __launch_bounds__(32 * kJoinWarps) paged_join_kernel(const PArgs a) {
    __shared__ __align__(16) float join[kJoinWarps][kPart];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x + 1;
    wait_for_predecessor();
    if (!begin_there(a, c) || !begin_there(a, a.ctas)) return;
    const int total = __ldcg(&a.begin[a.ctas].x);
    const int4 at = __ldcg(a.begin + c);         // b, unit, t, tiles
    const Shares share(a, total);
    if (c >= share.n || at.z == 0) return;
    const int t0 = share.first(c) - at.z, c0 = share.of(t0), c1 = share.of(t0 + at.w - 1);
    const int g = kv_head(a, at.y), hc = blockIdx.y, h = (at.y - g * a.chunks) * a.nh + hc;
    if (c0 != c - 1 || h >= a.G) return;
    const size_t row = static_cast<size_t>(at.x) * a.Hq + g * a.G + h;
    float M = -INFINITY, L = 0.0f;
    float4 O = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int s0 = c0 + warp; s0 <= c1; s0 += kJoinWarps * kJoinAhead) {
        float ms[kJoinAhead], ls[kJoinAhead];
        float4 os[kJoinAhead];
#pragma unroll
        for (int i = 0; i < kJoinAhead; ++i) {
            const int s = s0 + i * kJoinWarps;
            ms[i] = -INFINITY;
            ls[i] = 0.0f;
            os[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (s <= c1 && part_there(a, s, s == c0, hc)) {
                // the first share has the unit's beginning; it may have had another's end before
                const float* p = a.part + ((static_cast<size_t>(s) * 2 + (s == c0 ? 1 : 0)) * a.nh +
                                           hc) * kPart;
                ms[i] = __ldcg(p + kD);
                ls[i] = __ldcg(p + kD + 1);
                os[i] = __ldcg(reinterpret_cast<const float4*>(p) + lane);
            }
        }
        float mn = M;
#pragma unroll
        for (int i = 0; i < kJoinAhead; ++i) mn = fmaxf(mn, ms[i]);
        const float base = mn == -INFINITY ? 0.0f : mn;
        const float c = exp2_fast(M - base);
        M = mn;
        L *= c;
        O = make_float4(O.x * c, O.y * c, O.z * c, O.w * c);
#pragma unroll
        for (int i = 0; i < kJoinAhead; ++i) {
            const float x = exp2_fast(ms[i] - base);
            L = fmaf(x, ls[i], L);
            O = make_float4(fmaf(x, os[i].x, O.x), fmaf(x, os[i].y, O.y), fmaf(x, os[i].z, O.z),
                            fmaf(x, os[i].w, O.w));
        }
    }
    *reinterpret_cast<float4*>(&join[warp][4 * lane]) = O;
    if (lane == 0) {
        join[warp][kD] = M;
        join[warp][kD + 1] = L;
    }
    __syncthreads();
    const int e = threadIdx.x;
    if (e >= kD) return;
    M = -INFINITY;
#pragma unroll
    for (int i = 0; i < kJoinWarps; ++i) M = fmaxf(M, join[i][kD]);
    const float base = M == -INFINITY ? 0.0f : M;
    float Ls = 0.0f, Os = 0.0f;
#pragma unroll
    for (int i = 0; i < kJoinWarps; ++i) {
        const float c = exp2_fast(join[i][kD] - base);
        Ls = fmaf(c, join[i][kD + 1], Ls);
        Os = fmaf(c, join[i][e], Os);
    }
    if (mp_check(a.status, static_cast<long long>(row), static_cast<long long>(a.B) * a.Hq, kSitePagedOut))
        a.out[row * kD + e] = over_sum(Os, Ls);
}

constexpr int kSimtHeads = 4;                    // of a KV head, at most; more: mp_paged_mma.cu
constexpr int kSimtCtas = 2 * kPagedTcCtas;      // two an SM
// Tokens a CTA of a cluster may have more than its even share of all: they take as long as the second
// kernel, which the even shares' states need. One sequence x 8 heads, bf16, in a cluster or evenly: 2K
// tokens (a cluster's CTA has 128 more) 11.0 and 12.6 us, 8K (512) 18.5 and 19.4, 16K (1152) 27.0 and 24.3,
// 32K (2432) 43.7 and 34.0; float32, 16K 56.7 and 34.5.
constexpr int kJoinTokens = 512;
// Tokens of a cluster's CTA at most where sequences have lengths of their own: a long one among short ones
// leaves its CTAs alone with them. 19 sequences x 8 heads, bf16, one of 32K tokens and the others of 100:
// 272 us in clusters, 39 evenly; eight sequences, one of 4K: 25.3 and 15.8, all of 4K: 31.3 and 35.1.
constexpr int kRaggedTokens = 1024;
int simt_heads(int G) { return G <= 2 ? G : 4; }

typedef void (*PFn)(const PArgs);
template <int NH>
PFn simt(int* smem) {
    *smem = SimtSmem<NH>::kBytes;
    return paged_attention_simt_kernel<NH>;
}
PFn pick_simt(int nh, int* smem) {
    return nh == 1 ? simt<1>(smem) : (nh == 2 ? simt<2>(smem) : simt<4>(smem));
}

// How many clusters of so many CTAs the GPU holds at once, by whether the kernel is the tensor cores'
// (asked when the library is prepared on a device). A cluster's CTAs lie in one partition of the GPU, so
// that of clusters of eight CTAs of an SM each 15 fit, not 19.
constexpr int kMaxDevices = 64;
int g_clusters[kMaxDevices][2][kPagedMaxCluster + 1];

// The CTAs of the cluster that shares a unit of `tiles` tiles, 0 where all CTAs share all tiles: as many as
// leave all clusters running at once (two sequences x 8 heads x 8K tokens, bf16: 23.3 us, in clusters of
// eight, one of which would wait for the others to end, 33.5), unless a CTA then has kJoinTokens more
// than its even share.
int cluster_size(long long units, int tiles, int ctas, int tile_shift, bool ragged, const int* held) {
    int most = std::min(kPagedMaxCluster, tiles);
    while (most > 0 && held[most] < units) --most;
    if (most == 0) return 0;
    const int each = (tiles + most - 1) / most;
    const long long even = (units * tiles + ctas - 1) / ctas;
    if (ragged && each > kRaggedTokens >> tile_shift) return 0;
    return each - even <= kJoinTokens >> tile_shift ? (tiles + each - 1) / each : 0;
}

typedef void (*AppendFn)(const AppendArgs);
AppendFn pick_append(bool rows_bf16, bool cache_bf16) {
    if (rows_bf16) return cache_bf16 ? paged_append_kernel<Bf16, Bf16> : paged_append_kernel<Bf16, float>;
    return cache_bf16 ? paged_append_kernel<float, Bf16> : paged_append_kernel<float, float>;
}

PageRef page_ref(const mp_paged& c, const int32_t* lengths) {
    return PageRef{c.page_table, lengths, c.n_pages, c.page_size, c.n_slots, c.table_stride};
}

}  // namespace

cudaError_t launch_paged_append(const mp_rows& keys, const mp_rows& values, const mp_rows* q,
                                bool rows_bf16, const float* inv_freq, int rotary_dims,
                                bool interleaved, int B, int Hq, int Hkv, int m, int n_begin,
                                const int32_t* positions, const int32_t* counts,
                                const mp_paged& cache, void* q_out, void* keys_out, cudaStream_t st) {
    AppendArgs a;
    a.k = keys;
    a.v = values;
    a.q = q ? *q : keys;
    a.q_out = q_out;
    a.k_out = keys_out;
    a.keys = cache.keys;
    a.values = cache.values;
    a.positions = positions;
    a.counts = counts;
    a.inv_freq = inv_freq;
    a.pages = page_ref(cache, nullptr);
    a.pairs = inv_freq ? rotary_dims / 2 : 0;
    a.interleaved = interleaved;
    a.B = B;
    a.Hq = q ? Hq : 0;
    a.Hkv = Hkv;
    a.m = m;
    a.n_begin = n_begin;
    a.status = device_status_ptr();
    const int heads = a.Hq + 2 * Hkv;
    a.tok_shift = m >= 3 ? 2 : m - 1;            // up to kMaxToks tokens
    a.tok_blocks = (m + (1 << a.tok_shift) - 1) >> a.tok_shift;
    const int heads_a_cta = kAppRows >> a.tok_shift;
    const dim3 grid(static_cast<unsigned>(B) * a.tok_blocks, (heads + heads_a_cta - 1) / heads_a_cta);
    if (grid.y > 65535u) return cudaErrorInvalidValue;
    return launch_dependent(pick_append(rows_bf16, cache.dtype == MP_BF16), grid, dim3(kAppThreads), 0, st,
                            a);
}

size_t paged_attention_scratch_bytes(int Hq, int Hkv) {
    // of either kind of cache: who asks does not say which
    const int G = Hq / Hkv;
    const size_t parts = std::max(G <= kSimtHeads ? kSimtCtas * simt_heads(G) : 0, kPagedTcCtas * paged_tc_heads(G));
    return parts * 2 * kPart * sizeof(float) + (std::max(kSimtCtas, kPagedTcCtas) + 1) * sizeof(int4);
}

cudaError_t launch_paged_attention(const void* q, bool q_bf16, const mp_paged& cache, int B, int Hq,
                                   int Hkv, int n, const int32_t* lengths, float scale, float* out,
                                   void* workspace, size_t ws_bytes, cudaStream_t st) {
    PArgs a;
    a.q = q;
    a.keys = cache.keys;
    a.values = cache.values;
    a.pages = page_ref(cache, lengths);
    a.out = out;
    a.q_bf16 = q_bf16;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = Hq / Hkv;
    const bool tc = cache.dtype == MP_BF16, simt = !tc && a.G <= kSimtHeads;
    a.nh = simt ? simt_heads(a.G) : paged_tc_heads(a.G);
    a.chunks = (a.G + a.nh - 1) / a.nh;
    a.n = n;
    a.ctas = simt ? kSimtCtas : kPagedTcCtas;
    a.tile_shift = simt ? kSimtShift : kPagedTcShift;
    a.q_wide = (reinterpret_cast<uintptr_t>(q) & 15u) == 0u;
    a.page_shift = -1;
    for (int i = 3; i < 31; ++i)
        if (cache.page_size == 1 << i) a.page_shift = i;
    const int tiles = ((n - 1) >> a.tile_shift) + 1;
    const long long units = static_cast<long long>(B) * Hkv * a.chunks;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    a.cluster = cluster_size(units, tiles, a.ctas, a.tile_shift, lengths != nullptr, g_clusters[dev][simt ? 0 : 1]);
    a.scale = scale * kLog2E;
    a.status = device_status_ptr();
    a.ws_floats = static_cast<long long>(ws_bytes / sizeof(float));
    a.part = static_cast<float*>(workspace);
    a.begin = reinterpret_cast<int4*>(a.part + static_cast<size_t>(a.ctas) * 2 * a.nh * kPart);
    const unsigned grid = a.cluster ? static_cast<unsigned>(units) * a.cluster : a.ctas;
    int smem;
    const cudaError_t e = tc ? launch_paged_attention_tc(a, cache, grid, st)
                          : !simt ? launch_paged_attention_mma(a, grid, st)
                                  : launch_dependent(pick_simt(a.nh, &smem), dim3(grid), dim3(kSimtThreads),
                                                     smem, st, a, std::max(1, a.cluster));
    if (e != cudaSuccess || a.cluster) return e;
    // where every sequence has the same tiles, the shares may fall on whole units
    const long long total = units * tiles, shares = std::min<long long>(a.ctas, total);
    if (!lengths && total % shares == 0 && total / shares % tiles == 0) return e;
    if (shares < 2) return e;
    return launch_dependent(paged_join_kernel, dim3(static_cast<unsigned>(shares) - 1, std::min(a.nh, a.G)),
                            dim3(32 * kJoinWarps), 0, st, a);
}

cudaError_t prepare_paged() {
    cudaFuncAttributes fa;
    cudaError_t e;
    for (int i = 0; i < 4; ++i) {
        if ((e = cudaFuncGetAttributes(&fa, pick_append(i & 1, i & 2))) != cudaSuccess) return e;
    }
    for (int nh : {1, 2, 4}) {
        int smem;
        const PFn fn = pick_simt(nh, &smem);
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(fn, cudaFuncAttributePreferredSharedMemoryCarveout,
                                     cudaSharedmemCarveoutMaxShared);
        if (e != cudaSuccess) return e;
    }
    if ((e = prepare_paged_tc()) != cudaSuccess || (e = prepare_paged_mma()) != cudaSuccess) return e;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    for (int c = 1; c <= kPagedMaxCluster; ++c) {
        int smem;
        const PFn fn = pick_simt(4, &smem);      // all of them fit an SM twice, the tensor cores' once
        if ((e = max_clusters(fn, kSimtThreads, smem, c, &g_clusters[dev][0][c])) != cudaSuccess ||
            (e = paged_tc_clusters(c, &g_clusters[dev][1][c])) != cudaSuccess)
            return e;
    }
    return cudaFuncGetAttributes(&fa, paged_join_kernel);
}

}  // namespace mp
