// Exact attention of single query tokens over a float32 paged cache, for more than four query heads a KV
// head, on the warps' matrix instructions.
//
// On CUDA cores every head costs every key's and value's dims again. Here a number is split once for all
// heads, x = hi + lo, hi rounded to tf32's 11 bits and lo the next 11 (2^-23 of x at most is left out), and
// a product is hi hi + hi lo + lo hi (lo lo, 2^-22 of it at most, adds nothing to the accuracy of the sums:
// 3.7e-7 of the output's norm either way, 2.9e-7 on CUDA cores). A warp works by itself on tiles of 16
// tokens: scores S = K Q^T with the tokens as the 16 rows of m16n8k8 and eight heads as its columns, values
// O = V^T P with 16 dims as rows. Which dims a step of S multiplies, and which stand in a row of O, is chosen
// so that a lane's share of a row of K or V is whole 16-byte pieces. tcgen05 was not taken: its operands
// come from shared memory, so that both parts of every number would be written there and read again.
//
// 8 sequences x 8 heads x 8K tokens with 8 and 16 query heads each: 98 and 115 us (5.5 and 4.7 TB/s; on CUDA
// cores 113 and 202, with four heads 87). What is left over the memory's 79 us are the warps' own chains,
// two warps a scheduler that issue in 38% of the cycles; a matrix product more for lo lo costs 2 and 15 us.
//
// The matrix unit's sums round toward zero: they are kept short (S: 32 dims; O: a tile, from zero) and
// joined in float32.
//
// A warp's keys and values come through a ring of three places of 8 KB (cp.async; keys of a tile, its values,
// the next keys), across the units of the CTA's run (mp_paged.cuh). Rows that are not there are zeros.
#include <algorithm>

#include "mp_paged.cuh"

namespace mp {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kTokens = 16;                      // of a warp's tile
static_assert(kTokens * kWarps == 1 << kPagedTcShift, "the tiles of the CTA");
constexpr int kRing = 3, kPlace = kTokens * kD * 4;
constexpr int kPitch = 20;                       // tokens of a head's weights, apart without bank conflicts

template <int NT>                                // 8 NT heads
struct MmaSmem {
    static constexpr int kHeads = 8 * NT;
    static constexpr int kOffWeights = kWarps * kRing * kPlace;          // [warp][head][kPitch]
    static constexpr int kOffMl = kOffWeights + kWarps * kHeads * kPitch * 4;
    // two column tiles: queries [16 steps][NT][lane] of hi, hi, lo, lo; and a cluster's states
    static constexpr int kOffQ = kOffMl + kWarps * kHeads * 8;
    static constexpr int kQ = NT == 2 ? 16 * NT * 32 * 16 : kHeads * kPart * 4;
    static constexpr int kOffPlan = kOffQ + kQ;
    static constexpr int kBytes = kOffPlan + static_cast<int>(sizeof(PlanSmem));
    static_assert(kHeads * kD * 4 <= kPlace, "a warp's state takes the place of a tile");
    static_assert(kHeads * kPart * 4 <= kQ && kBytes <= 232448, "shared memory");
};

__device__ __forceinline__ void copy16_or_zero(uint32_t dst, const void* src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(live ? 16 : 0)
                 : "memory");
}
constexpr uint32_t kTf32 = 0xffffe000u;          // the bits of a float that tf32 has
__device__ __forceinline__ void two_parts(float x, uint32_t& hi, uint32_t& lo) {
    hi = (__float_as_uint(x) + 0x1000u) & kTf32;
    lo = __float_as_uint(x - __uint_as_float(hi)) & kTf32;
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                 "{%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int NT>
__global__ void __launch_bounds__(kThreads, 1) paged_attention_mma_kernel(const PArgs a) {
    using S = MmaSmem<NT>;
    constexpr int NH = S::kHeads;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;       // of a fragment: row or column, step or column pair
    float* weights = reinterpret_cast<float*>(smem + S::kOffWeights) + warp * NH * kPitch;
    float2* ml = reinterpret_cast<float2*>(smem + S::kOffMl);            // [warp][NH]
    uint4* queries = reinterpret_cast<uint4*>(smem + S::kOffQ);
    float* share = reinterpret_cast<float*>(smem + S::kOffQ);
    uint8_t* ring = smem + warp * kRing * kPlace;
    wait_for_predecessor();
    allow_dependents();
    Walk w = plan_run(a, *reinterpret_cast<PlanSmem*>(smem + S::kOffPlan));
    const int unit_b = w.b, unit = w.unit;       // of a cluster: its only ones
    if (a.cluster && w.left == 0) {              // fewer tiles than CTAs
        for (int i = tid; i < NH * kPart; i += kThreads)
            share[i] = i % kPart == kD ? -INFINITY : 0.0f;
    }
    // ---- the place to fill next: keys or values of a tile; its two groups of eight tokens lie in a page
    // each, looked up a tile ahead. Byte i of `live`: the tokens of the two groups in place i.
    Walk ahead = w;
    int ahead_here = w.left > 0 ? w.here() : 0, ahead_k = 0, page[2], row[2] = {0, 0};
    uint32_t live = 0u, now = 0u;
    bool values_next = false;
    auto entries = [&]() {
        const int tok = ((ahead.t + ahead_k) << kPagedTcShift) + kTokens * warp;
        const int32_t* slots = a.pages.table + static_cast<long long>(ahead.b) * a.pages.stride;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            page[i] = ahead.left > 0 && tok + 8 * i < ahead.len ? page_in(a, slots, slot_of(a, tok + 8 * i)) : -1;
    };
    entries();
    auto issue = [&](int place) {
        if (ahead.left > 0) {
            if (!values_next) {
                now = 0u;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int tok = ((ahead.t + ahead_k) << kPagedTcShift) + kTokens * warp + 8 * i;
                    const bool there = page[i] >= 0 && page[i] < a.pages.n_pages;
                    row[i] = there ? (page[i] * a.Hkv + kv_head(a, ahead.unit)) * a.pages.page_size +
                                         (tok - slot_of(a, tok) * a.pages.page_size)
                                   : 0;
                    if (there && mp_check(a.status, row[i] + 7ll,
                                          static_cast<long long>(a.pages.n_pages) * a.Hkv * a.pages.page_size,
                                          kSitePagedRow))
                        now |= static_cast<uint32_t>(min(8, ahead.len - tok)) << (4 * i);
                }
            }
            live = (live & ~(255u << (8 * place))) | now << (8 * place);
            if (now) {
                const float* pool = static_cast<const float*>(values_next ? a.values : a.keys) + 4 * lane;
                const uint32_t dst = smem_u32(ring) + place * kPlace;
#pragma unroll
                for (int i = 0; i < kTokens; ++i) {
                    const bool ok = (i & 7) < static_cast<int>(now >> (4 * (i >> 3)) & 15u);
                    copy16_or_zero(dst + i * kD * 4 + ((lane ^ (i & 7)) << 4),
                                   pool + (ok ? static_cast<size_t>(row[i >> 3] + (i & 7)) * kD : 0), ok);
                }
            }
            if (values_next) {
                if (++ahead_k == ahead_here) {
                    ahead.next(a, ahead_here);
                    ahead_k = 0;
                    if (ahead.left > 0) ahead_here = ahead.here();
                }
                entries();
            }
            values_next = !values_next;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto landed = [&]() {
        asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
        __syncwarp();
    };
    // piece p of row r of the place
    auto piece = [&](int place, int r, int p) {
        return *reinterpret_cast<const float4*>(ring + place * kPlace + r * kD * 4 + ((p ^ (r & 7)) << 4));
    };
#pragma unroll
    for (int i = 0; i < kRing; ++i) issue(i);
    int place = 0;
    while (w.left > 0) {
        const int here = w.here(), kg = kv_head(a, w.unit), h0 = (w.unit - kg * a.chunks) * NH;
        const int heads = min(NH, a.G - h0);
        const size_t row0 = static_cast<size_t>(w.b) * a.Hq + kg * a.G + h0;
        // ---- queries: step i multiplies dims 32 (i / 4) + 8 t + 2 (i % 4) (as k = t) and the next (t + 4)
        uint32_t qh[NT == 1 ? 32 : 1], ql[NT == 1 ? 32 : 1];
        if constexpr (NT == 1) {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                if (g < heads) load_query4(a, (row0 + g) * kD + 32 * (c >> 1) + 8 * t + 4 * (c & 1), x);
#pragma unroll
                for (int i = 0; i < 4; ++i) two_parts(x[i], qh[4 * c + i], ql[4 * c + i]);
            }
        } else {
            for (int i = tid; i < 8 * NT * 32; i += kThreads) {          // two steps at a time
                const int l = i & 31, nt = i >> 5 & (NT - 1), c = i / (32 * NT), h = 8 * nt + (l >> 2);
                float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                if (h < heads) load_query4(a, (row0 + h) * kD + 32 * (c >> 1) + 8 * (l & 3) + 4 * (c & 1), x);
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) two_parts(x[j], hi[j], lo[j]);
                queries[((2 * c) * NT + nt) * 32 + l] = make_uint4(hi[0], hi[1], lo[0], lo[1]);
                queries[((2 * c + 1) * NT + nt) * 32 + l] = make_uint4(hi[2], hi[3], lo[2], lo[3]);
            }
            __syncthreads();
        }
        float m[NT][2], l[NT][2], o[NT][8][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                m[nt][i] = -INFINITY;
                l[nt][i] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[nt][i][j] = 0.0f;
        }
        for (int k = 0; k < here; ++k) {
            landed();                            // the tile's keys
            const uint32_t tokens = live >> (8 * place) & 255u;
            float s[NT][4];
            if (tokens) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[nt][i] = 0.0f;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    constexpr int kParts = NT == 1 ? 3 : 2;              // chains of sums: hi hi, lo hi, hi lo
                    float part[kParts][NT][4];
#pragma unroll
                    for (int x = 0; x < kParts; ++x)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int i = 0; i < 4; ++i) part[x][nt][i] = 0.0f;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float4 x = piece(place, g, 8 * c + 2 * t + j);
                        const float4 y = piece(place, g + 8, 8 * c + 2 * t + j);
                        const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int step = 4 * c + 2 * j + i;
                            uint32_t hi[4], lo[4];
                            two_parts(xs[2 * i], hi[0], lo[0]);
                            two_parts(ys[2 * i], hi[1], lo[1]);
                            two_parts(xs[2 * i + 1], hi[2], lo[2]);
                            two_parts(ys[2 * i + 1], hi[3], lo[3]);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                uint4 q;
                                if constexpr (NT == 1)
                                    q = make_uint4(qh[2 * step], qh[2 * step + 1], ql[2 * step], ql[2 * step + 1]);
                                else
                                    q = queries[(step * NT + nt) * 32 + lane];
                                mma(part[0][nt], hi, q.x, q.y);
                                mma(part[1][nt], lo, q.x, q.y);
                                mma(part[kParts - 1][nt], hi, q.z, q.w);
                            }
                        }
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            s[nt][i] += part[0][nt][i] +
                                        (NT == 1 ? part[1][nt][i] + part[kParts - 1][nt][i] : part[1][nt][i]);
                }
            }
            __syncwarp();                        // the keys are read
            issue(place);
            place = place == kRing - 1 ? 0 : place + 1;
            float corr[NT][2];
            if (tokens) {
                // ---- s[nt][2 r + i]: token g + 8 r, head 8 nt + 2 t + i
                const bool there[2] = {g < static_cast<int>(tokens & 15u), g < static_cast<int>(tokens >> 4)};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float x = there[0] ? s[nt][i] * a.scale : -INFINITY;
                        const float y = there[1] ? s[nt][2 + i] * a.scale : -INFINITY;
                        float mn = fmaxf(x, y);
#pragma unroll
                        for (int off = 4; off <= 16; off <<= 1)
                            mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, off));
                        mn = fmaxf(m[nt][i], mn);
                        const float from = mn == -INFINITY ? 0.0f : mn;
                        corr[nt][i] = exp2_fast(m[nt][i] - from);
                        const float p0 = exp2_fast(x - from), p1 = exp2_fast(y - from);
                        l[nt][i] = fmaf(l[nt][i], corr[nt][i], p0 + p1);
                        m[nt][i] = mn;
                        float* at = weights + (8 * nt + 2 * t + i) * kPitch + g;
                        at[0] = p0;
                        at[8] = p1;
                    }
                }
                __syncwarp();
            }
            landed();                            // the tile's values
            if (tokens) {
                uint32_t ph[NT][4], pl[NT][4];   // tokens t, t + 4, t + 8, t + 12 of head g
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        two_parts(weights[(8 * nt + g) * kPitch + t + 4 * i], ph[nt][i], pl[nt][i]);
                // piece 4 g + i: dims 16 g + 4 i ..; two of them a row g and g + 8 of column tile 2 i, two of the next
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float d[2][NT][4];
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int j = 0; j < 4; ++j) d[x][nt][j] = 0.0f;
#pragma unroll
                    for (int st = 0; st < 2; ++st) {
                        const float4 x = piece(place, 8 * st + t, 4 * g + i);
                        const float4 y = piece(place, 8 * st + t + 4, 4 * g + i);
                        const float v[2][4] = {{x.x, x.y, y.x, y.y}, {x.z, x.w, y.z, y.w}};
#pragma unroll
                        for (int mt = 0; mt < 2; ++mt) {
                            uint32_t hi[4], lo[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) two_parts(v[mt][j], hi[j], lo[j]);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                mma(d[mt][nt], lo, ph[nt][2 * st], ph[nt][2 * st + 1]);
                                mma(d[mt][nt], hi, pl[nt][2 * st], pl[nt][2 * st + 1]);
                                mma(d[mt][nt], hi, ph[nt][2 * st], ph[nt][2 * st + 1]);
                            }
                        }
                    }
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                o[nt][2 * i + mt][j] = fmaf(o[nt][2 * i + mt][j], corr[nt][j & 1], d[mt][nt][j]);
                }
            }
            __syncwarp();                        // the values and the weights are read
            if (k + 1 < here) {
                issue(place);
                place = place == kRing - 1 ? 0 : place + 1;
            }
        }
        // ---- the warps' states, each in the place of the values it took last, joined in order
        float* state = reinterpret_cast<float*>(ring + place * kPlace);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int off = 4; off <= 16; off <<= 1)
                    l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], off);
                const int h = 8 * nt + 2 * t + i;
#pragma unroll
                for (int mt = 0; mt < 8; ++mt)
                    *reinterpret_cast<float2*>(state + h * kD + 16 * g + 2 * mt) =
                        make_float2(o[nt][mt][i], o[nt][mt][2 + i]);
                if (g == 0) ml[warp * NH + h] = make_float2(m[nt][i], l[nt][i]);
            }
        }
        __syncthreads();
        const int e = tid & (kD - 1);
        for (int h = tid / kD; h < heads; h += kThreads / kD) {
            float M = -INFINITY, L = 0.0f, O = 0.0f;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) M = fmaxf(M, ml[i * NH + h].x);
            const float from = M == -INFINITY ? 0.0f : M;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
                const float2 x = ml[i * NH + h];
                const float c = exp2_fast(x.x - from);
                L = fmaf(c, x.y, L);
                O = fmaf(c, reinterpret_cast<const float*>(smem + (i * kRing + place) * kPlace)[h * kD + e], O);
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
    zero_empty(a, tid, kThreads);
    if (a.cluster) {
        __syncthreads();
        join_cluster(a, share, unit_b, unit);
    }
}

typedef void (*MmaFn)(const PArgs);
MmaFn pick_mma(int nh, int* smem) {
    *smem = nh == 8 ? MmaSmem<1>::kBytes : MmaSmem<2>::kBytes;
    return nh == 8 ? paged_attention_mma_kernel<1> : paged_attention_mma_kernel<2>;
}

}  // namespace

cudaError_t launch_paged_attention_mma(const PArgs& a, unsigned grid, cudaStream_t st) {
    int smem;
    const MmaFn fn = pick_mma(a.nh, &smem);
    return launch_dependent(fn, dim3(grid), dim3(kThreads), smem, st, a, std::max(1, a.cluster));
}

cudaError_t prepare_paged_mma() {
    for (int nh : {8, 16}) {
        int smem;
        const MmaFn fn = pick_mma(nh, &smem);
        cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(fn, cudaFuncAttributePreferredSharedMemoryCarveout,
                                     cudaSharedmemCarveoutMaxShared);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace mp
