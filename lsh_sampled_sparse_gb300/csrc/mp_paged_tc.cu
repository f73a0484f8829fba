// Exact attention of single query tokens over a bf16 paged cache, on the tcgen05 tensor cores.
//
// A tile is 128 tokens. Scores: S = K Q^T with the tile's keys as the 128 rows of the MMA and the
// query heads as its columns, sums in tensor memory, a token a lane. Values: O = V^T P with the 128
// dims as rows (the same layout of V in shared memory read with its dims along M) and the heads'
// weights as columns. Keys and values so go from memory to the tensor cores by TMA alone: no register
// and no instruction of theirs, whatever the heads that share them. A float32 number (a query element
// of a float32 query, a weight) meets the bf16 ones as three bf16 terms, 24 bits, a column each; a bf16
// query is one term. Products are exact, sums float32.
//
// TMA: keys and values are tensors [page x head][8-token groups][2 halves][8 tokens][64 dims], boxes one
// page's part of a tile. In shared memory a group of 8 tokens by 64 dims is one 128-byte-swizzled
// kilobyte, which K reads as 8 rows along M and V as 8 steps along K. A box whose slot holds no page,
// or that begins behind the sequence's end, is taken from outside the tensor: it reads as zeros, and
// no memory is touched.
//
// Structure, one CTA an SM, on a run of tiles of its own (mp_paged.cuh):
//   warps 0-3  softmax: S from tensor memory, masks, running maximum (over a warp by redux, over the
//              four through shared memory), weights in three terms to shared memory; the last tile's O
//              from tensor memory into float32 registers, a dim a thread
//   warp 4     TMA producer: rings of K and V tiles of 32 KB, a box a lane
//   warp 5     allocates tensor memory, issues the MMAs: S of the next tile before O of this one
//   warp 6     queries of the next unit into shared memory
// The sums of a tile start from zero and are added up in registers: the tensor core's own sums round
// toward zero, which stays small over 128 tokens.
//
// Bound by memory: 8 heads x 96K tokens, four query heads each, 66.5 us (6.1 TB/s with start and join), two
// sequences of 128K with eight 164 (6.5 TB/s), 32 sequences of up to 32K 443 to 473 by their lengths (6.8). The
// same sums on CUDA cores took 94, 404 and 692 us: each query head costs them every key's and value's dims
// again. 8 sequences x 8 heads x 16K tokens with 1, 4, 8 and 16 heads 88, 92, 94 and 97 us: the softmax warps'
// work on a tile's 128 x heads weights of three terms begins to show at 16.
//
// Every wait is bounded; on expiry the CTA records MP_ERR_TIMEOUT in the device status word, stops
// issuing work and still frees its tensor memory.
#include <algorithm>

#include "mp_paged.cuh"
#include "mp_tcgen05.cuh"

namespace mp {
namespace {

constexpr int kTile = 1 << kPagedTcShift;        // tokens
static_assert(kTile == kD, "the MMA's 128 rows are a tile's tokens, or the dims");
constexpr int kSoftWarps = 4, kSoftThreads = 32 * kSoftWarps;
constexpr int kWarps = 7, kThreads = 32 * kWarps;
constexpr uint32_t kStage = kTile * kD * 2;      // 32 KB: a tile of K or of V
constexpr uint32_t kGroup = 2048;                // 8 tokens: two swizzled kilobytes
constexpr int kTerms = 3;

// NH query heads a unit, QT terms a query element
template <int NH, int QT>
struct Lay {
    static constexpr int kN = (kTerms * NH + 15) / 16 * 16;              // columns of O: of the weights
    static constexpr int kNq = (QT * NH + 15) / 16 * 16;                 // columns of S: of the queries
    static constexpr uint32_t kTmemS = 64, kTmemO = 128, kTmem = 256;    // S, S, O: columns apart
    static constexpr int kKStages = 3, kVStages = NH == 16 && QT == 3 ? 2 : 3;
    static constexpr uint32_t kP = kN * kD * 2, kQ = kNq * kD * 2;       // rows of 256 bytes
    static constexpr uint32_t kOffV = kKStages * kStage;
    static constexpr uint32_t kOffP = kOffV + kVStages * kStage;
    static constexpr uint32_t kOffQ = kOffP + kP;
    static constexpr uint32_t kOffBars = kOffQ + 2 * kQ;
    static constexpr uint32_t kOffMax = kOffBars + 256;                  // [2][warps][NH]
    static constexpr uint32_t kOffSum = kOffMax + 2 * kSoftWarps * NH * 4;   // [warps][NH]
    static constexpr uint32_t kOffPlan = kOffSum + kSoftWarps * NH * 4;
    static constexpr uint32_t kBytes = kOffPlan + sizeof(PlanSmem) + 1024;   // + alignment slack
    static_assert(kN <= kTmemS && kBytes <= 232448 - 64, "tensor memory, shared memory");
    static_assert(kP % 1024 == 0 && kQ % 1024 == 0, "swizzled operands start on 1024-byte boundaries");
};

// Three bf16 terms of two floats, packed (low: the first)
__device__ __forceinline__ uint32_t pack_bf16(float low, float high) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(high), "f"(low));
    return r;
}
__device__ __forceinline__ void three_terms(float a, float b, uint32_t (&t)[kTerms]) {
#pragma unroll
    for (int i = 0; i < kTerms; ++i) {
        t[i] = pack_bf16(a, b);
        a -= __uint_as_float(t[i] << 16);
        b -= __uint_as_float(t[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ float warp_max(float x) {                     // of what is not NaN
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ void softmax_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(kSoftThreads) : "memory");
}

template <int NH, int QT>
__global__ void __launch_bounds__(kThreads, 1)
    paged_attention_tc_kernel(const __grid_constant__ CUtensorMap kmap,
                              const __grid_constant__ CUtensorMap vmap, const PArgs a) {
    using L = Lay<NH, QT>;
    constexpr int N = L::kN;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_word;
    volatile int* abort_flag = &abort_word;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = smem_u32(smem);
    const uint32_t k_full = base + L::kOffBars, k_empty = k_full + 8 * L::kKStages;
    const uint32_t v_full = k_empty + 8 * L::kKStages, v_empty = v_full + 8 * L::kVStages;
    const uint32_t s_full = v_empty + 8 * L::kVStages, s_empty = s_full + 16;
    const uint32_t q_full = s_empty + 16, q_empty = q_full + 16;
    const uint32_t p_full = q_empty + 16, o_full = p_full + 8;
    if (tid == 0) {
        for (int i = 0; i < 2 * (L::kKStages + L::kVStages); ++i) mbar_init(k_full + 8 * i, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full + 8 * i, 1);
            mbar_init(s_empty + 8 * i, kSoftWarps);
            mbar_init(q_full + 8 * i, 1);
            mbar_init(q_empty + 8 * i, 1);
        }
        mbar_init(p_full, kSoftWarps);
        mbar_init(o_full, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 4 && lane == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&kmap)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&vmap)) : "memory");
    }
    if (warp == 5) tmem_alloc(smem_u32(&tmem_slot), L::kTmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const uint32_t tmem_o = tmem + L::kTmemO;
    wait_for_predecessor();
    allow_dependents();
    Walk w = plan_run(a, *reinterpret_cast<PlanSmem*>(smem + L::kOffPlan));
    // a cluster's states: in the place of the first tile of K, once it is scored
    float* share = reinterpret_cast<float*>(smem);
    const int unit_b = w.b, unit = w.unit;       // of a cluster: its only ones

    const int box_rows = min(kTile, a.pages.page_size & -a.pages.page_size);
    if (warp < kSoftWarps) {
        // ---------------- softmax ----------------
        if (a.cluster && w.left == 0) {          // fewer tiles than CTAs
            for (int h = 0; h < NH; ++h) share[h * kPart + tid] = 0.0f;
            if (tid < NH) {
                share[tid * kPart + kD] = -INFINITY;
                share[tid * kPart + kD + 1] = 0.0f;
            }
        }
        const uint32_t quad = static_cast<uint32_t>(warp * 32) << 16;    // this warp's TMEM lanes
        const uint32_t chunk = (tid & 63) >> 3;
        const uint32_t p_at = base + L::kOffP + (tid >> 6) * (N * 128) + (chunk << 4) + (tid & 7) * 2;
        float* sums = reinterpret_cast<float*>(smem + L::kOffSum);
        bool aborted = false;
        auto wait = [&](uint32_t bar, int phase) {
            if (!aborted)
                aborted = !__all_sync(0xffffffffu, mbar_wait(bar, phase & 1, abort_flag, a.status));
        };
        // the unit at hand, and the one before, whose last tile's values are still to come while this
        // one's first scores are worked on
        struct Unit {
            int b, g, h0, t, len;
            bool whole;
        };
        Unit now{0, 0, 0, 0, 0, false}, last = now;
        const int32_t* slots = nullptr;
        const int total = w.left;
        int here = 0, k = 0, page = -1;
        float m[NH], l[NH], o[NH];
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            m[h] = -INFINITY;
            l[h] = o[h] = 0.0f;
        }
        for (int it = 0; total > 0; ++it) {
            const bool more = it < total, fresh = k == here;             // fresh: a unit's first, or the end
            float m_last[NH], l_last[NH], s[NH], corr[NH];
            if (fresh) {
                last = now;
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    m_last[h] = m[h];
                    l_last[h] = l[h];
                    m[h] = -INFINITY;
                    l[h] = 0.0f;
                }
                if (more) {
                    here = w.here();
                    k = 0;
                    const int g = kv_head(a, w.unit);
                    now = Unit{w.b, g, (w.unit - g * a.chunks) * NH, w.t, w.len, here == w.tiles};
                    slots = a.pages.table + static_cast<long long>(w.b) * a.pages.stride;
                    const int tok = now.t * kTile + tid;
                    page = tok < now.len ? page_in(a, slots, slot_of(a, tok)) : -1;
                    w.next(a, here);
                }
            }
            const int tok0 = (now.t + k) * kTile;
            if (more) {
                wait(s_full + 8 * (it & 1), it >> 1);
                if (!aborted) {
                    tc_fence_after();
                    const uint32_t from = tmem + quad + (it & 1) * L::kTmemS;
                    uint32_t t0[NH];
                    tmem_ld(from, t0);
                    if constexpr (QT == 3) {
                        uint32_t t1[NH], t2[NH];
                        tmem_ld(from + NH, t1);
                        tmem_ld(from + 2 * NH, t2);
                        tmem_ld_wait();
#pragma unroll
                        for (int h = 0; h < NH; ++h)
                            s[h] = __uint_as_float(t0[h]) +
                                   (__uint_as_float(t1[h]) + __uint_as_float(t2[h]));
                    } else {
                        tmem_ld_wait();
#pragma unroll
                        for (int h = 0; h < NH; ++h) s[h] = __uint_as_float(t0[h]);
                    }
                } else {
#pragma unroll
                    for (int h = 0; h < NH; ++h) s[h] = 0.0f;
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_empty + 8 * (it & 1));
                const bool live = page >= 0 && page < a.pages.n_pages;   // and before the end
                const int tok = tok0 + kTile + tid;
                page = k + 1 < here && tok < now.len ? page_in(a, slots, slot_of(a, tok)) : -1;
                // ---- the tile's maxima, over the warp and over the four
                float* most = reinterpret_cast<float*>(smem + L::kOffMax) + (it & 1) * kSoftWarps * NH;
                float mine[NH];
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    s[h] = live ? s[h] * a.scale : -INFINITY;
                    mine[h] = warp_max(s[h]);
                }
                if (lane == 0) {
#pragma unroll
                    for (int h = 0; h < NH; h += 4)
                        *reinterpret_cast<float4*>(most + warp * NH + h) =
                            make_float4(mine[h], mine[h + 1], mine[h + 2], mine[h + 3]);
                }
                softmax_sync();
#pragma unroll
                for (int h = 0; h < NH; h += 4) {
                    float4 x = *reinterpret_cast<const float4*>(most + h);
#pragma unroll
                    for (int i = 1; i < kSoftWarps; ++i) {
                        const float4 y = *reinterpret_cast<const float4*>(most + i * NH + h);
                        x = make_float4(fmaxf(x.x, y.x), fmaxf(x.y, y.y), fmaxf(x.z, y.z),
                                        fmaxf(x.w, y.w));
                    }
                    const float xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float mn = fmaxf(m[h + j], xs[j]);
                        const float from = mn == -INFINITY ? 0.0f : mn;
                        corr[h + j] = exp2_fast(m[h + j] - from);
                        s[h + j] = exp2_fast(s[h + j] - from);           // the weight
                        l[h + j] = fmaf(l[h + j], corr[h + j], s[h + j]);
                        m[h + j] = mn;
                    }
                }
            }
            // ---- the last tile's values; the weights take the place of the last ones then
            if (it > 0) {
                wait(o_full, it - 1);
                if (!aborted) {
                    tc_fence_after();
                    uint32_t t0[NH], t1[NH], t2[NH];
                    tmem_ld(tmem_o + quad, t0);
                    tmem_ld(tmem_o + quad + NH, t1);
                    tmem_ld(tmem_o + quad + 2 * NH, t2);
                    tmem_ld_wait();
#pragma unroll
                    for (int h = 0; h < NH; ++h)
                        o[h] += __uint_as_float(t0[h]) +
                                (__uint_as_float(t1[h]) + __uint_as_float(t2[h]));
                }
                tc_fence_before();
            }
            if (more) {
#pragma unroll
                for (int h = 0; h < NH; h += 2) {
                    uint32_t t[kTerms];
                    three_terms(s[h], s[h + 1], t);
#pragma unroll
                    for (int i = 0; i < kTerms; ++i) {
                        const int n0 = i * NH + h;
                        asm volatile("st.shared.u16 [%0], %1;" ::"r"((p_at ^ ((n0 & 7) << 4)) + n0 * 128),
                                     "h"(static_cast<uint16_t>(t[i])) : "memory");
                        asm volatile("st.shared.u16 [%0], %1;" ::"r"(
                                         (p_at ^ (((n0 + 1) & 7) << 4)) + (n0 + 1) * 128),
                                     "h"(static_cast<uint16_t>(t[i] >> 16)) : "memory");
                    }
                }
                // ---- rows of V from the sequence's end to the end of their box: a weight of 0 does not
                // undo a NaN there (boxes behind it read as zeros)
                if (tok0 + kTile > now.len) {
                    const int stage = it % L::kVStages, row0 = now.len - tok0;
                    const int lines = ((row0 + box_rows - 1) / box_rows * box_rows - row0) * 16;
                    wait(v_full + 8 * stage, it / L::kVStages);
                    for (int x = tid; !aborted && x < lines; x += kSoftThreads) {
                        const int row = row0 + (x >> 4);                 // 16 pieces of 16 bytes a row
                        *reinterpret_cast<uint4*>(smem + L::kOffV + stage * kStage +
                                                  (row >> 3) * kGroup + (x >> 3 & 1) * 1024 +
                                                  (row & 7) * 128 + (x & 7) * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full);
            }
            if (!fresh) {
#pragma unroll
                for (int h = 0; h < NH; ++h) o[h] *= corr[h];
            } else {
                if (it > 0) {
                    // ---- the last unit's state: its weights' sums by a reduce-scatter over the lanes (to
                    // 32 / NH of them), then over the warps; a dim a thread
                    float* r = l_last;
#pragma unroll
                    for (int lv = 0; (NH / 2 >> lv) >= 1; ++lv) {
                        const int off = 16 >> lv, keep = NH / 2 >> lv;
                        const bool up = (lane & off) != 0;
#pragma unroll
                        for (int i = 0; i < keep; ++i) {
                            const float send = up ? r[i] : r[i + keep];
                            r[i] = (up ? r[i + keep] : r[i]) + __shfl_xor_sync(0xffffffffu, send, off);
                        }
                    }
#pragma unroll
                    for (int off = 16 / NH; off >= 1; off >>= 1)
                        r[0] += __shfl_xor_sync(0xffffffffu, r[0], off);
                    // (one copy of the sums: a warp may still read those of the unit before. Where a tile
                    // follows, the maxima's barrier stands between; behind the last one stands this)
                    if (!more) softmax_sync();
                    if ((lane & (32 / NH - 1)) == 0) sums[warp * NH + lane * NH / 32] = r[0];
                    softmax_sync();
                    const int heads = aborted ? 0 : min(NH, a.G - last.h0);
                    const size_t row0 = static_cast<size_t>(last.b) * a.Hq + last.g * a.G + last.h0;
#pragma unroll
                    for (int h = 0; h < NH; ++h) {
                        if (h >= heads) break;
                        const float sum = (sums[h] + sums[NH + h]) + (sums[2 * NH + h] + sums[3 * NH + h]);
                        if (a.cluster) {
                            share[h * kPart + tid] = o[h];
                            if (tid == 0) {
                                share[h * kPart + kD] = m_last[h];
                                share[h * kPart + kD + 1] = sum;
                            }
                        } else if (last.whole) {
                            if (mp_check(a.status, static_cast<long long>(row0 + h),
                                         static_cast<long long>(a.B) * a.Hq, kSitePagedOut))
                                a.out[(row0 + h) * kD + tid] = over_sum(o[h], sum);
                        } else if (part_there(a, blockIdx.x, last.t == 0, h)) {
                            float* p = part_of(a, last.t == 0, h);
                            p[tid] = o[h];
                            if (tid == 0) {
                                p[kD] = m_last[h];
                                p[kD + 1] = sum;
                            }
                        }
                    }
                }
#pragma unroll
                for (int h = 0; h < NH; ++h) o[h] = 0.0f;
                if (!more) break;
            }
            ++k;
        }
    } else if (warp == 4) {
        // ---------------- TMA producer ----------------
        // a batch: the table's entries of the next 32 boxes of a unit, an entry a lane, looked up while
        // the last batch's tiles are copied
        const int boxes = kTile / box_rows;      // of a tile
        const int box_shift = __ffs(boxes) - 1, batch = 32 >> box_shift;
        struct Batch {
            int tiles, page, head, group;        // tiles in it; the entry, the KV head, the group of a page
        };
        int k = 0;
        auto look_up = [&]() {
            Batch x{0, -1, 0, 0};
            if (w.left <= 0) return x;
            const int here = w.here(), tok = (w.t + k) * kTile + lane * box_rows;
            x.tiles = min(batch, here - k);
            x.head = kv_head(a, w.unit);
            if (tok < w.len && lane < x.tiles << box_shift) {
                const int slot = slot_of(a, tok);
                x.page = page_in(a, a.pages.table + static_cast<long long>(w.b) * a.pages.stride, slot);
                x.group = (tok - slot * a.pages.page_size) >> 3;
            }
            k += x.tiles;
            if (k == here) {
                w.next(a, here);
                k = 0;
            }
            return x;
        };
        int it = 0;
        bool ok = true;
        for (Batch x = look_up(); x.tiles > 0 && ok;) {
            const Batch ahead = look_up();
            // outside the tensor where there is no page
            const bool there = x.page >= 0 && x.page < a.pages.n_pages;
            const int at = there ? x.page * a.Hkv + x.head : a.pages.n_pages * a.Hkv;
            const uint32_t dst = base + (lane & (boxes - 1)) * (box_rows / 8) * kGroup;
            for (int i = 0; i < x.tiles; ++i, ++it) {
                const int ks = it % L::kKStages, vs = it % L::kVStages;
                const bool mine = lane >> box_shift == i;
                if (!__all_sync(0xffffffffu, mbar_wait(k_empty + 8 * ks, (it / L::kKStages & 1) ^ 1,
                                                       abort_flag, a.status))) {
                    ok = false;
                    break;
                }
                if (lane == 0) mbar_arrive_expect_tx(k_full + 8 * ks, kStage);
                __syncwarp();
                if (mine) tma_load_5d(dst + ks * kStage, &kmap, k_full + 8 * ks, 0, 0, 0, x.group, at);
                if (!__all_sync(0xffffffffu, mbar_wait(v_empty + 8 * vs, (it / L::kVStages & 1) ^ 1,
                                                       abort_flag, a.status))) {
                    ok = false;
                    break;
                }
                if (lane == 0) mbar_arrive_expect_tx(v_full + 8 * vs, kStage);
                __syncwarp();
                if (mine)
                    tma_load_5d(dst + L::kOffV + vs * kStage, &vmap, v_full + 8 * vs, 0, 0, 0, x.group, at);
            }
            x = ahead;
        }
        if (!ok && lane == 0) {
            // let the loads already issued land before the CTA can exit (bounded): those of tile `it`
            // may have stopped after K
            volatile int never = 0;
            for (int i = max(0, it - L::kKStages + 1); i <= it; ++i)
                mbar_wait(k_full + 8 * (i % L::kKStages), i / L::kKStages & 1, &never, a.status,
                          kWaitLimitNs / 8);
            for (int i = max(0, it - L::kVStages); i < it; ++i)
                mbar_wait(v_full + 8 * (i % L::kVStages), i / L::kVStages & 1, &never, a.status,
                          kWaitLimitNs / 8);
        }
    } else if (warp == 5) {
        // ---------------- MMA issuer ----------------
        if (lane == 0 && w.left > 0) {
            const uint32_t s_desc = make_idesc(kTile, L::kNq), o_desc = make_idesc(kD, N, true);
            const int total = w.left;
            int seg = 0, in_seg = w.here();      // tiles of the unit not scored yet
            auto wait = [&](uint32_t bar, int phase) {
                return mbar_wait(bar, phase & 1, abort_flag, a.status);
            };
            bool fresh = true;                   // the next tile is its unit's first here
            auto score = [&](int it) {           // S of tile it
                const int ks = it % L::kKStages, slot = seg & 1;
                if (fresh && !wait(q_full + 8 * slot, seg >> 1)) return false;
                fresh = false;
                if (!wait(k_full + 8 * ks, it / L::kKStages) ||
                    !wait(s_empty + 8 * (it & 1), (it >> 1) ^ 1))
                    return false;
                tc_fence_after();
                const uint32_t k_at = base + ks * kStage, q_at = base + L::kOffQ + slot * L::kQ;
#pragma unroll
                for (int x = 0; x < kD / 16; ++x)
                    tc_mma(tmem + (it & 1) * L::kTmemS,
                           sw128_desc(k_at + (x >> 2) * 1024 + (x & 3) * 32, kGroup),
                           sw128_desc(q_at + (x >> 2) * (L::kNq * 128) + (x & 3) * 32), s_desc, x > 0);
                tc_commit(k_empty + 8 * ks);
                tc_commit(s_full + 8 * (it & 1));
                if (--in_seg == 0) {
                    tc_commit(q_empty + 8 * slot);
                    ++seg;
                    fresh = true;
                    w.next(a, w.here());
                    if (w.left > 0) in_seg = w.here();
                }
                return true;
            };
            bool ok = score(0);
            for (int it = 0; it < total && ok; ++it) {
                if (it + 1 < total && !(ok = score(it + 1))) break;
                const int vs = it % L::kVStages;
                if (!(ok = wait(p_full, it) && wait(v_full + 8 * vs, it / L::kVStages))) break;
                tc_fence_after();
                const uint32_t v_at = base + L::kOffV + vs * kStage, p_at = base + L::kOffP;
#pragma unroll
                for (int x = 0; x < kTile / 16; ++x)
                    tc_mma(tmem_o, sw128_desc(v_at + x * 2 * kGroup, kGroup, 1024),
                           sw128_desc(p_at + (x >> 2) * (N * 128) + (x & 3) * 32), o_desc, x > 0);
                tc_commit(v_empty + 8 * vs);
                tc_commit(o_full);
            }
        }
    } else {
        // ---------------- queries ----------------
        int seg = 0;
        while (w.left > 0) {
            const int here = w.here(), g = kv_head(a, w.unit), h0 = (w.unit - g * a.chunks) * NH;
            const int heads = min(NH, a.G - h0);
            const size_t row0 = static_cast<size_t>(w.b) * a.Hq + g * a.G + h0;
            if (!__all_sync(0xffffffffu, mbar_wait(q_empty + 8 * (seg & 1), (seg >> 1 & 1) ^ 1,
                                                   abort_flag, a.status)))
                break;
            uint8_t* dst = smem + L::kOffQ + (seg & 1) * L::kQ + (lane >> 4) * (L::kNq * 128);
            float x[NH][4];
#pragma unroll
            for (int h = 0; h < NH; ++h)
                load_query4(a, (row0 + min(h, heads - 1)) * kD + 4 * lane, x[h]);
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                uint32_t t0[kTerms], t1[kTerms];
                three_terms(x[h][0], x[h][1], t0);
                three_terms(x[h][2], x[h][3], t1);
#pragma unroll
                for (int i = 0; i < QT; ++i) {
                    const int n = i * NH + h;
                        *reinterpret_cast<uint2*>(dst + n * 128 +
                                                  ((((lane & 15) >> 1) ^ (n & 7)) << 4) +
                                                  (lane & 1) * 8) = make_uint2(t0[i], t1[i]);
                }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full + 8 * (seg & 1));
            ++seg;
            w.next(a, here);
        }
        zero_empty(a, lane, 32);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 5) {
        __syncwarp();
        tmem_dealloc(tmem, L::kTmem);
    }
    if (a.cluster) join_cluster(a, share, unit_b, unit);
}

typedef void (*TcFn)(const CUtensorMap, const CUtensorMap, const PArgs);
template <int NH, int QT>
TcFn tc(uint32_t* smem) {
    *smem = Lay<NH, QT>::kBytes;
    return paged_attention_tc_kernel<NH, QT>;
}
TcFn pick_tc(int nh, bool q_bf16, uint32_t* smem) {
    switch (nh) {
        case 4: return q_bf16 ? tc<4, 1>(smem) : tc<4, 3>(smem);
        case 8: return q_bf16 ? tc<8, 1>(smem) : tc<8, 3>(smem);
        default: return q_bf16 ? tc<16, 1>(smem) : tc<16, 3>(smem);
    }
}

bool page_map(CUtensorMap* map, const void* pool, const mp_paged& c, int Hkv) {
    const cuuint64_t page_bytes = static_cast<cuuint64_t>(c.page_size) * kD * 2;
    const cuuint64_t dims[5] = {64, 8, 2, static_cast<cuuint64_t>(c.page_size / 8),
                                static_cast<cuuint64_t>(c.n_pages) * Hkv};
    const cuuint64_t strides[4] = {kD * 2, 128, kGroup, page_bytes};
    const cuuint32_t rows = std::min(kTile, c.page_size & -c.page_size);
    const cuuint32_t box[5] = {64, 8, 2, rows / 8, 1}, step[5] = {1, 1, 1, 1, 1};
    return encode_tiled_fn()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(pool), dims,
                             strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

int paged_tc_heads(int G) { return G <= 4 ? 4 : (G <= 8 ? 8 : 16); }

cudaError_t launch_paged_attention_tc(const PArgs& a, const mp_paged& cache, unsigned grid,
                                      cudaStream_t st) {
    if (!encode_tiled_fn()) return cudaErrorNotSupported;
    CUtensorMap kmap, vmap;
    if (!page_map(&kmap, cache.keys, cache, a.Hkv) || !page_map(&vmap, cache.values, cache, a.Hkv))
        return cudaErrorInvalidValue;
    uint32_t smem;
    const TcFn fn = pick_tc(a.nh, a.q_bf16, &smem);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, fn, kmap, vmap, a);
}

cudaError_t paged_tc_clusters(int size, int* n) {
    uint32_t smem;
    const TcFn fn = pick_tc(4, true, &smem);
    return max_clusters(fn, kThreads, smem, size, n);
}

cudaError_t prepare_paged_tc() {
    for (int i = 0; i < 6; ++i) {
        uint32_t smem;
        const TcFn fn = pick_tc(4 << i / 2, i & 1, &smem);
        cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(smem));
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(fn, cudaFuncAttributePreferredSharedMemoryCarveout,
                                     cudaSharedmemCarveoutMaxShared);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace mp
