// A paged K/V cache at full precision: tokens appended with their rotary positions applied on the
// way, and exact attention of single query tokens over the pages. The pages of the reference keep
// K and V in one piece and have no counterpart; the layout is the one magicpig.h describes.
//
// The kernels are launched as dependents of what precedes them in the stream: their lives begin
// before it has written what they read. So no load here is a non-coherent one, which would promise
// that nobody writes its memory meanwhile; ordinary loads stay behind the wait.
#include <algorithm>
#include <type_traits>

#include "mp_paged.cuh"

namespace mp {
namespace {

constexpr int kSms = 152;                        // of a GB300; a workspace's size is the same on the
                                                 // host alone
using Bf16 = __nv_bfloat16;

// ------------------------------------------------------------------------------------------------
// Append. Pair j of a row at position p turns by a = p inv_freq[j]; in half turns a / pi = 2 frac(p t)
// with t = inv_freq[j] / (2 pi). t mod 1 is taken to 64 fractional bits once a thread (in float64),
// p t mod 1 is then one wrapping 64-bit product, exact, and cos and sin are those of a number in
// [-1, 1] half turns: no loss at far positions, where p inv_freq in float32 is off by whole fractions
// of a turn.
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
    int pairs, interleaved, B, Hq, Hkv, m, n_begin, toks, tok_blocks, rows;
    int* status;                                 // index checks of the MP_CHECKS build
};

constexpr int kAppThreads = 256;
constexpr int kRowLanes = 8;                     // lanes a row, 2 x 8 dims each
constexpr int kAppRows = kAppThreads / kRowLanes;
constexpr int kMaxToks = 4;                      // tokens a CTA turns

// 8 elements as floats, and back
__device__ __forceinline__ void load_row8(const float* p, float (&x)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load_row8(const Bf16* p, float (&x)[8]) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void store_row8(float* p, const float (&x)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store_row8(Bf16* p, const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// A CTA takes `toks` tokens of one sequence and a share of their rows (of the query heads, then the
// key heads, then the value heads): the angles of a token are made once for all its heads.
template <typename T, typename C>
__global__ void __launch_bounds__(kAppThreads) paged_append_kernel(const AppendArgs a) {
    __shared__ __align__(16) float2 turn[kMaxToks][kD / 2];
    const int tid = threadIdx.x;
    const int b = blockIdx.x / a.tok_blocks, i0 = static_cast<int>(blockIdx.x % a.tok_blocks) * a.toks;
    wait_for_predecessor();
    const int live = a.counts ? min(a.m, a.counts[b]) : a.m;
    const int toks = min(a.toks, live - i0);
    if (toks <= 0) return;
    const long long p0 = (a.positions ? static_cast<long long>(a.positions[b]) : a.n_begin) + i0;
    for (int x = tid; x < toks * a.pairs; x += kAppThreads) {
        const int i = x / a.pairs, j = x - i * a.pairs;
        double t = static_cast<double>(a.inv_freq[j]) * 0.15915494309189533577;   // 1 / (2 pi)
        t -= floor(t);
        const unsigned long long step = __double2ull_rz(t * 18446744073709551616.0);     // 2^64
        const long long frac = static_cast<long long>(step * static_cast<unsigned long long>(p0 + i));
        float s, c;
        sincospif(static_cast<float>(frac) * 0x1p-63f, &s, &c);
        turn[i][j] = make_float2(c, s);
    }
    __syncthreads();
    const int lane = tid & (kRowLanes - 1);
    // this lane's two pieces of 8 dims: a pair's two halves, or whole pairs, or dims that stay
    const int turned = a.pairs / 8;              // lanes whose pieces turn
    int da = 16 * lane, db = 16 * lane + 8;
    if (!a.interleaved && lane < turned) {
        da = 8 * lane;
        db = a.pairs + 8 * lane;
    }
    const long long cap = static_cast<long long>(a.pages.n_slots) * a.pages.page_size;
    const int heads = a.Hq + 2 * a.Hkv;
    for (int r = blockIdx.y * kAppRows + tid / kRowLanes; r < heads * toks; r += gridDim.y * kAppRows) {
        const int h = r / toks, i = r - h * toks;
        const int kind = h < a.Hq ? 0 : (h < a.Hq + a.Hkv ? 1 : 2);
        const mp_rows& from = kind == 0 ? a.q : (kind == 1 ? a.k : a.v);
        const int g = kind == 0 ? h : (kind == 1 ? h - a.Hq : h - a.Hq - a.Hkv);
        const T* src = static_cast<const T*>(from.data) + b * from.stride_b + g * from.stride_h +
                       (i0 + i) * from.stride_m;
        float x[8], y[8];
        load_row8(src + da, x);
        load_row8(src + db, y);
        if (kind < 2 && lane < turned) {
            const float2* cs = &turn[i][8 * lane];
            if (a.interleaved) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 u = cs[e], w = cs[e + 4];
                    const float x0 = x[2 * e], y0 = y[2 * e];
                    x[2 * e] = fmaf(x0, u.x, -(x[2 * e + 1] * u.y));
                    x[2 * e + 1] = fmaf(x[2 * e + 1], u.x, x0 * u.y);
                    y[2 * e] = fmaf(y0, w.x, -(y[2 * e + 1] * w.y));
                    y[2 * e + 1] = fmaf(y[2 * e + 1], w.x, y0 * w.y);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float2 u = cs[e];
                    const float x0 = x[e];
                    x[e] = fmaf(x0, u.x, -(y[e] * u.y));
                    y[e] = fmaf(y[e], u.x, x0 * u.y);
                }
            }
        }
        if (kind == 0) {
            const long long row = (static_cast<long long>(b) * a.Hq + g) * a.m + i0 + i;
            if (mp_check(a.status, row, static_cast<long long>(a.B) * a.Hq * a.m, kSitePagedOut)) {
                T* dst = static_cast<T*>(a.q_out) + row * kD;
                store_row8(dst + da, x);
                store_row8(dst + db, y);
            }
            continue;
        }
        if (kind == 1 && a.k_out) {
            const long long row = (static_cast<long long>(b) * a.Hkv + g) * a.m + i0 + i;
            if (mp_check(a.status, row, static_cast<long long>(a.B) * a.Hkv * a.m, kSitePagedOut)) {
                C* dst = static_cast<C*>(a.k_out) + row * kD;
                store_row8(dst + da, x);
                store_row8(dst + db, y);
            }
        }
        const long long p = p0 + i;
        if (p < 0 || p >= cap) continue;
        const long long row = paged_row(a.pages, a.pages.table + static_cast<long long>(b) *
                                                                     a.pages.stride,
                                        static_cast<int>(p), a.Hkv, g);
        if (row >= 0 && mp_check(a.status, row, static_cast<long long>(a.pages.n_pages) * a.Hkv *
                                                    a.pages.page_size, kSitePagedRow)) {
            C* dst = static_cast<C*>(kind == 1 ? a.keys : a.values) + row * kD;
            store_row8(dst + da, x);
            store_row8(dst + db, y);
        }
    }
}

// A float32 cache, on CUDA cores: a warp takes groups of four tokens, a lane four dims of each. The NH scores of four
// tokens are summed over the lanes by a reduce-scatter, which leaves a score a lane (two lanes where
// NH = 4), the softmax steps are lane-parallel, weights come back through shared memory.
constexpr int kSimtWarps = 8;
constexpr int kSimtThreads = 32 * kSimtWarps;
constexpr int kSimtTile = 4 * kSimtWarps;        // tokens

template <int NH>
__global__ void __launch_bounds__(kSimtThreads, 2) paged_attention_simt_kernel(const PArgs a) {
    __shared__ PlanSmem plan;
    __shared__ __align__(16) float weights[kSimtWarps][4 * NH + NH];
    __shared__ __align__(16) float join[kSimtWarps][NH][kPart];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    wait_for_predecessor();
    allow_dependents();
    Walk w = plan_run(a, plan);
    while (w.left > 0) {
        const int here = w.here(), g = w.unit / a.chunks, h0 = (w.unit - g * a.chunks) * NH;
        const int heads = min(NH, a.G - h0);
        const size_t row0 = static_cast<size_t>(w.b) * a.Hq + g * a.G + h0;
        const int32_t* slots = a.pages.table + static_cast<long long>(w.b) * a.pages.stride;
        float q[NH][4];
#pragma unroll
        for (int h = 0; h < NH; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                q[h][e] = h < heads ? load_elem(a.q, a.q_bf16, (row0 + h) * kD + 4 * lane + e) : 0.0f;
        // a group of tokens: four of one page (pages hold multiples of eight)
        float4 kn[4], vn[4];
        int live = 0;
        auto load = [&](int k) {
            const int tok = (w.t + k) * kSimtTile + 4 * warp;
            live = 0;
            if (k < here && tok < w.len) {
                const long long row = paged_row(a.pages, slots, tok, a.Hkv, g);
                if (row >= 0 && mp_check(a.status, row + 3, static_cast<long long>(a.pages.n_pages) *
                                                                a.Hkv * a.pages.page_size,
                                         kSitePagedRow))
                    live = min(4, w.len - tok);
                const float* kp = static_cast<const float*>(a.keys) + row * kD + 4 * lane;
                const float* vp = static_cast<const float*>(a.values) + row * kD + 4 * lane;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (i < live) {
                        kn[i] = *reinterpret_cast<const float4*>(kp + i * kD);
                        vn[i] = *reinterpret_cast<const float4*>(vp + i * kD);
                    } else {
                        kn[i] = vn[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    }
                }
            }
        };
        float m = -INFINITY, l = 0.0f, o[NH][4];
#pragma unroll
        for (int h = 0; h < NH; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[h][e] = 0.0f;
        load(0);
        for (int k = 0; k < here; ++k) {
            const int now = live;
            float v[4][4], s[4 * NH];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 x = kn[i];
                v[i][0] = vn[i].x;
                v[i][1] = vn[i].y;
                v[i][2] = vn[i].z;
                v[i][3] = vn[i].w;
#pragma unroll
                for (int h = 0; h < NH; ++h)
                    s[i * NH + h] = fmaf(x.w, q[h][3], fmaf(x.z, q[h][2],
                                                            fmaf(x.y, q[h][1], x.x * q[h][0])));
            }
            load(k + 1);
            if (now == 0) continue;
#pragma unroll
            for (int lv = 0; (16 >> lv) >= (NH == 8 ? 1 : 2); ++lv) {
                const int off = 16 >> lv, keep = (2 * NH) >> lv;
                const bool up = (lane & off) != 0;
#pragma unroll
                for (int i = 0; i < keep; ++i) {
                    const float send = up ? s[i] : s[i + keep];
                    s[i] = (up ? s[i + keep] : s[i]) + __shfl_xor_sync(0xffffffffu, send, off);
                }
            }
            float logit = s[0];
            if (NH == 4) logit += __shfl_xor_sync(0xffffffffu, logit, 1);
            logit = (lane >> 3) < now ? logit * a.scale : -INFINITY;
            float mt = fmaxf(logit, __shfl_xor_sync(0xffffffffu, logit, 8));
            mt = fmaxf(m, fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 16)));
            const float base = mt == -INFINITY ? 0.0f : mt;
            const float corr = exp2_fast(m - base), p = exp2_fast(logit - base);
            m = mt;
            l = fmaf(l, corr, p);
            const int at = NH == 8 ? lane : lane >> 1;                   // token NH + head
            weights[warp][at] = p;
            if (lane < 8) weights[warp][4 * NH + at] = corr;
            __syncwarp();
#pragma unroll
            for (int h = 0; h < NH; h += 4) {
                const float4 c = *reinterpret_cast<const float4*>(&weights[warp][4 * NH + h]);
                const float cc[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[h + j][e] *= cc[j];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int h = 0; h < NH; h += 4) {
                    const float4 c = *reinterpret_cast<const float4*>(&weights[warp][i * NH + h]);
                    const float pp[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[h + j][e] = fmaf(pp[j], v[i][e], o[h + j][e]);
                }
            __syncwarp();
        }
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        // ---- the warps' states, joined in order
        __syncthreads();                                                 // the last unit's are read
#pragma unroll
        for (int h = 0; h < NH; ++h)
            *reinterpret_cast<float4*>(&join[warp][h][4 * lane]) =
                make_float4(o[h][0], o[h][1], o[h][2], o[h][3]);
        if (lane < 8 && (NH == 8 || (lane & 1) == 0)) {
            join[warp][NH == 8 ? lane : lane >> 1][kD] = m;
            join[warp][NH == 8 ? lane : lane >> 1][kD + 1] = l;
        }
        __syncthreads();
        const int e = tid & (kD - 1);
        for (int h = tid / kD; h < heads; h += kSimtThreads / kD) {
            float M = -INFINITY, L = 0.0f, O = 0.0f;
#pragma unroll
            for (int i = 0; i < kSimtWarps; ++i) M = fmaxf(M, join[i][h][kD]);
            const float base = M == -INFINITY ? 0.0f : M;
#pragma unroll
            for (int i = 0; i < kSimtWarps; ++i) {
                const float c = exp2_fast(join[i][h][kD] - base);
                L = fmaf(c, join[i][h][kD + 1], L);
                O = fmaf(c, join[i][h][e], O);
            }
            if (here == w.tiles) {
                if (mp_check(a.status, static_cast<long long>(row0 + h),
                             static_cast<long long>(a.B) * a.Hq, kSitePagedOut))
                    a.out[(row0 + h) * kD + e] = L == 0.0f ? 0.0f : O / L;
            } else {
                float* p = part_of(a, w.t == 0, h);
                p[e] = O;
                if (e == 0) {
                    p[kD] = M;
                    p[kD + 1] = L;
                }
            }
        }
        w.next(a, here);
    }
}

// The parts of a query row, joined in a fixed order: warp w folds parts w, w + kJoinWarps, ...,
// kJoinAhead of them loaded at once, four dims a lane; then the warps in order. A part that holds
// nothing has m = -inf and zeros; NaN passes through its zero factor. A row that one CTA had to itself is
// left as that CTA wrote it; rows of a sequence of length 0 are zero.
constexpr int kJoinWarps = 8, kJoinAhead = 4;
__global__ void __launch_bounds__(32 * kJoinWarps) paged_join_kernel(const PArgs a) {
    __shared__ __align__(16) float join[kJoinWarps][kPart];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = blockIdx.x;
    const int b = row / a.Hq, h = row - b * a.Hq, g = h / a.G, ch = (h - g * a.G) / a.nh;
    const int hc = h - g * a.G - ch * a.nh, unit = g * a.chunks + ch, per_tile = a.Hkv * a.chunks;
    wait_for_predecessor();
    const int tiles = tiles_of(a, length_of(a, b));
    if (tiles == 0) {
        if (threadIdx.x < kD) a.out[static_cast<size_t>(row) * kD + threadIdx.x] = 0.0f;
        return;
    }
    const long long each = static_cast<long long>(per_tile) * tiles;
    const long long total = a.pages.lengths ? __ldcg(a.before + a.B) : each * a.B;
    const long long t0 = (a.pages.lengths ? __ldcg(a.before + b) : each * b) +
                         static_cast<long long>(unit) * tiles;
    const int shares = shares_of(a, total);
    const int c0 = share_with(total, shares, t0), c1 = share_with(total, shares, t0 + tiles - 1);
    if (c0 == c1) return;
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
            if (s <= c1) {
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
    if (mp_check(a.status, row, static_cast<long long>(a.B) * a.Hq, kSitePagedOut))
        a.out[static_cast<size_t>(row) * kD + e] = Ls == 0.0f ? 0.0f : Os / Ls;
}

constexpr int kSimtCtas = 2 * kSms;
int simt_heads(int G) { return G <= 4 ? 4 : 8; }

typedef void (*PFn)(const PArgs);
PFn pick_simt(int nh) {
    return nh == 4 ? paged_attention_simt_kernel<4> : paged_attention_simt_kernel<8>;
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
    // tokens a CTA: as many as leave two CTAs an SM; rows split over CTAs where there are fewer
    const int heads = a.Hq + 2 * Hkv;
    a.toks = 1;
    while (a.toks < kMaxToks && static_cast<long long>(B) * m >= 4ll * kSms * a.toks) a.toks *= 2;
    a.tok_blocks = (m + a.toks - 1) / a.toks;
    const long long blocks = static_cast<long long>(B) * a.tok_blocks;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
    const long long passes = (static_cast<long long>(heads) * a.toks + kAppRows - 1) / kAppRows;
    const unsigned split = static_cast<unsigned>(
        std::max<long long>(1, std::min<long long>(passes, 4 * kSms / std::max<long long>(blocks, 1))));
    return launch_dependent(pick_append(rows_bf16, cache.dtype == MP_BF16),
                            dim3(static_cast<unsigned>(blocks), split), dim3(kAppThreads), 0, st, a);
}

size_t paged_attention_scratch_bytes(int B, int Hq, int Hkv) {
    // of either kind of cache: who asks does not say which
    const size_t parts = std::max(kSimtCtas * simt_heads(Hq / Hkv),
                                  kPagedTcCtas * paged_tc_heads(Hq / Hkv));
    return parts * 2 * kPart * sizeof(float) + (static_cast<size_t>(B) + 1) * sizeof(long long);
}

cudaError_t launch_paged_attention(const void* q, bool q_bf16, const mp_paged& cache, int B, int Hq,
                                   int Hkv, int n, const int32_t* lengths, float scale, float* out,
                                   void* workspace, cudaStream_t st) {
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
    const bool tc = cache.dtype == MP_BF16;
    a.nh = tc ? paged_tc_heads(a.G) : simt_heads(a.G);
    a.chunks = (a.G + a.nh - 1) / a.nh;
    a.n = n;
    a.ctas = tc ? kPagedTcCtas : kSimtCtas;
    a.tile = tc ? kPagedTcTile : kSimtTile;
    a.scale = scale * 1.4426950408889634f;
    a.status = device_status_ptr();
    a.part = static_cast<float*>(workspace);
    a.before = reinterpret_cast<long long*>(a.part + static_cast<size_t>(a.ctas) * 2 * a.nh * kPart);
    const cudaError_t e = tc ? launch_paged_attention_tc(a, cache, st)
                             : launch_dependent(pick_simt(a.nh), dim3(a.ctas), dim3(kSimtThreads), 0,
                                                st, a);
    if (e != cudaSuccess) return e;
    return launch_dependent(paged_join_kernel, dim3(static_cast<unsigned>(B) * Hq),
                            dim3(32 * kJoinWarps), 0, st, a);
}

cudaError_t prepare_paged() {
    cudaFuncAttributes fa;
    cudaError_t e;
    for (int i = 0; i < 4; ++i) {
        if ((e = cudaFuncGetAttributes(&fa, pick_append(i & 1, i & 2))) != cudaSuccess) return e;
    }
    for (int nh : {4, 8})
        if ((e = cudaFuncGetAttributes(&fa, pick_simt(nh))) != cudaSuccess) return e;
    if ((e = prepare_paged_tc()) != cudaSuccess) return e;
    return cudaFuncGetAttributes(&fa, paged_join_kernel);
}

}  // namespace mp
