// A K/V cache held in 4 bits: rows written from bf16 or fp32 keys and values, rows read back, and
// exact attention of single query tokens over the cache. The pages keep K and V at the model's
// precision and have no counterpart; the layout is the one magicpig.h describes.
//
// A group of 64 dims x_e (two per row) is held by z, the largest bf16 <= min x, s, the smallest
// bf16 with z + 15 s >= max x, and codes c_e = rint((x_e - z) / s), so |x_e - (z + s c_e)| <= s / 2.
// 15 s is exact in float32 (8 + 4 bits), so that it reaches max - z exactly where it reaches that
// difference rounded up.
//
// The kernels are launched as dependents of what precedes them in the stream: their lives begin
// before it has written what they read. So no load here is a non-coherent one, which would promise
// that nobody writes its memory meanwhile; ordinary loads stay behind the wait.
#include <algorithm>

#include <cuda_fp16.h>

#include "mp_internal.cuh"

namespace mp {
namespace {

constexpr int kCodeBytes = MP_KV4_CODE_BYTES;
constexpr int kSms = 152;                        // of a GB300; a plan, and so a workspace's size,
                                                 // is the same on the host alone

__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float min_nan(float a, float b, float c) {
    float r;
    asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Two floats in one 64-bit register: the packed instructions halve the issue slots that the codes
// of a row take, which is what bounds their writing.
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 pack2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpack2(F2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// The high half of a float is a bf16: rounding down drops the low half, one step further from
// zero for a negative value whose low half is not 0.
__device__ __forceinline__ uint32_t bf16_below(float x) {
    const uint32_t u = __float_as_uint(x), t = u >> 16;
    return t + ((u >> 31) != 0u && (u & 0xffffu) != 0u ? 1u : 0u);
}

// s (low half) and z (high half) of a group from its minimum and maximum; NaN in both for a group
// that has no finite pair (min_nan and max_nan pass a NaN on). s starts at the bf16 below a product
// that is less than d / 15 by a millionth, so at most two steps below the smallest with 15 s >= d.
__device__ __forceinline__ uint32_t group_params(float lo, float hi) {
    const uint32_t z = bf16_below(lo);
    const float d = __fsub_ru(hi, __uint_as_float(z << 16));
    uint32_t s = __float_as_uint(d * 0.0666666f) >> 16;
    if (15.0f * __uint_as_float(s << 16) < d) ++s;
    if (15.0f * __uint_as_float(s << 16) < d) ++s;
    const bool finite = (z & 0x7f80u) != 0x7f80u && (s & 0x7f80u) < 0x7f80u && d < INFINITY;
    return finite ? (s | (z << 16)) : 0x7fc07fc0u;
}

// rint((x - z) / s), ties to even, decided in 64 bits where x lies next to a border. f is off by one
// at most; d = (x - z) - f s is exact around s / 2 (x - z rounded to 53 bits, as the definition has
// it), so the comparison decides as the rounded quotient would.
__device__ __noinline__ uint32_t code_exact(float x, float z, float s) {
    const float t = x - z;
    float f = rintf(__fdiv_rn(t, s));
    const float h = 0.5f * s;
    if (!(fabsf(fmaf(-f, s, t)) < h * (1.0f - 3.8e-6f)) || s < 1e-30f) {
        const double d = fma(-static_cast<double>(f), static_cast<double>(s),
                             static_cast<double>(x) - static_cast<double>(z));
        const double hd = 0.5 * static_cast<double>(s);
        const bool odd = static_cast<int>(f) & 1;
        if (d > hd || (d == hd && odd)) f += 1.0f;
        else if (d < -hd || (d == -hd && odd)) f -= 1.0f;
    }
    return static_cast<uint32_t>(static_cast<int>(f));
}

// The codes of a lane's kPairs pairs x of a group, in order, as words of eight.
// With t = x - z, the quotient t / s is rounded to an integer f by adding 1.5 2^23, and t - f s,
// which one fused multiply-add gives exactly near s / 2, tells whether f is the nearest integer.
// Values that are bf16 (kBf16) often lie half-way: 1 / s as two floats rounds their quotient
// properly first, so that the addition sends a tie to the even integer, and |t - f s| > s / 2 alone
// asks for 64 bits; t is exact then too, unless x is tiny and a border lies at x = 0. Other values
// ask for 64 bits within 2^-18 of a border; steps near the ends of float32's range do always.
template <bool kBf16, int kPairs>
__device__ __forceinline__ void codes_of(const F2 (&x)[kPairs], uint32_t pr,
                                         uint32_t (&w)[kPairs / 4]) {
    const float s = __uint_as_float(pr << 16), z = __uint_as_float(pr & 0xffff0000u);
    if (!(s > 0.0f)) {                           // constant, or not a number
#pragma unroll
        for (int k = 0; k < kPairs / 4; ++k) w[k] = 0u;
        return;
    }
    const F2 round = pack2(12582912.0f, 12582912.0f), back = pack2(-12582912.0f, -12582912.0f);
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
    const float low = fmaf(-s, inv, 1.0f) * inv;
    const F2 inv2 = pack2(inv, inv), low2 = pack2(low, low), minus_z = pack2(-z, -z),
             minus_s = pack2(-s, -s);
    float worst = 0.0f;
#pragma unroll
    for (int k = 0; k < kPairs / 4; ++k) {
        w[k] = 0u;
#pragma unroll
        for (int i = 3; i >= 0; --i) {
            const F2 t = add2(x[4 * k + i], minus_z);
            const F2 y = kBf16 ? add2(fma2(t, inv2, mul2(t, low2)), round) : fma2(t, inv2, round);
            const float2 off = unpack2(fma2(add2(y, back), minus_s, t));
            worst = fmaxf(fmaxf(worst, fabsf(off.x)), fabsf(off.y));
            // the low bits of y are its integer; what its high bits add up to is taken off below
            const float2 yf = unpack2(y);
            w[k] = (w[k] << 4) + __float_as_uint(yf.y);
            w[k] = (w[k] << 4) + __float_as_uint(yf.x);
        }
        w[k] -= 0x4b400000u * 0x11111111u;
    }
    bool ask = kBf16 ? worst > 0.5f * s : worst >= 0.5f * s * (1.0f - 3.8e-6f);
    ask = ask || s < 1e-30f || s > 1e30f;
    if (kBf16) {
        const float c = floorf(-z * inv);                        // is z + (c + 1/2) s = 0 ?
        if (c >= 0.0f && c < 15.0f && fmaf(c + 0.5f, s, z) == 0.0f) {
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                const float2 v = unpack2(x[i]);
                ask = ask || fabsf(v.x) < 1e-4f * s || fabsf(v.y) < 1e-4f * s;
            }
        }
    }
    if (ask) {
        const float near = 0.5f * s * (1.0f - 3.8e-6f);
        const bool all = s < 1e-30f || s > 1e30f;
        auto code = [&](float v) -> uint32_t {
            const float y = __fadd_rn(__fmul_rn(v - z, inv), 12582912.0f);
            if (all || !(fabsf(fmaf(12582912.0f - y, s, v - z)) < near)) return code_exact(v, z, s);
            return __float_as_uint(y) & 15u;
        };
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            const float2 v = unpack2(x[i]);
            const uint32_t pair = code(v.x) | (code(v.y) << 4);
            w[i >> 2] = (i & 3) == 0 ? pair : w[i >> 2] | (pair << (8 * (i & 3)));
        }
    }
}

struct RowArgs {
    const void* keys;                            // of the rows to write; outputs of a read
    const void* values;
    const float* centre;
    const int32_t* positions;
    uint8_t* k_codes;
    uint8_t* v_codes;
    uint8_t* params;
    uint32_t rows;                               // B * Hkv * m
    uint32_t blocks;                             // of kRowThreads / (lanes a row) rows
    uint32_t m;
    int Hkv, n_begin, ncap;
    int* status;                                 // index checks of the MP_CHECKS build
};

constexpr int kRowThreads = 256;
// Lanes a row of 128 dims: 8 with 16 dims each, or, to write many bf16 rows, 4 with 32 dims each:
// what a lane does once for its dims (bounds, parameters, addresses) took more issue slots than
// their codes (786432 rows: 111 us with 8 lanes, 96 us with 4). The longer code starts later: 256
// rows take 2.9 us with 8 lanes, 4.1 us with 4.
constexpr int kReadLanes = 8;
constexpr uint32_t kManyRows = 2 * kSms * (kRowThreads / 4);     // two CTAs an SM of 4-lane rows
int write_lanes(bool bf16, uint32_t rows) { return bf16 && rows >= kManyRows ? 4 : 8; }

// Where a lane's row of block `blk` (kRowThreads / kLanes rows) is: head and token in the call, row
// of the cache over all heads (-1: outside the cache, or past the call's rows). A block spans two heads at
// most where a head has more rows than a block: one division, of uniform numbers, does then.
struct RowAt {
    uint32_t r, bh;
    long long row;
};
template <int kLanes>
__device__ __forceinline__ RowAt row_at(const RowArgs& a, uint32_t blk) {
    constexpr uint32_t kRowsPerCta = kRowThreads / kLanes;
    const uint32_t r0 = blk * kRowsPerCta, r = r0 + threadIdx.x / kLanes;
    RowAt w;
    w.r = min(r, a.rows - 1u);
    uint32_t i;
    if (a.m >= kRowsPerCta) {
        w.bh = r0 / a.m;
        i = w.r - w.bh * a.m;
        if (i >= a.m) {
            ++w.bh;
            i -= a.m;
        }
    } else {
        w.bh = w.r / a.m;
        i = w.r - w.bh * a.m;
    }
    const long long pos =
        static_cast<long long>(a.positions ? a.positions[w.bh / a.Hkv] : a.n_begin) + i;
    w.row = r < a.rows && pos >= 0 && pos < a.ncap
                ? static_cast<long long>(w.bh) * a.ncap + pos : -1;
    return w;
}

__device__ __forceinline__ long long cache_rows(const RowArgs& a) {
    return static_cast<long long>(a.rows / a.m) * a.ncap;
}

// 32 bytes of a row: one access where they are aligned (kWide: a whole sector a lane; two accesses
// of 16 bytes touch every sector twice), else two.
template <bool kWide>
__device__ __forceinline__ void load32(const void* p, uint32_t* w) {
    if constexpr (kWide) {
        asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                       "=r"(w[6]), "=r"(w[7])
                     : "l"(p));
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4 v = static_cast<const uint4*>(p)[i];
            w[4 * i] = v.x;
            w[4 * i + 1] = v.y;
            w[4 * i + 2] = v.z;
            w[4 * i + 3] = v.w;
        }
    }
}
template <bool kWide>
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
    if constexpr (kWide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
                     "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            static_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2],
                                                   w[4 * i + 3]);
    }
}

__device__ __forceinline__ F2 of_bf16x2(uint32_t w) {
    return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
// The least and the largest of a lane's dims (NaN if one is)
template <int kPairs>
__device__ __forceinline__ float2 bounds_of(const F2 (&x)[kPairs]) {
    const float2 v = unpack2(x[0]);
    float lo = min_nan(v.x, v.y), hi = max_nan(v.x, v.y);
#pragma unroll
    for (int i = 1; i < kPairs; ++i) {
        const float2 u = unpack2(x[i]);
        lo = min_nan(lo, u.x, u.y);
        hi = max_nan(hi, u.x, u.y);
    }
    return make_float2(lo, hi);
}
// The same of bf16 pairs as they are in memory
template <int kPairs>
__device__ __forceinline__ float2 bounds_of(const uint32_t (&w)[kPairs]) {
    uint32_t lo = w[0], hi = w[0];
#pragma unroll
    for (int i = 1; i < kPairs; ++i) {
        asm("min.NaN.bf16x2 %0, %0, %1;" : "+r"(lo) : "r"(w[i]));
        asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(hi) : "r"(w[i]));
    }
    return make_float2(min_nan(__uint_as_float(lo << 16), __uint_as_float(lo & 0xffff0000u)),
                       max_nan(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u)));
}

// The parameters of a group from the bounds of its kLanes lanes.
template <int kLanes>
__device__ __forceinline__ uint32_t lanes_params(float2 v) {
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) {
        v.x = min_nan(v.x, __shfl_xor_sync(0xffffffffu, v.x, o));
        v.y = max_nan(v.y, __shfl_xor_sync(0xffffffffu, v.y, o));
    }
    return group_params(v.x, v.y);
}
template <int kWords>
__device__ __forceinline__ void store_codes(uint8_t* p, const uint32_t (&w)[kWords]) {
    if constexpr (kWords == 4)
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}

// A CTA takes every gridDim.x-th block of rows and loads the next block's keys and values before it
// codes the ones it has: with a block a CTA and no loop, a third of the time went by between a
// warp's loads and its stores. 786432 rows of bf16 (8 heads x 96K tokens) take 98 us (5.3 TB/s; the
// bytes alone 76 us) and are bound by issue slots and by the arithmetic pipes; fp32 rows, with
// twice the bytes, by memory (524288 rows: 94 us, 6.5 TB/s).
template <typename T, bool kWide, int kLanes>
__global__ void __launch_bounds__(kRowThreads, sizeof(T) == 2 && kLanes == 8 ? 3 : 2)
    kv4_write_kernel(const RowArgs a) {
    constexpr bool kBf16 = sizeof(T) == 2;
    constexpr int kDims = kD / kLanes, kPairs = kDims / 2;
    constexpr int kWords = kDims * sizeof(T) / 4;
    const int rl = threadIdx.x & (kLanes - 1);
    const F2 minus = pack2(-1.0f, -1.0f);
    uint32_t kw[kWords], vw[kWords];
    auto load = [&](uint32_t r) {
        const size_t at = static_cast<size_t>(r) * kD + kDims * rl;
#pragma unroll
        for (int j = 0; j < kWords / 8; ++j) {
            load32<kWide>(static_cast<const T*>(a.keys) + at + j * (32 / sizeof(T)), kw + 8 * j);
            load32<kWide>(static_cast<const T*>(a.values) + at + j * (32 / sizeof(T)), vw + 8 * j);
        }
    };
    auto pairs_of = [](const uint32_t (&w)[kWords], F2 (&x)[kPairs]) {
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            if constexpr (kBf16) x[j] = of_bf16x2(w[j]);
            else x[j] = pack2(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
        }
    };
    wait_for_predecessor();
    RowAt w = row_at<kLanes>(a, blockIdx.x);
    load(w.r);
    for (uint32_t blk = blockIdx.x; blk < a.blocks; blk += gridDim.x) {
        F2 x[kPairs], v[kPairs];
        pairs_of(kw, x);
        pairs_of(vw, v);
        float2 vb;
        if constexpr (kBf16) vb = bounds_of(vw);
        else vb = bounds_of(v);
        const RowAt now = w;
        if (blk + gridDim.x < a.blocks) {
            w = row_at<kLanes>(a, blk + gridDim.x);
            load(w.r);
        }
        if (a.centre) {
            const float4* mu = reinterpret_cast<const float4*>(
                a.centre + static_cast<size_t>(now.bh) * kD + kDims * rl);
#pragma unroll
            for (int j = 0; j < kPairs / 2; ++j) {
                const float4 c = mu[j];
                x[2 * j] = fma2(pack2(c.x, c.y), minus, x[2 * j]);       // k - c, one rounding
                x[2 * j + 1] = fma2(pack2(c.z, c.w), minus, x[2 * j + 1]);
            }
        }
        const uint32_t kp = lanes_params<kLanes / 2>(bounds_of(x));
        const uint32_t vp = lanes_params<kLanes / 2>(vb);
        uint32_t kc[kPairs / 4], vc[kPairs / 4];
        codes_of<false>(x, kp, kc);
        codes_of<kBf16>(v, vp, vc);
        const uint32_t kp1 = __shfl_down_sync(0xffffffffu, kp, kLanes / 2);
        const uint32_t vp1 = __shfl_down_sync(0xffffffffu, vp, kLanes / 2);
        if (now.row >= 0 && mp_check(a.status, now.row, cache_rows(a), kSiteKv4Row)) {
            store_codes(a.k_codes + now.row * kCodeBytes + kDims / 2 * rl, kc);
            store_codes(a.v_codes + now.row * kCodeBytes + kDims / 2 * rl, vc);
            if (rl == 0)
                *reinterpret_cast<uint4*>(a.params + now.row * 16) = make_uint4(kp, kp1, vp, vp1);
        }
    }
}

template <bool kWide>
__device__ __forceinline__ void store16(float* p, const float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = __float_as_uint(x[8 * i + k]);
        store32<kWide>(p + 8 * i, w);
    }
}
template <bool kWide>
__device__ __forceinline__ void store16(__nv_bfloat16* p, const float (&x)[16]) {
    uint32_t w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
        w[k] = *reinterpret_cast<const uint32_t*>(&h);
    }
    store32<kWide>(p, w);
}

// z + s c, one rounding
__device__ __forceinline__ void values16(uint2 c, uint32_t pr, float (&x)[16]) {
    const float s = __uint_as_float(pr << 16), z = __uint_as_float(pr & 0xffff0000u);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const uint32_t n = ((i < 8 ? c.x : c.y) >> (4 * (i & 7))) & 15u;
        x[i] = fmaf(s, __uint_as_float(n | 0x4b000000u) - 8388608.0f, z);
    }
}

// Eight lanes a row, the next block's codes loaded before a block is stored. Bound by memory, most
// of it stores: 786432 rows to bf16 take 87 us (5.9 TB/s), 524288 rows to fp32 105-109 us.
template <typename T, bool kWide>
__global__ void __launch_bounds__(kRowThreads) kv4_read_kernel(const RowArgs a) {
    const int rl = threadIdx.x & (kReadLanes - 1);
    uint2 kc, vc;
    uint32_t kp, vp;
    auto load = [&](long long row) {
        kc = vc = make_uint2(0u, 0u);
        kp = vp = 0u;
        if (row >= 0 && mp_check(a.status, row, cache_rows(a), kSiteKv4Row)) {
            kc = *reinterpret_cast<const uint2*>(a.k_codes + row * kCodeBytes + 8 * rl);
            vc = *reinterpret_cast<const uint2*>(a.v_codes + row * kCodeBytes + 8 * rl);
            const uint32_t* p = reinterpret_cast<const uint32_t*>(a.params + row * 16) + (rl >> 2);
            kp = p[0];
            vp = p[2];
        }
    };
    wait_for_predecessor();
    RowAt w = row_at<kReadLanes>(a, blockIdx.x);
    load(w.row);
    for (uint32_t blk = blockIdx.x; blk < a.blocks; blk += gridDim.x) {
        const RowAt now = w;
        float k[16], v[16];
        values16(kc, kp, k);
        values16(vc, vp, v);
        if (blk + gridDim.x < a.blocks) {
            w = row_at<kReadLanes>(a, blk + gridDim.x);
            load(w.row);
        }
        if (a.centre && now.row >= 0) {
            const float4* mu = reinterpret_cast<const float4*>(
                a.centre + static_cast<size_t>(now.bh) * kD + 16 * rl);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 c = mu[i];
                k[4 * i] = __fadd_rn(k[4 * i], c.x);
                k[4 * i + 1] = __fadd_rn(k[4 * i + 1], c.y);
                k[4 * i + 2] = __fadd_rn(k[4 * i + 2], c.z);
                k[4 * i + 3] = __fadd_rn(k[4 * i + 3], c.w);
            }
        }
        if (blk * (kRowThreads / kReadLanes) + threadIdx.x / kReadLanes < a.rows &&
            mp_check(a.status, now.r, a.rows, kSiteKv4Out)) {
            const size_t at = static_cast<size_t>(now.r) * kD + 16 * rl;
            store16<kWide>(static_cast<T*>(const_cast<void*>(a.keys)) + at, k);
            store16<kWide>(static_cast<T*>(const_cast<void*>(a.values)) + at, v);
        }
    }
}

// ------------------------------------------------------------------------------------------------
// Exact attention of one query token per sequence.
//
// With a key's codes c, step s and minimum z per group, q.k = sum_g s_g (sum_e q_e c_e) + z_g sum_e
// q_e, and the value sum likewise: the products of codes with queries and of codes with weights
// are matrix products of small exact integers, which the warp's tensor-core instruction m16n8k16
// (fp16 in, fp32 sums) takes with the 16 tokens or 16 dims as its rows and the query heads as its
// eight columns, each number of theirs as two fp16 halves (22 bits): two columns a head (up to four
// heads, NT = 1), or a column a head and two products (up to eight, NT = 2, over the same unpacked
// codes). Steps and minima join outside, in fp32.
// The tcgen05 instructions want 128 rows and operands unpacked into shared memory, where a byte of
// codes would become four; here codes go from shared memory to fragments in registers, three
// quarters of an instruction of unpacking a value.
//
// A warp takes tiles of 64 tokens on its own, two in flight (cp.async; rows of 64 bytes whose
// 16-byte pieces are exchanged so that ldmatrix meets no bank conflict): logits of the tile, one
// step of the running maximum, weights, weighted codes summed from zero and added to the running
// sums in fp32. The tensor core's own sums round toward zero. They are kept short, and near zero:
// the codes of tokens 8-15 of a fragment enter as 15 - c under negative weights, and what that and
// the minima make up, sum w z over tokens 0-7 and sum w (z + 15 s) over tokens 8-15, is summed in
// fp32 token by token, where the two cancel as well. Without it the mean code of 7.5 times the
// weights would stand against a sum that is 100 times smaller, and its rounding with it. (z + 15 s
// may pass the largest float32 where the values held do not, from 2^126 on, which the header names:
// sums of halves of it took 1.5% longer over 2 x 64/8 heads x 128K tokens, 68.7 against 67.7 us.)
// ------------------------------------------------------------------------------------------------
struct A4Args {
    const void* q;
    const uint8_t* k_codes;
    const uint8_t* v_codes;
    const uint8_t* params;
    const int32_t* lengths;
    float* part;                                 // [row][split][kPart]: o, m, l
    float* out;
    int q_bf16, q_wide, Hq, Hkv, G, n, ncap, splits, chunks, cluster;
    int tiles_per_split;
    float scale;                                 // of q.k, times log2 e
    long long rows;                              // B * Hq
    int* status;                                 // index checks of the MP_CHECKS build
};
constexpr int kPart = kD + 4;
constexpr int kAttWarps = 4;
constexpr int kAttThreads = 32 * kAttWarps;
constexpr int kTile = 64;                        // tokens of a warp's tile
constexpr int kSub = kTile / 16;                 // fragments of 16 tokens in it
constexpr int kParamBytes = 2 * MP_KV4_PARAMS;
constexpr int kStageK = 0, kStageV = kTile * kCodeBytes, kStageP = 2 * kTile * kCodeBytes;
constexpr int kStageBytes = kStageP + kTile * kParamBytes;
constexpr int kAttStages = 2;
constexpr int kAttSmem = kAttWarps * kAttStages * kStageBytes;
constexpr int kClusterSplits = 8;                // up to so many splits are joined within a cluster
constexpr int kMergePitch = kD + 4;              // floats a (warp, head) leaves for the CTA's merge
static_assert(kAttThreads == kD, "the merge: a thread per dim");
static_assert((kAttWarps + 1) * 8 * kMergePitch * 4 <= kAttSmem, "the merge reuses the stages");

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// Zeros where the source is not live; `valid` stands in for its address then.
__device__ __forceinline__ void copy16_or_zero(uint32_t dst, const void* src, const void* valid,
                                               bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
                 "l"(live ? src : valid), "r"(live ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Eight codes of a word as four fp16 pairs: with c0 .. c3 the codes of its low half and c4 .. c7 of
// its high half, the pairs are (c0, c4) 2^-10, (c0 + 16 c1, c4 + 16 c5) 2^-24 and the same of c2, c3,
// c6, c7; the other matrix takes the sums of two codes apart again. A byte is a subnormal fp16 as
// it stands, which the tensor core takes but adds as if it were 2^-14 large: of a sum of two codes
// that costs c1 nothing (16 times smaller), but c0 by itself would keep 17 bits only (outputs off by
// 6e-6 instead of 6e-7), and is multiplied up to a normal number. Six instructions for eight codes,
// four of them on the integer pipe.
__device__ __forceinline__ void unpack_pairs(uint32_t w, uint32_t (&h)[4]) {
    h[1] = __byte_perm(w, 0u, 0x4240);
    h[3] = __byte_perm(w, 0u, 0x4341);
    h[0] = mul_f16x2(h[1] & 0x000f000fu, 0x74007400u);           // 2^14
    h[2] = mul_f16x2(h[3] & 0x000f000fu, 0x74007400u);
}

// The leading 11 bits of x; two floats as fp16
__device__ __forceinline__ float leading_bits(float x) {
    return __uint_as_float(__float_as_uint(x) & 0xffffe000u);
}
__device__ __forceinline__ uint32_t pack_f16(float low, float high) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(high), "f"(low));
    return r;
}

// What row r + 8 half of a lane's products holds for its head nt: the sum of two columns, or (NT = 2)
// one that has both halves' products
template <int NT>
__device__ __forceinline__ float head_of(const float (&c)[4], int half, int nt) {
    return NT == 1 ? c[2 * half] + c[2 * half + 1] : c[2 * half + nt];
}

// Eight elements of a query from element i on: the loads, where the queries are aligned for loads
// of 16 bytes, and later the values (zeros where there is no query).
struct Query8 {
    uint4 a, b;
};
__device__ __forceinline__ Query8 load_query8(const A4Args& a, size_t i, bool live) {
    Query8 v;
    v.a = v.b = make_uint4(0u, 0u, 0u, 0u);
    if (live && a.q_wide) {
        if (a.q_bf16) {
            v.a = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + i);
        } else {
            const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(a.q) + i);
            v.a = p[0];
            v.b = p[1];
        }
    }
    return v;
}
__device__ __forceinline__ void values_of(const Query8& v, const A4Args& a, size_t i, bool live,
                                          float (&x)[8]) {
    const uint32_t w[8] = {v.a.x, v.a.y, v.a.z, v.a.w, v.b.x, v.b.y, v.b.z, v.b.w};
    if (!a.q_wide) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = live ? load_elem(a.q, a.q_bf16, i + e) : 0.0f;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[e] = __uint_as_float(!a.q_bf16 ? w[e]
                                             : (e & 1) ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16);
    }
}

// One CTA per (head of keys and values, split of its tokens, chunk of 4 NT query heads of the
// group). Lane (r, t) = (lane / 4, lane % 4) holds query head t (2 t and 2 t + 1 where NT = 2) of the
// logits, weights and sums: tokens r and r + 8 of a fragment, dims 32 m + 4 r .. + 3.
//
// Four query heads a KV head: 32 sequences x 8 heads x 32K tokens take 199 us (6.1 TB/s, bound by
// memory), 1 x 8 x 96K 24.1 us, of which about 6 are the launch, the queries and the join. Eight:
// 2 x 8 x 128K take 66.7 us (4.5 TB/s); there a tile's arithmetic (1320 instructions a warp) takes
// longer than its bytes, at two CTAs an SM, for which the registers do. More than eight: every chunk
// of eight copies and unpacks the codes for itself (4 sequences x 128K tokens of one KV head with 8,
// 16 and 32 query heads: 25, 38 and 64 us). Like the other kernels here
// it is launched as a dependent of what precedes it in the stream and waits for that before its
// first access: queued calls follow each other 2 to 3 us sooner (1 x 8 x 96K 26.7 -> 23.7 us).
template <int NT>
__global__ void __launch_bounds__(kAttThreads, NT == 1 ? 3 : 2)
    kv4_attention_kernel(const A4Args a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = lane >> 2, t = lane & 3;
    const int split = static_cast<int>(blockIdx.x % a.splits);
    const unsigned ch = blockIdx.x / a.splits % a.chunks;
    const size_t bh = blockIdx.x / a.splits / a.chunks;
    const int b = static_cast<int>(bh / a.Hkv);
    const int h0 = static_cast<int>(ch) * 4 * NT;                        // first head of the chunk
    const size_t row0 = static_cast<size_t>(b) * a.Hq + bh % a.Hkv * a.G + h0;
    const int heads = min(4 * NT, a.G - h0);
    wait_for_predecessor();
    // the merge may start. Without one the dependent is another call, whose CTAs would take the
    // places of this one's that end first (4 x 8 heads of 16K tokens 18.5 -> 22.2 us)
    if (a.splits > 1 && !a.cluster) allow_dependents();
    const int len = a.lengths ? max(0, min(a.n, a.lengths[b])) : a.n;
    const int tile0 = split * a.tiles_per_split;
    const long long split_end = static_cast<long long>(tile0 + a.tiles_per_split) * kTile;
    int end = static_cast<int>(min(static_cast<long long>(len), split_end));     // tokens [.., end)
    if (!mp_check(a.status, end, static_cast<long long>(a.ncap) + 1, kSiteKv4Row)) end = 0;
    const int ntiles = (end - tile0 * kTile + kTile - 1) / kTile;        // <= 0: none
    const int mine = ntiles > warp ? (ntiles - warp + kAttWarps - 1) / kAttWarps : 0;

    const uint32_t stage0 = smem_u32(smem) + warp * kAttStages * kStageBytes;
    const uint8_t* kg = a.k_codes + bh * a.ncap * kCodeBytes;
    const uint8_t* vg = a.v_codes + bh * a.ncap * kCodeBytes;
    const uint8_t* pg = a.params + bh * a.ncap * kParamBytes;
    // a tile's copies: 16-byte piece lane % 4 of rows lane / 4 + 8 i to piece (lane % 4) ^
    // (row / 2 % 4); rows past the end read as zero
    const uint32_t swz = (lane >> 2) * kCodeBytes + (((lane & 3) ^ ((lane >> 3) & 3)) << 4);
    const size_t first = static_cast<size_t>(tile0 + warp) * kTile;
    const uint8_t* kp = kg + (first + (lane >> 2)) * kCodeBytes + 16 * (lane & 3);
    const uint8_t* vp = vg + (first + (lane >> 2)) * kCodeBytes + 16 * (lane & 3);
    const uint8_t* pp = pg + (first + lane) * kParamBytes;
    int left = end - static_cast<int>(first);    // tokens from the next tile to copy on
    auto issue = [&](int it) {
        const uint32_t st = stage0 + (it & 1) * kStageBytes;
        if (left >= kTile) {
#pragma unroll
            for (int i = 0; i < kTile / 8; ++i) {
                copy16(st + kStageK + 8 * i * kCodeBytes + swz, kp + 8 * i * kCodeBytes);
                copy16(st + kStageV + 8 * i * kCodeBytes + swz, vp + 8 * i * kCodeBytes);
            }
#pragma unroll
            for (int i = 0; i < kTile / 32; ++i)
                copy16(st + kStageP + (32 * i + lane) * kParamBytes, pp + 32 * i * kParamBytes);
        } else if (left > 0) {
#pragma unroll 1
            for (int i = 0; i < kTile / 8; ++i) {
                const bool live = 8 * i + (lane >> 2) < left;
                copy16_or_zero(st + kStageK + 8 * i * kCodeBytes + swz, kp + 8 * i * kCodeBytes, kg,
                               live);
                copy16_or_zero(st + kStageV + 8 * i * kCodeBytes + swz, vp + 8 * i * kCodeBytes, vg,
                               live);
            }
#pragma unroll 1
            for (int i = 0; i < kTile / 32; ++i)
                copy16_or_zero(st + kStageP + (32 * i + lane) * kParamBytes,
                               pp + 32 * i * kParamBytes, pg, 32 * i + lane < left);
        }
        kp += kAttWarps * kTile * kCodeBytes;
        vp += kAttWarps * kTile * kCodeBytes;
        pp += kAttWarps * kTile * kParamBytes;
        left -= kAttWarps * kTile;
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // the queries' loads first: behind the tiles of the whole GPU they would hold up the first step
    Query8 raw[4];
    const int qh = NT == 1 ? r >> 1 : r;                                 // this lane's column's head
#pragma unroll
    for (int m = 0; m < 4; ++m)
        raw[m] = load_query8(a, (row0 + qh) * kD + 32 * m + 8 * t, qh < heads);
    issue(0);
    issue(1);

    // ---- the queries as column fragments, qb[0] of the leading halves and qb[1] of the rest, a
    // column a head, or for NT = 1 qb[0] alone: column 2 h is head h's leading half, 2 h + 1 the rest.
    // A lane loads its column's head (dims 32 m + 8 t ..), scaled by a power of two so that the
    // largest element lies in [2^4, 2^5); fac undoes it on the logits, and the 2^-10 of the codes.
    // Against the pairs of unpack_pairs stand q0 - q1 / 16 and 2^14 q1 / 16.
    uint32_t qb[NT][4][4];
    float fac[NT], qsum[NT][2];
    {
        float x[4][8];
        uint32_t big = 0u;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            values_of(raw[m], a, (row0 + qh) * kD + 32 * m + 8 * t, qh < heads, x[m]);
#pragma unroll
            for (int e = 0; e < 8; ++e) big = max(big, __float_as_uint(x[m][e]) & 0x7fffffffu);
        }
        big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
        const uint32_t ex = min(max(big >> 23, 5u), 247u);
        const float down = __uint_as_float((258u - ex) << 23);
        const float up = __uint_as_float((ex + 6u) << 23);
        float sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int m = 0; m < 4; ++m) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[m][e] *= down;
                sum[m >> 1] += x[m][e];
            }
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                x[m][e] = fmaf(x[m][e + 1], -0.0625f, x[m][e]);
                x[m][e + 1] *= 1024.0f;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                // the leading half rounded to nearest, the rest
                const __half2 lead = __floats2half2_rn(x[m][e], x[m][e + 4]);
                const float2 lf = __half22float2(lead);
                const __half2 rem = __floats2half2_rn(x[m][e] - lf.x, x[m][e + 4] - lf.y);
                const __half2 first = NT == 1 && (r & 1) ? rem : lead;
                qb[0][m][e] = *reinterpret_cast<const uint32_t*>(&first);
                if constexpr (NT == 2) qb[1][m][e] = *reinterpret_cast<const uint32_t*>(&rem);
            }
        }
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 1);
            sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 2);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int from = 8 * t + 4 * nt;                             // a lane of the head's column
#pragma unroll
            for (int g = 0; g < 2; ++g)
                qsum[nt][g] = 0x1p-10f * __shfl_sync(0xffffffffu, sum[g], from);
            // not 0, which an infinite logit would turn into NaN; as a subnormal number it is off by
            // 2^-150, times logits of up to 2^126 within their own rounding
            fac[nt] = fmaxf(__shfl_sync(0xffffffffu, a.scale * up, from), 0x1p-149f);
        }
    }

    // running maximum of the logits as the products leave them, the same times fac
    float m_run[NT], base_run[NT], l_run[NT], mid_run[NT][2], o_run[NT][4][4], top[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        m_run[nt] = base_run[nt] = -INFINITY;
        l_run[nt] = mid_run[nt][0] = mid_run[nt][1] = top[nt][0] = top[nt][1] = 0.0f;
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) o_run[nt][m][e] = 0.0f;
    }
    // ldmatrix: matrices 0, 1 are the two pieces of a group of dims of tokens 0-7 of a fragment,
    // 2, 3 those of tokens 8-15; the other group's pieces differ in bit 5 of the address
    const uint32_t lm = (8 * (lane >> 4) + (lane & 7)) * kCodeBytes +
                        ((((lane >> 3) & 1) ^ ((lane >> 1) & 3)) << 4);

    for (int it = 0; it < mine; ++it) {
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncwarp();
        const uint32_t st = stage0 + (it & 1) * kStageBytes;
        const uint8_t* prm = smem + (st - smem_u32(smem)) + kStageP + r * kParamBytes;
        const int key0 = (tile0 + warp + it * kAttWarps) * kTile;

        // ---- logits (fac of them, base 2) of tokens 16 j + r and 16 j + 8 + r, a group at a time
        float lg[NT][2 * kSub];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            float c[kSub][4];
            uint32_t kw[kSub][4];
#pragma unroll
            for (int j = 0; j < kSub; ++j) {
                ldmatrix4(kw[j], st + kStageK + 16 * j * kCodeBytes + (lm ^ (g << 5)));
#pragma unroll
                for (int e = 0; e < 4; ++e) c[j][e] = 0.0f;
            }
            // the fragments' products side by side: those of one fragment wait for each other
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                uint32_t x0[kSub][4], x1[kSub][4];
#pragma unroll
                for (int j = 0; j < kSub; ++j) {
                    unpack_pairs(kw[j][m], x0[j]);
                    unpack_pairs(kw[j][m + 2], x1[j]);
                }
#pragma unroll
                for (int nt = NT - 1; nt >= 0; --nt)
#pragma unroll
                    for (int i = 0; i < 4; i += 2)
#pragma unroll
                        for (int j = 0; j < kSub; ++j)
                            mma16816(c[j], x0[j][i], x1[j][i], x0[j][i + 1], x1[j][i + 1],
                                     qb[nt][2 * g + m][i], qb[nt][2 * g + m][i + 1]);
            }
#pragma unroll
            for (int i = 0; i < 2 * kSub; ++i) {
                const uint32_t p =
                    *reinterpret_cast<const uint32_t*>(prm + 8 * i * kParamBytes + 4 * g);
                const float s = __uint_as_float(p << 16), z = __uint_as_float(p & 0xffff0000u);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float u = g == 0 ? z * qsum[nt][g] : fmaf(z, qsum[nt][g], lg[nt][i]);
                    lg[nt][i] = fmaf(s, head_of<NT>(c[i >> 1], i & 1, nt), u);
                }
            }
        }
        if (key0 + kTile > end) {
#pragma unroll
            for (int i = 0; i < 2 * kSub; ++i)
                if (key0 + 8 * i + r >= end)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) lg[nt][i] = -INFINITY;
        }

        // ---- one step of the running softmax; weights in place of the logits
        float corr[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float mt = lg[nt][0];
#pragma unroll
            for (int i = 1; i < 2 * kSub; ++i) mt = fmaxf(mt, lg[nt][i]);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
            const float mn = fmaxf(m_run[nt], mt);
            const float base = mn == -INFINITY ? 0.0f : mn * fac[nt];
            corr[nt] = exp2_fast(base_run[nt] - base);
            m_run[nt] = mn;
            base_run[nt] = mn == -INFINITY ? -INFINITY : base;
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 2 * kSub; ++i) {
                lg[nt][i] = exp2_fast(fmaf(lg[nt][i], fac[nt], -base));
                sum += lg[nt][i];
            }
            l_run[nt] = fmaf(l_run[nt], corr[nt], sum);
        }

        // ---- weighted codes of the tile, a group at a time. Weights times steps become fp16
        // halves, scaled by a power of two, 2^(138 - ex), which brings the head's largest product so
        // far (`top`, in units of the present base) to [2^11, 2^12); 2^(ex - 138) takes it back,
        // with the 2^-10 of the codes. Where a step exceeds 8 top, which its weight may undo, the
        // tile's own products are looked at: a head's tokens are held to 2^-36 of a product that
        // its sum contains, whatever the steps of tokens without weight and other heads' weights.
        // (By the tile's largest step alone a token of no weight, 2^34 times larger than the rest,
        // moved outputs by 3%.) Looking at every tile's products costs 3% (8 x 96K tokens 24.6
        // against 24.2 us, 32 x 8 x 32K 206 against 199). NaN is not the largest of anything and
        // goes through.
        {
            uint32_t vmax[2] = {0u, 0u};
#pragma unroll
            for (int i = 0; i < 2 * kSub; ++i) {
                const uint2 p = *reinterpret_cast<const uint2*>(prm + 8 * i * kParamBytes + 8);
                vmax[0] = __vmaxu2(vmax[0], p.x);
                vmax[1] = __vmaxu2(vmax[1], p.y);
            }
            bool above = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    top[nt][g] *= corr[nt];
                    above = above || !(__uint_as_float(vmax[g] << 16) <= 8.0f * top[nt][g]);
                }
            if (__any_sync(0xffffffffu, above)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int i = 0; i < 2 * kSub; ++i) {
                        const uint2 p =
                            *reinterpret_cast<const uint2*>(prm + 8 * i * kParamBytes + 8);
                        top[nt][0] = fmaxf(top[nt][0], lg[nt][i] * __uint_as_float(p.x << 16));
                        top[nt][1] = fmaxf(top[nt][1], lg[nt][i] * __uint_as_float(p.y << 16));
                    }
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) {
                        top[nt][0] = fmaxf(top[nt][0], __shfl_xor_sync(0xffffffffu, top[nt][0], o));
                        top[nt][1] = fmaxf(top[nt][1], __shfl_xor_sync(0xffffffffu, top[nt][1], o));
                    }
                }
            }
        }
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            uint32_t pw[2 * kSub];
#pragma unroll
            for (int i = 0; i < 2 * kSub; ++i)
                pw[i] = *reinterpret_cast<const uint32_t*>(prm + 8 * i * kParamBytes + 8 + 4 * g);
            float down[NT], up[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const uint32_t ex = max(__float_as_uint(top[nt][g]) >> 23, 14u);
                down[nt] = __uint_as_float((265u - ex) << 23);
                up[nt] = __uint_as_float((ex - 1u) << 23);
            }
            float acc[2][2][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mid_run[nt][g] *= corr[nt];
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[m][i][e] = 0.0f;
#pragma unroll
            for (int j = 0; j < kSub; ++j) {
                uint32_t vw[4], x[4][4], wb[NT][2];
                ldmatrix4_trans(vw, st + kStageV + 16 * j * kCodeBytes + (lm ^ (g << 5)));
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const uint32_t p = pw[2 * j + half];
                    const float s = __uint_as_float(p << 16);
                    float mid = __uint_as_float(p & 0xffff0000u);
                    if (half) mid = fmaf(15.0f, s, mid);
                    float w[NT], lead[NT];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const float u = lg[nt][2 * j + half];
                        mid_run[nt][g] = fmaf(u, mid, mid_run[nt][g]);
                        w[nt] = u * s * (half ? -down[nt] : down[nt]);
                        lead[nt] = leading_bits(w[nt]);
                    }
                    if constexpr (NT == 1) {
                        wb[0][half] = transpose8x8(pack_f16(lead[0], w[0] - lead[0]));
                    } else {
                        wb[0][half] = transpose8x8(pack_f16(lead[0], lead[1]));
                        wb[1][half] = transpose8x8(pack_f16(w[0] - lead[0], w[1] - lead[1]));
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) unpack_pairs(i < 2 ? vw[i] : ~vw[i], x[i]);
#pragma unroll
                for (int nt = NT - 1; nt >= 0; --nt)             // the rests first: they round less
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            mma16816(acc[m][i], x[m][2 * i], x[m][2 * i + 1], x[m + 2][2 * i],
                                     x[m + 2][2 * i + 1], wb[nt][0], wb[nt][1]);
            }
            if (g == 1) {
                __syncwarp();
                issue(it + 2);
            }
            // the second row of a pair holds its own dim's sum 16 times and the first one's once,
            // in units 2^14 smaller
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float one = head_of<NT>(acc[m][i], 0, nt);
                        const float two = fmaf(head_of<NT>(acc[m][i], 1, nt), 16384.0f, -one);
                        float* o = &o_run[nt][2 * g + m][2 * i];
                        o[0] = fmaf(one, up[nt], o[0] * corr[nt]);
                        o[1] = fmaf(two, up[nt] * 0.0625f, o[1] * corr[nt]);
                    }
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");

    // ---- sums over the lanes of a head, then the CTA's four warps in order
    __syncthreads();
    float* join = reinterpret_cast<float*>(smem);        // [head][warp][kMergePitch]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            l_run[nt] += __shfl_xor_sync(0xffffffffu, l_run[nt], o);
            mid_run[nt][0] += __shfl_xor_sync(0xffffffffu, mid_run[nt][0], o);
            mid_run[nt][1] += __shfl_xor_sync(0xffffffffu, mid_run[nt][1], o);
        }
        float* dst = join + ((NT * t + nt) * kAttWarps + warp) * kMergePitch;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const float mid = mid_run[nt][m >> 1];
            const float (&o)[4] = o_run[nt][m];
            *reinterpret_cast<float4*>(dst + 32 * m + 4 * r) =
                make_float4(o[0] + mid, o[1] + mid, o[2] + mid, o[3] + mid);
        }
        if (r == 0) {
            dst[kD] = base_run[nt];
            dst[kD + 1] = l_run[nt];
        }
    }
    __syncthreads();
    const int e = threadIdx.x;
    float* share = join + 4 * NT * kAttWarps * kMergePitch;              // [head][kMergePitch]
    for (int h = 0; h < heads; ++h) {
        const float* src = join + h * kAttWarps * kMergePitch;
        float M = -INFINITY, L = 0.0f, O = 0.0f;
#pragma unroll
        for (int w = 0; w < kAttWarps; ++w) M = fmaxf(M, src[w * kMergePitch + kD]);
#pragma unroll
        for (int w = 0; w < kAttWarps; ++w) {
            const float mw = src[w * kMergePitch + kD];
            const float s = mw == -INFINITY ? 0.0f : exp2_fast(mw - M);  // empty: zeros
            L = fmaf(s, src[w * kMergePitch + kD + 1], L);
            O = fmaf(s, src[w * kMergePitch + e], O);
        }
        if (!mp_check(a.status, static_cast<long long>(row0 + h), a.rows, kSiteKv4Out)) continue;
        if (a.splits == 1) {
            a.out[(row0 + h) * kD + e] = L == 0.0f ? 0.0f : O / L;
        } else if (a.cluster) {
            float* p = share + h * kMergePitch;
            p[e] = O;
            if (e == 0) {
                p[kD] = M;
                p[kD + 1] = L;
            }
        } else {
            float* p = a.part + ((row0 + h) * a.splits + split) * kPart;
            p[e] = O;
            if (e == 0) {
                p[kD] = M;
                p[kD + 1] = L;
            }
        }
    }
    // few splits are one cluster: each CTA joins some of the heads from the CTAs' shared memory
    // (against the second kernel: 4 x 8 heads of 16K tokens 18.8 -> 18.4 us, 16 sequences of up to
    // 5000 22.5 -> 21.0 us, and a launch less; not over several waves, where the CTAs of a cluster
    // would hold their places until the longest is done: 155 us against 176 us for 32 sequences of
    // 16K to 32K tokens)
    if (a.cluster) {
        cluster_barrier();
        for (int h = split; h < heads; h += a.splits) {
            const uint32_t at = smem_u32(share + h * kMergePitch);
            float ms[kClusterSplits], ls[kClusterSplits], os[kClusterSplits], M = -INFINITY;
#pragma unroll
            for (int s = 0; s < kClusterSplits; ++s) {
                ms[s] = -INFINITY;
                ls[s] = os[s] = 0.0f;
                if (s < a.splits) {
                    const uint32_t there = peer_address(at, s);
                    ms[s] = load_peer(there + 4 * kD);
                    ls[s] = load_peer(there + 4 * (kD + 1));
                    os[s] = load_peer(there + 4 * e);
                }
                M = fmaxf(M, ms[s]);
            }
            const float base = M == -INFINITY ? 0.0f : M;
            float L = 0.0f, O = 0.0f;
#pragma unroll
            for (int s = 0; s < kClusterSplits; ++s) {
                const float c = exp2_fast(ms[s] - base);
                L = fmaf(c, ls[s], L);
                O = fmaf(c, os[s], O);
            }
            a.out[(row0 + h) * kD + e] = L == 0.0f ? 0.0f : O / L;
        }
        cluster_barrier();                       // no CTA leaves while another reads from it
    }
}

// The splits of a query row, joined in a fixed order: warp w folds splits w, w + kMergeWarps, ...,
// kMergeAhead of them loaded at once, four dims a lane; then the warps in order. A split that
// holds nothing has m = -inf and zeros; NaN passes through its zero factor.
constexpr int kMergeWarps = 16, kMergeAhead = 4;
__global__ void __launch_bounds__(32 * kMergeWarps) kv4_merge_kernel(const A4Args a) {
    __shared__ __align__(16) float join[kMergeWarps][kMergePitch];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, splits = a.splits;
    const size_t row = blockIdx.x;
    wait_for_predecessor();
    const float* p = a.part + row * splits * kPart;
    float M = -INFINITY, L = 0.0f;
    float4 O = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int s0 = warp; s0 < splits; s0 += kMergeWarps * kMergeAhead) {
        float ms[kMergeAhead], ls[kMergeAhead];
        float4 os[kMergeAhead];
#pragma unroll
        for (int i = 0; i < kMergeAhead; ++i) {
            const int s = s0 + i * kMergeWarps;
            ms[i] = -INFINITY;
            ls[i] = 0.0f;
            os[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (s < splits) {
                const float* ps = p + static_cast<size_t>(s) * kPart;
                ms[i] = __ldcg(ps + kD);
                ls[i] = __ldcg(ps + kD + 1);
                os[i] = __ldcg(reinterpret_cast<const float4*>(ps) + lane);
            }
        }
        float mn = M;
#pragma unroll
        for (int i = 0; i < kMergeAhead; ++i) mn = fmaxf(mn, ms[i]);
        const float base = mn == -INFINITY ? 0.0f : mn;
        const float c = exp2_fast(M - base);
        M = mn;
        L *= c;
        O = make_float4(O.x * c, O.y * c, O.z * c, O.w * c);
#pragma unroll
        for (int i = 0; i < kMergeAhead; ++i) {
            const float w = exp2_fast(ms[i] - base);
            L = fmaf(w, ls[i], L);
            O = make_float4(fmaf(w, os[i].x, O.x), fmaf(w, os[i].y, O.y), fmaf(w, os[i].z, O.z),
                            fmaf(w, os[i].w, O.w));
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
    for (int w = 0; w < kMergeWarps; ++w) M = fmaxf(M, join[w][kD]);
    const float base = M == -INFINITY ? 0.0f : M;
    float Ls = 0.0f, Os = 0.0f;
#pragma unroll
    for (int w = 0; w < kMergeWarps; ++w) {
        const float c = exp2_fast(join[w][kD] - base);
        Ls = fmaf(c, join[w][kD + 1], Ls);
        Os = fmaf(c, join[w][e], Os);
    }
    a.out[row * kD + e] = Ls == 0.0f ? 0.0f : Os / Ls;
}

// How an attention call is laid over the GPU.
struct AttPlan {
    int nt, chunks, splits, tiles_per_split;
    bool cluster;                                // the splits of a unit are one cluster
};
constexpr int kPlans = 6;                        // no split; k CTAs an SM; waves of `resident`
int plan_ctas(int k, int resident) { return k <= resident ? k : (k - resident + 1) * resident; }
int resident_ctas(int nt) { return nt == 1 ? 3 : 2; }
int steps_of(int n) { return (n - 1) / (kTile * kAttWarps) + 1; }
int heads_plan(int G, int* nt) {                 // chunks of query heads, of 4 nt each
    *nt = G <= 4 ? 1 : 2;
    return (G + 4 * *nt - 1) / (4 * *nt);
}
// The most splits that attention_plan takes for n tokens or fewer
long long most_splits(int B, int Hq, int Hkv, int n) {
    int nt;
    const long long units = static_cast<long long>(B) * Hkv * heads_plan(Hq / Hkv, &nt);
    return std::min<long long>({256, kSms * plan_ctas(kPlans - 1, resident_ctas(nt)) / units,
                                steps_of(n)});
}
// How many splits: the least of a model of a call's time, in units of 10 ns, over the counts that
// fill one, two or three CTAs an SM, and three in two or three waves. Measured with NT = 1 (one to
// three CTAs an SM, 2 to 12 steps each, a step being a tile a warp): what a step takes on an SM
// with k CTAs when memory does not hold it up is 0.86, 0.66 and 0.72 us over k; memory gives 6.67
// TB/s whatever the layout; and 5.3, 6.2 and 8.7 us come on top, 4.0 where nothing is split. More
// CTAs than the call needs lose: 8 heads of 96K tokens take 25.0 us in 152 CTAs, 23.3 in 280 and
// 26.0 in 440. Sequences shorter than n (`ragged`; the lengths are on the device, and are taken to
// average 3/4 n, as if spread evenly between n / 2 and n) leave memory less to do, and a CTA of a
// later wave goes where a short one has ended, but the CTAs of one wave wait for the longest.
// Planned as if all were n, 32 x 8 heads of 16K to 32K tokens take 195 us against 163, of 0 to 32K
// 186 against 128, 5 x 12 heads of 36K to 72K 131 against 84. Lengths that are all far below n still
// go by the splits of n: 20000 tokens of n = 98304 take 21.9 us, and 9.6 where n is 20000. With NT = 2
// (1.20 and 1.07 us) each wave more costs 2.5 us (20 sequences of up to 9000 tokens, 16 heads over 2:
// 21.7 us in 720 CTAs, 19.5 in 240).
AttPlan attention_plan(int B, int Hq, int Hkv, int n, bool ragged) {
    AttPlan p;
    p.chunks = heads_plan(Hq / Hkv, &p.nt);
    const long long units = static_cast<long long>(B) * Hkv * p.chunks;
    const int steps = steps_of(n), resident = resident_ctas(p.nt);
    const int step_cost[2][3] = {{86, 66, 72}, {120, 107, 107}};
    const double memory = static_cast<double>(B) * Hkv * n * (2 * kCodeBytes + kParamBytes) /
                          66700.0 * (ragged ? 0.75 : 1.0);
    double best = -1.0;
    for (int k = 0; k < kPlans; ++k) {
        const long long most =
            k == 0 ? 1 : std::min<long long>(256, kSms * plan_ctas(k, resident) / units);
        if (most < 1 || (k > 0 && most < 2)) continue;
        const int each = static_cast<int>((steps + most - 1) / most);
        const int used = (steps + each - 1) / each;
        const long long busy = (units * used + kSms - 1) / kSms;         // CTAs of the fullest SM
        const int at_once = static_cast<int>(std::min<long long>(busy, resident));
        double steps_there = static_cast<double>((busy + at_once - 1) / at_once * at_once) * each;
        if (ragged && busy > resident) steps_there = 0.75 * steps_there + 0.25 * resident * each;
        const bool clustered = used > 1 && used <= kClusterSplits && busy <= resident;
        const double split_fixed[3] = {530.0, 620.0, 870.0};
        double fixed = used == 1 ? 400.0 : split_fixed[at_once - 1] - (clustered ? 40.0 : 0.0);
        if (p.nt == 2) fixed += 250.0 * static_cast<double>((busy - 1) / at_once);
        const double compute = steps_there * step_cost[p.nt - 1][at_once - 1];
        const double cost = fixed + std::max(memory, compute);
        if (best < 0.0 || cost < best) {
            best = cost;
            p.splits = used;
            p.tiles_per_split = each * kAttWarps;
            p.cluster = clustered;
        }
    }
    return p;
}

RowArgs row_args(const mp_kv4& c, const float* centre, int B, int Hkv, int m, int n_begin,
                 const int32_t* positions) {
    RowArgs a;
    a.centre = centre;
    a.positions = positions;
    a.k_codes = static_cast<uint8_t*>(c.k_codes);
    a.v_codes = static_cast<uint8_t*>(c.v_codes);
    a.params = static_cast<uint8_t*>(c.params);
    a.rows = static_cast<uint32_t>(B) * Hkv * m;
    a.Hkv = Hkv;
    a.m = m;
    a.n_begin = n_begin;
    a.ncap = c.n_capacity;
    a.status = device_status_ptr();
    return a;
}
typedef void (*RowFn)(const RowArgs);
RowFn pick_write(bool bf16, bool wide, int lanes) {
    using Bf16 = __nv_bfloat16;
    if (!bf16) return wide ? kv4_write_kernel<float, true, 8> : kv4_write_kernel<float, false, 8>;
    if (lanes == 8)
        return wide ? kv4_write_kernel<Bf16, true, 8> : kv4_write_kernel<Bf16, false, 8>;
    return wide ? kv4_write_kernel<Bf16, true, 4> : kv4_write_kernel<Bf16, false, 4>;
}
RowFn pick_read(bool bf16, bool wide) {
    using Bf16 = __nv_bfloat16;
    if (bf16) return wide ? kv4_read_kernel<Bf16, true> : kv4_read_kernel<Bf16, false>;
    return wide ? kv4_read_kernel<float, true> : kv4_read_kernel<float, false>;
}
bool wide_rows(const void* keys, const void* values) {
    return ((reinterpret_cast<uintptr_t>(keys) | reinterpret_cast<uintptr_t>(values)) & 31u) == 0u;
}
// As many CTAs as the GPU holds at once, or as there are blocks
unsigned row_ctas(RowArgs& a, int lanes, int per_sm) {
    const uint32_t per_cta = kRowThreads / lanes;
    a.blocks = (a.rows + per_cta - 1) / per_cta;
    return std::min<unsigned>(a.blocks, kSms * per_sm);
}

}  // namespace

cudaError_t launch_kv4_write(const void* keys, const void* values, bool bf16, const float* centre,
                             int B, int Hkv, int m, int n_begin, const int32_t* positions,
                             const mp_kv4& cache, cudaStream_t st) {
    RowArgs a = row_args(cache, centre, B, Hkv, m, n_begin, positions);
    a.keys = keys;
    a.values = values;
    const int lanes = write_lanes(bf16, a.rows);
    const unsigned ctas = row_ctas(a, lanes, bf16 && lanes == 8 ? 3 : 2);
    return launch_dependent(pick_write(bf16, wide_rows(keys, values), lanes), dim3(ctas),
                            dim3(kRowThreads), 0, st, a);
}

cudaError_t launch_kv4_read(const mp_kv4& cache, const float* centre, int B, int Hkv, int m,
                            int n_begin, const int32_t* positions, void* keys, void* values,
                            bool bf16, cudaStream_t st) {
    RowArgs a = row_args(cache, centre, B, Hkv, m, n_begin, positions);
    a.keys = keys;
    a.values = values;
    const unsigned ctas = row_ctas(a, kReadLanes, 4);
    return launch_dependent(pick_read(bf16, wide_rows(keys, values)), dim3(ctas),
                            dim3(kRowThreads), 0, st, a);
}

size_t kv4_attention_scratch_bytes(int B, int Hq, int Hkv, int n) {
    // the most splits that a plan of up to n tokens can have: the plans themselves have more for some
    // n than for larger ones (4 x 8 heads: a cluster at 16384 tokens, 9 splits in memory at 16128)
    const long long splits = most_splits(B, Hq, Hkv, n);
    return splits < 2 ? 0 : static_cast<size_t>(B) * Hq * splits * kPart * sizeof(float);
}

bool kv4_attention_uses_scratch(int B, int Hq, int Hkv, int n) {
    // in either layout: who asks does not say whether lengths will differ
    for (bool ragged : {false, true}) {
        const AttPlan p = attention_plan(B, Hq, Hkv, n, ragged);
        if (p.splits > 1 && !p.cluster) return true;
    }
    return false;
}

cudaError_t launch_kv4_attention(const void* q, bool q_bf16, const mp_kv4& cache, int B, int Hq,
                                 int Hkv, int n, const int32_t* lengths, float scale, float* out,
                                 void* workspace, cudaStream_t st) {
    const AttPlan p = attention_plan(B, Hq, Hkv, n, lengths != nullptr);
    A4Args a;
    a.q = q;
    a.k_codes = static_cast<const uint8_t*>(cache.k_codes);
    a.v_codes = static_cast<const uint8_t*>(cache.v_codes);
    a.params = static_cast<const uint8_t*>(cache.params);
    a.lengths = lengths;
    a.part = static_cast<float*>(workspace);
    a.out = out;
    a.q_bf16 = q_bf16;
    a.q_wide = (reinterpret_cast<uintptr_t>(q) & 15u) == 0u;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = Hq / Hkv;
    a.n = n;
    a.ncap = cache.n_capacity;
    a.splits = p.splits;
    a.cluster = p.cluster;
    a.chunks = p.chunks;
    a.tiles_per_split = p.tiles_per_split;
    a.rows = static_cast<long long>(B) * Hq;
    a.status = device_status_ptr();
    a.scale = scale * 1.4426950408889634f;
    const long long ctas = static_cast<long long>(B) * Hkv * p.splits * p.chunks;
    if (ctas > 0x7fffffffll) return cudaErrorInvalidValue;
    const cudaError_t e = launch_dependent(
        p.nt == 1 ? kv4_attention_kernel<1> : kv4_attention_kernel<2>,
        dim3(static_cast<unsigned>(ctas)), dim3(kAttThreads), kAttSmem, st, a,
        p.cluster ? p.splits : 1);
    if (e != cudaSuccess || p.splits == 1 || p.cluster) return e;
    return launch_dependent(kv4_merge_kernel, dim3(static_cast<unsigned>(B) * Hq),
                            dim3(32 * kMergeWarps), 0, st, a);
}

cudaError_t prepare_kv4() {
    cudaFuncAttributes fa;
    cudaError_t e;
    for (int i = 0; i < 4; ++i) {
        for (int lanes : {4, 8})
            if ((e = cudaFuncGetAttributes(&fa, pick_write(i & 1, i & 2, lanes))) != cudaSuccess)
                return e;
        if ((e = cudaFuncGetAttributes(&fa, pick_read(i & 1, i & 2))) != cudaSuccess) return e;
    }
    void (*att[2])(const A4Args) = {kv4_attention_kernel<1>, kv4_attention_kernel<2>};
    for (auto fn : att) {
        if ((e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      kAttSmem)) != cudaSuccess)
            return e;
        if ((e = cudaFuncSetAttribute(fn, cudaFuncAttributePreferredSharedMemoryCarveout,
                                      cudaSharedmemCarveoutMaxShared)) != cudaSuccess)
            return e;
    }
    return cudaFuncGetAttributes(&fa, kv4_merge_kernel);
}

}  // namespace mp
