// A K/V cache held in 4 bits: rows written from bf16 or fp32 keys and values, rows read back, and
// exact attention of single query tokens over the cache. The pages keep K and V at the model's
// precision and have no counterpart; the layout is the one magicpig.h describes.
//
// A group of 64 dims x_e (two per row) is held by z, the largest bf16 <= min x, s, the smallest
// bf16 with z + 15 s >= max x, and codes c_e = rint((x_e - z) / s), so |x_e - (z + s c_e)| <= s / 2.
// 15 s is exact in float32 (8 + 4 bits), so s is RU_bf16(RU((max - z)) / 15): if 15 s reaches the
// rounded-up difference it reaches the exact one, and conversely.
#include <algorithm>

#include "mp_internal.cuh"

namespace mp {
namespace {

constexpr int kGroup = MP_KV4_GROUP;
constexpr int kGroups = kD / kGroup;
constexpr int kCodeBytes = MP_KV4_CODE_BYTES;

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

// The high half of a float is a bf16: rounding down drops the low half, one step further from
// zero for a negative value whose low half is not 0; rounding up mirrors it.
__device__ __forceinline__ uint32_t bf16_below(float x) {
    const uint32_t u = __float_as_uint(x), t = u >> 16;
    return t + ((u >> 31) != 0u && (u & 0xffffu) != 0u ? 1u : 0u);
}
__device__ __forceinline__ uint32_t bf16_above_positive(float x) {
    const uint32_t u = __float_as_uint(x);
    return (u >> 16) + ((u & 0xffffu) != 0u ? 1u : 0u);
}

// s (low half) and z (high half) of a group from its minimum and maximum; NaN in both for a group
// that has no finite pair (min_nan and max_nan pass a NaN on).
__device__ __forceinline__ uint32_t group_params(float lo, float hi) {
    const uint32_t z = bf16_below(lo);
    const float d = __fsub_ru(hi, __uint_as_float(z << 16));
    const uint32_t s = bf16_above_positive(__fdiv_ru(d, 15.0f));
    const bool finite = (z & 0x7f80u) != 0x7f80u && (s & 0x7f80u) != 0x7f80u && d == d;
    return finite ? (s | (z << 16)) : 0x7fc07fc0u;
}

// rint((x - z) / s) from the definition in 64 bits: what decides next to a border.
__device__ __noinline__ uint32_t code_exact(float x, float z, float s) {
    const double v = (static_cast<double>(x) - static_cast<double>(z)) / static_cast<double>(s);
    return static_cast<uint32_t>(static_cast<int>(rint(v)));
}

struct RowArgs {
    const void* keys;                            // of the rows to write; outputs of a read
    const void* values;
    const float* centre;
    const int32_t* positions;
    uint8_t* k_codes;
    uint8_t* v_codes;
    uint8_t* params;
    long long rows;                              // B * Hkv * m
    int Hkv, m, n_begin, ncap;
};

// The cache row (over all heads) of row r of the call, or -1 where it falls outside the cache.
__device__ __forceinline__ long long cache_row(const RowArgs& a, long long r) {
    const long long bh = r / a.m;
    const int i = static_cast<int>(r - bh * a.m);
    const long long pos =
        static_cast<long long>(a.positions ? __ldg(a.positions + bh / a.Hkv) : a.n_begin) + i;
    return pos >= 0 && pos < a.ncap ? bh * a.ncap + pos : -1;
}

constexpr int kRowThreads = 256;

// A half-warp per row, 8 dims (one word of codes) a lane; a group is 8 lanes.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) kv4_write_kernel(const RowArgs a) {
    const int hl = threadIdx.x & 15;
    const long long r = (static_cast<long long>(blockIdx.x) * kRowThreads + threadIdx.x) >> 4;
    const bool live = r < a.rows;
    const long long row = live ? cache_row(a, r) : -1;
    for (int value = 0; value < 2; ++value) {
        float x[8];
        const T* src = static_cast<const T*>(value ? a.values : a.keys);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = row >= 0 ? to_float(src[r * kD + 8 * hl + i]) : 0.0f;
        if (!value && a.centre && live) {
            const float* mu = a.centre + (r / a.m) * kD + 8 * hl;
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __fsub_rn(x[i], mu[i]);
        }
        float lo = x[0], hi = x[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) {
            lo = min_nan(lo, x[i]);
            hi = max_nan(hi, x[i]);
        }
#pragma unroll
        for (int o = 4; o; o >>= 1) {
            lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
            hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        }
        const uint32_t pr = group_params(lo, hi);
        const float s = __uint_as_float(pr << 16), z = __uint_as_float(pr & 0xffff0000u);
        uint32_t w = 0u;
        if (s > 0.0f) {
#pragma unroll
            for (int i = 0; i < 8; ++i) w |= code_exact(x[i], z, s) << (4 * i);
        }
        if (row >= 0) {
            uint8_t* codes = value ? a.v_codes : a.k_codes;
            *reinterpret_cast<uint32_t*>(codes + row * kCodeBytes + 4 * hl) = w;
            if ((hl & 7) == 0)
                *reinterpret_cast<uint32_t*>(a.params + row * 16 + 8 * value + 4 * (hl >> 3)) = pr;
        }
    }
}

template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads) kv4_read_kernel(const RowArgs a) {
    const int hl = threadIdx.x & 15;
    const long long r = (static_cast<long long>(blockIdx.x) * kRowThreads + threadIdx.x) >> 4;
    if (r >= a.rows) return;
    const long long row = cache_row(a, r);
    for (int value = 0; value < 2; ++value) {
        T* dst = static_cast<T*>(const_cast<void*>(value ? a.values : a.keys)) + r * kD + 8 * hl;
        uint32_t w = 0u, pr = 0u;
        if (row >= 0) {
            w = *reinterpret_cast<const uint32_t*>((value ? a.v_codes : a.k_codes) +
                                                   row * kCodeBytes + 4 * hl);
            pr = *reinterpret_cast<const uint32_t*>(a.params + row * 16 + 8 * value + 4 * (hl >> 3));
        }
        const float s = __uint_as_float(pr << 16), z = __uint_as_float(pr & 0xffff0000u);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float x = fmaf(s, static_cast<float>((w >> (4 * i)) & 15u), z);
            if (!value && a.centre && row >= 0)
                x = __fadd_rn(x, a.centre[(r / a.m) * kD + 8 * hl + i]);
            dst[i] = from_float<T>(x);
        }
    }
}

// ------------------------------------------------------------------------------------------------
// Exact attention of one query token: one CTA per (split of the tokens, query row), a warp per
// token, four dims a lane; partial softmaxes merged by a second kernel.
// ------------------------------------------------------------------------------------------------
struct A4Args {
    const void* q;
    const uint8_t* k_codes;
    const uint8_t* v_codes;
    const uint8_t* params;
    const int32_t* lengths;
    float* part;                                 // [row][split][kPart]: o, m, l
    float* out;
    int q_bf16, Hq, Hkv, n, ncap, splits, per_split;
    float scale;
};
constexpr int kPart = kD + 4;
constexpr int kAttWarps = 4;

__device__ __forceinline__ int length_of(const A4Args& a, int b) {
    return a.lengths ? max(0, min(a.n, __ldg(a.lengths + b))) : a.n;
}

__global__ void __launch_bounds__(32 * kAttWarps) kv4_attention_kernel(const A4Args a) {
    __shared__ float sm[kAttWarps][kPart];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long row = blockIdx.x / a.splits;
    const int split = static_cast<int>(blockIdx.x % a.splits);
    const int b = static_cast<int>(row / a.Hq), h = static_cast<int>(row % a.Hq);
    const long long bh = static_cast<long long>(b) * a.Hkv + h / (a.Hq / a.Hkv);
    const int k0 = split * a.per_split, k1 = min(length_of(a, b), k0 + a.per_split);
    float q[4], o[4] = {0.0f, 0.0f, 0.0f, 0.0f}, m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = load_elem(a.q, a.q_bf16, row * kD + 4 * lane + i) * a.scale;
    for (int k = k0 + warp; k < k1; k += kAttWarps) {
        const long long at = bh * a.ncap + k;
        const uint32_t kw = *reinterpret_cast<const uint16_t*>(a.k_codes + at * kCodeBytes + 2 * lane);
        const uint32_t vw = *reinterpret_cast<const uint16_t*>(a.v_codes + at * kCodeBytes + 2 * lane);
        const uint32_t kp = *reinterpret_cast<const uint32_t*>(a.params + at * 16 + 4 * (lane >> 4));
        const uint32_t vp = *reinterpret_cast<const uint32_t*>(a.params + at * 16 + 8 + 4 * (lane >> 4));
        const float ks = __uint_as_float(kp << 16), kz = __uint_as_float(kp & 0xffff0000u);
        const float vs = __uint_as_float(vp << 16), vz = __uint_as_float(vp & 0xffff0000u);
        float d = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            d = fmaf(q[i], fmaf(ks, static_cast<float>((kw >> (4 * i)) & 15u), kz), d);
#pragma unroll
        for (int s = 16; s; s >>= 1) d += __shfl_xor_sync(0xffffffffu, d, s);
        const float mn = fmaxf(m, d);
        const float corr = expf(m - mn), w = expf(d - mn);
        l = fmaf(l, corr, w);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[i] = fmaf(w, fmaf(vs, static_cast<float>((vw >> (4 * i)) & 15u), vz), o[i] * corr);
        m = mn;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) sm[warp][4 * lane + i] = o[i];
    if (lane == 0) {
        sm[warp][kD] = m;
        sm[warp][kD + 1] = l;
    }
    __syncthreads();
    const int e = threadIdx.x;
    float M = -INFINITY, L = 0.0f, O = 0.0f;
    for (int w = 0; w < kAttWarps; ++w) M = max_nan(M, sm[w][kD]);
    for (int w = 0; w < kAttWarps; ++w) {
        const float c = sm[w][kD] == -INFINITY ? 0.0f : expf(sm[w][kD] - M);
        if (sm[w][kD] == -INFINITY && sm[w][kD + 1] == 0.0f) continue;
        L = fmaf(c, sm[w][kD + 1], L);
        O = fmaf(c, sm[w][e], O);
    }
    float* p = a.part + (row * a.splits + split) * kPart;
    p[e] = O;
    if (e == 0) {
        p[kD] = M;
        p[kD + 1] = L;
    }
}

__global__ void __launch_bounds__(kD) kv4_merge_kernel(const float* part, int splits, float* out) {
    const long long row = blockIdx.x;
    const int e = threadIdx.x;
    const float* p = part + row * splits * kPart;
    float M = -INFINITY, L = 0.0f, O = 0.0f;
    for (int s = 0; s < splits; ++s) M = max_nan(M, p[s * kPart + kD]);
    for (int s = 0; s < splits; ++s) {
        const float ms = p[s * kPart + kD], ls = p[s * kPart + kD + 1];
        if (ms == -INFINITY && ls == 0.0f) continue;
        const float c = expf(ms - M);
        L = fmaf(c, ls, L);
        O = fmaf(c, p[s * kPart + e], O);
    }
    out[row * kD + e] = L == 0.0f ? 0.0f : O / L;
}

int attention_splits(int n) { return std::max(1, std::min(64, (n + 255) / 256)); }

RowArgs row_args(const mp_kv4& c, const float* centre, int B, int Hkv, int m, int n_begin,
                 const int32_t* positions) {
    RowArgs a;
    a.centre = centre;
    a.positions = positions;
    a.k_codes = static_cast<uint8_t*>(c.k_codes);
    a.v_codes = static_cast<uint8_t*>(c.v_codes);
    a.params = static_cast<uint8_t*>(c.params);
    a.rows = static_cast<long long>(B) * Hkv * m;
    a.Hkv = Hkv;
    a.m = m;
    a.n_begin = n_begin;
    a.ncap = c.n_capacity;
    return a;
}
unsigned row_ctas(long long rows) {
    constexpr int kPerCta = kRowThreads / 16;
    return static_cast<unsigned>((rows + kPerCta - 1) / kPerCta);
}

}  // namespace

cudaError_t launch_kv4_write(const void* keys, const void* values, bool bf16, const float* centre,
                             int B, int Hkv, int m, int n_begin, const int32_t* positions,
                             const mp_kv4& cache, cudaStream_t st) {
    RowArgs a = row_args(cache, centre, B, Hkv, m, n_begin, positions);
    a.keys = keys;
    a.values = values;
    if (bf16) kv4_write_kernel<__nv_bfloat16><<<row_ctas(a.rows), kRowThreads, 0, st>>>(a);
    else kv4_write_kernel<float><<<row_ctas(a.rows), kRowThreads, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_kv4_read(const mp_kv4& cache, const float* centre, int B, int Hkv, int m,
                            int n_begin, const int32_t* positions, void* keys, void* values,
                            bool bf16, cudaStream_t st) {
    RowArgs a = row_args(cache, centre, B, Hkv, m, n_begin, positions);
    a.keys = keys;
    a.values = values;
    if (bf16) kv4_read_kernel<__nv_bfloat16><<<row_ctas(a.rows), kRowThreads, 0, st>>>(a);
    else kv4_read_kernel<float><<<row_ctas(a.rows), kRowThreads, 0, st>>>(a);
    return cudaGetLastError();
}

size_t kv4_attention_scratch_bytes(int B, int Hq, int Hkv, int n) {
    (void)Hkv;
    return static_cast<size_t>(B) * Hq * attention_splits(n) * kPart * sizeof(float);
}

cudaError_t launch_kv4_attention(const void* q, bool q_bf16, const mp_kv4& cache, int B, int Hq,
                                 int Hkv, int n, const int32_t* lengths, float scale, float* out,
                                 void* workspace, cudaStream_t st) {
    A4Args a;
    a.q = q;
    a.k_codes = static_cast<const uint8_t*>(cache.k_codes);
    a.v_codes = static_cast<const uint8_t*>(cache.v_codes);
    a.params = static_cast<const uint8_t*>(cache.params);
    a.lengths = lengths;
    a.part = static_cast<float*>(workspace);
    a.out = out;
    a.q_bf16 = q_bf16;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.n = n;
    a.ncap = cache.n_capacity;
    a.splits = attention_splits(n);
    a.per_split = (n + a.splits - 1) / a.splits;
    a.scale = scale;
    const unsigned rows = static_cast<unsigned>(B) * Hq;
    kv4_attention_kernel<<<rows * a.splits, 32 * kAttWarps, 0, st>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    kv4_merge_kernel<<<rows, kD, 0, st>>>(a.part, a.splits, out);
    return cudaGetLastError();
}

cudaError_t prepare_kv4() {
    cudaFuncAttributes fa;
    cudaError_t e;
    if ((e = cudaFuncGetAttributes(&fa, kv4_write_kernel<__nv_bfloat16>)) != cudaSuccess) return e;
    if ((e = cudaFuncGetAttributes(&fa, kv4_write_kernel<float>)) != cudaSuccess) return e;
    if ((e = cudaFuncGetAttributes(&fa, kv4_read_kernel<__nv_bfloat16>)) != cudaSuccess) return e;
    if ((e = cudaFuncGetAttributes(&fa, kv4_read_kernel<float>)) != cudaSuccess) return e;
    if ((e = cudaFuncGetAttributes(&fa, kv4_attention_kernel)) != cudaSuccess) return e;
    return cudaFuncGetAttributes(&fa, kv4_merge_kernel);
}

}  // namespace mp
