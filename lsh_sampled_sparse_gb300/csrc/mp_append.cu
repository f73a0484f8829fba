// Incremental append of decode tokens: the codes of a short range of keys [n0, n1), written into
// the 32-key words they share with keys already encoded (whose bits are kept).
//
// The pages compute the centre and build the tables once, before decoding ("MagicPIG: LSH
// Sampling for Efficient LLM Generation", method details, data preprocessing and centering), and
// are silent on tokens generated afterwards; each new key is encoded here with the centre of the
// build, bit_{i,j} = [w_j . (k_i - mu) > 0], the same definition as the build.
#include <algorithm>

#include "mp_internal.cuh"

namespace mp {
namespace {

constexpr int kAppendWarps = 4;                                // >= the words a range touches
static_assert(kAppendWarps >= (kAppendMaxKeys + 31) / 32 + 1, "a warp per touched word");
constexpr int kAppendThreads = kAppendWarps * 32;
constexpr int kStageBatch = 16;                                // loads a thread issues at once
constexpr int kAppendPlanes = 32;                              // hyperplanes per CTA (one a lane)
constexpr int kAppendKeysAtOnce = 4;                           // independent sums a lane carries

// One CTA per (chunk of 32 hyperplanes, head). The chunk of W and the range's centred keys are
// staged in shared memory, kStageBatch loads in flight per thread; warp w then takes the range's
// w-th 32-key word, lane j hyperplane j0 + j, and rewrites that word's bits of the range only (each
// (plane, word) has one owner, so a plain read-modify-write). Each sum runs over e in order,
// fmaf(W[e][j], k[e] - mu[e], acc): the arithmetic of the CUDA-core block encoder.
__global__ void __launch_bounds__(kAppendThreads)
    encode_append_kernel(const void* keys, int keys_bf16, const float* centre, const void* W,
                         int w_bf16, int head_rows, int row0, int n0, int n1, int C, int cblk,
                         uint32_t* codes, int* status) {
    extern __shared__ __align__(16) float sm[];
    float* Ws = sm;                                   // [kD][kAppendPlanes]
    float* kbar = sm + kD * kAppendPlanes;            // [n1 - n0][kD]
    const int bh = blockIdx.y, j0 = blockIdx.x * kAppendPlanes, tid = threadIdx.x;
    const int lane = tid & 31, warp = tid >> 5;
    const int m = n1 - n0;
    for (int base = 0; base < kD * kAppendPlanes; base += kAppendThreads * kStageBatch) {
        float v[kStageBatch];
#pragma unroll
        for (int u = 0; u < kStageBatch; ++u) {
            const int idx = base + u * kAppendThreads + tid;
            const int e = idx / kAppendPlanes, j = j0 + idx % kAppendPlanes;
            v[u] = idx < kD * kAppendPlanes && j < C
                       ? load_elem(W, w_bf16, static_cast<size_t>(e) * C + j) : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < kStageBatch; ++u) {
            const int idx = base + u * kAppendThreads + tid;
            if (idx < kD * kAppendPlanes) Ws[idx] = v[u];
        }
    }
    for (int base = 0; base < m * kD; base += kAppendThreads * kStageBatch) {
        float v[kStageBatch];
#pragma unroll
        for (int u = 0; u < kStageBatch; ++u) {
            const int idx = base + u * kAppendThreads + tid;
            v[u] = idx < m * kD && mp_check(status, row0 + idx / kD, head_rows, kSiteEncodeRow)
                       ? load_elem(keys, keys_bf16,
                                   (static_cast<size_t>(bh) * head_rows + row0 + idx / kD) * kD +
                                       idx % kD) -
                             centre[static_cast<size_t>(bh) * kD + idx % kD]
                       : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < kStageBatch; ++u) {
            const int idx = base + u * kAppendThreads + tid;
            if (idx < m * kD) kbar[idx] = v[u];
        }
    }
    __syncthreads();
    const int w = n0 / 32 + warp;                     // absolute 32-key word
    const int k0 = max(n0, w * 32), k1 = min(n1, w * 32 + 32);
    const int j = j0 + lane;
    if (k0 >= k1 || j >= C) return;
    uint32_t bits = 0u;
    for (int r0 = k0; r0 < k1; r0 += kAppendKeysAtOnce) {
        const float* kr[kAppendKeysAtOnce];
        float P[kAppendKeysAtOnce];
#pragma unroll
        for (int u = 0; u < kAppendKeysAtOnce; ++u) {
            kr[u] = kbar + static_cast<size_t>(min(r0 + u, k1 - 1) - n0) * kD;   // past k1: a repeat
            P[u] = 0.0f;
        }
#pragma unroll 4
        for (int e = 0; e < kD; ++e) {
            const float wv = Ws[e * kAppendPlanes + lane];
#pragma unroll
            for (int u = 0; u < kAppendKeysAtOnce; ++u) P[u] = fmaf(wv, kr[u][e], P[u]);
        }
#pragma unroll
        for (int u = 0; u < kAppendKeysAtOnce; ++u)
            if (r0 + u < k1 && P[u] > 0.0f) bits |= 1u << ((r0 + u) & 31);
    }
    const uint32_t range = bits_below(k1 - w * 32) & ~bits_below(k0 - w * 32);
    uint32_t* dst = codes + ((static_cast<size_t>(bh) * cblk + w / kWordsPerBlock) * C + j) *
                                kWordsPerBlock + w % kWordsPerBlock;
    if (mp_check(status, w / kWordsPerBlock, cblk, kSiteEncodeCodes))
        *dst = (*dst & ~range) | bits;
}

// The codes of a few tokens of every sequence at places of its own: the definition and the sums of
// the kernel above (each over e in order), laid out for many heads with a key or a few each. A CTA takes
// 128 hyperplanes and sixteen rows at a time of whole heads. A lane sums four hyperplanes by four rows, from
// shared memory (a lane is given 1.5 bytes a sum that way; with one hyperplane a lane and eight rows, 4.5
// bytes, the sums took three times as long); the signs meet in shared memory, and the thread a hyperplane
// belongs to sends the bits to their words. What is left of a row or a few is the layout's: a key's K L bits lie
// in as many words 128 bytes apart (32 sequences x 8 heads at (10, 150), a key each: 384000 words, for which DRAM
// is read 979000 sectors of 32 bytes, 31 MB; 13.6 to 14.3 us). Tens of rows are bound by the sums, in float32 on
// CUDA cores: 64 rows of each of those heads 207 us, 30 TFLOP/s.
struct AtArgs {
    const void* keys;
    const void* W;
    const float* centre;
    const int32_t* positions;
    uint32_t* codes;
    int* status;
    int BH, Hkv, m, ncap, C, cblk, heads, wide;   // wide: rows of W aligned for four elements
};
constexpr int kAtThreads = kD;                                 // and hyperplanes of a CTA
constexpr int kAtSums = 4;                                     // rows a warp sums, and hyperplanes a lane
constexpr int kAtRows = kAtThreads / 32 * kAtSums;             // rows of a pass

__device__ __forceinline__ void four_of(const __nv_bfloat16* p, float (&w)[4]) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = __uint_as_float(v.x << 16);
    w[1] = __uint_as_float(v.x & 0xffff0000u);
    w[2] = __uint_as_float(v.y << 16);
    w[3] = __uint_as_float(v.y & 0xffff0000u);
}
__device__ __forceinline__ void four_of(const float* p, float (&w)[4]) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
}

template <typename TW>
struct FourOf {
    using type = uint2;
};
template <>
struct FourOf<float> {
    using type = uint4;
};

// T, TW: the types of the keys and of W (at run time each load would wait behind a branch of its own)
template <typename T, typename TW>
__global__ void __launch_bounds__(kAtThreads) encode_rows_at_kernel(const AtArgs a) {
    extern __shared__ __align__(16) uint8_t at_smem[];
    TW* Ws = reinterpret_cast<TW*>(at_smem);                   // [kD][kAtThreads]
    __shared__ __align__(16) float kbar[kAtRows][kD];
    __shared__ __align__(4) uint8_t side[kAtRows][kAtThreads]; // 1: the hyperplane's positive side
    __shared__ int bit_of[kAtRows];                            // a row's bit of its word
    __shared__ long long word_of[kAtRows + 1];                 // the word, of hyperplane 0; -1: nowhere
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int j = blockIdx.x * kAtThreads + tid, bh0 = blockIdx.y * a.heads;
    const int all = (min(a.BH, bh0 + a.heads) - bh0) * a.m;
    const bool live = j < a.C;
    uint32_t* mine = a.codes + static_cast<size_t>(j) * kWordsPerBlock;
    wait_for_predecessor();
    allow_dependents();
    // W's piece: four hyperplanes a lane where its rows are aligned for that
    if (a.wide) {
        using Four = typename FourOf<TW>::type;
        constexpr int kAhead = 256 / sizeof(Four);             // all loads first, then the stores
        const int j4 = min(static_cast<int>(blockIdx.x) * kAtThreads + 4 * lane, a.C - 4);
#pragma unroll 1
        for (int e0 = warp; e0 < kD; e0 += kAhead * (kAtThreads / 32)) {
            Four w[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                w[i] = *reinterpret_cast<const Four*>(
                    static_cast<const TW*>(a.W) +
                    static_cast<size_t>(e0 + i * (kAtThreads / 32)) * a.C + j4);
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                *reinterpret_cast<Four*>(Ws + (e0 + i * (kAtThreads / 32)) * kAtThreads + 4 * lane) = w[i];
        }
    } else {
        constexpr int kAhead = 32;
#pragma unroll 1
        for (int e0 = 0; e0 < kD; e0 += kAhead) {
            TW w[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                w[i] = static_cast<const TW*>(a.W)[static_cast<size_t>(e0 + i) * a.C + min(j, a.C - 1)];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) Ws[(e0 + i) * kAtThreads + tid] = w[i];
        }
    }
    for (int r0 = 0; r0 < all; r0 += kAtRows) {
        const int rows = min(kAtRows, all - r0);
        T k[kAtRows];
        float mu[kAtRows];
#pragma unroll
        for (int r = 0; r < kAtRows; ++r) {
            const int at = r0 + min(r, rows - 1);
            if (!mp_check(a.status, static_cast<long long>(bh0) * a.m + at, static_cast<long long>(a.BH) * a.m,
                          kSiteEncodeRow))
                continue;
            k[r] = static_cast<const T*>(a.keys)[(static_cast<size_t>(bh0) * a.m + at) * kD + tid];
            mu[r] = a.centre[static_cast<size_t>(bh0 + at / a.m) * kD + tid];
        }
        __syncthreads();                                       // the last pass's rows are read
        if (tid <= kAtRows) {
            const int r = r0 + min(tid, rows - 1), bh = bh0 + r / a.m;
            const long long p = static_cast<long long>(a.positions[bh / a.Hkv]) + r % a.m;
            const int blk = static_cast<int>(p >> 10);
            const bool there = tid < rows && p >= 0 && p < a.ncap;
            word_of[tid] = there ? (static_cast<long long>(bh) * a.cblk + blk) * a.C * kWordsPerBlock +
                                       (static_cast<int>(p) & (kKeysPerBlock - 1)) / 32
                                 : -1;
            if (tid < kAtRows) bit_of[tid] = static_cast<int>(p & 31);
        }
#pragma unroll
        for (int r = 0; r < kAtRows; ++r) kbar[r][tid] = to_float(k[r]) - mu[r];
        __syncthreads();
        if (kAtSums * warp < rows) {
            float sum[kAtSums][4] = {};
            const float* k = kbar[kAtSums * warp];
#pragma unroll 4
            for (int e = 0; e < kD; e += 4) {
                float4 x[kAtSums];
                float w[4][4];
#pragma unroll
                for (int u = 0; u < kAtSums; ++u) x[u] = *reinterpret_cast<const float4*>(k + u * kD + e);
#pragma unroll
                for (int i = 0; i < 4; ++i) four_of(Ws + (e + i) * kAtThreads + 4 * lane, w[i]);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int u = 0; u < kAtSums; ++u) {
                        const float xi = i == 0 ? x[u].x : (i == 1 ? x[u].y : (i == 2 ? x[u].z : x[u].w));
#pragma unroll
                        for (int c = 0; c < 4; ++c) sum[u][c] = fmaf(w[i][c], xi, sum[u][c]);
                    }
            }
#pragma unroll
            for (int u = 0; u < kAtSums; ++u)
                *reinterpret_cast<uint32_t*>(&side[kAtSums * warp + u][4 * lane]) =
                    (sum[u][0] > 0.0f ? 1u : 0u) | (sum[u][1] > 0.0f ? 0x100u : 0u) |
                    (sum[u][2] > 0.0f ? 0x10000u : 0u) | (sum[u][3] > 0.0f ? 0x1000000u : 0u);
        }
        __syncthreads();
        if (!live) continue;
        // rows of one word follow each other: their bits go out after the last, those to set and those
        // to clear, by operations that L2 carries out and nobody waits for (words loaded, changed and
        // stored: 49 MB read instead of 31, 23 to 31 us instead of 14)
        uint32_t set = 0u, clear = 0u;
#pragma unroll
        for (int u = 0; u < kAtRows; ++u) {
            const long long w = word_of[u];
            if (w < 0) continue;
            const uint32_t bit = 1u << bit_of[u];
            if (side[u][tid]) set |= bit;
            else clear |= bit;
            if (w != word_of[u + 1]) {
                if (!mp_check(a.status, w + static_cast<long long>(j) * kWordsPerBlock,
                              static_cast<long long>(a.BH) * a.cblk * a.C * kWordsPerBlock, kSiteEncodeCodes))
                    set = clear = 0u;
                if (set) atomicOr(mine + w, set);
                if (clear) atomicAnd(mine + w, ~clear);
                set = clear = 0u;
            }
        }
    }
}

void (*pick_at(bool keys_bf16, bool w_bf16))(const AtArgs) {
    using Bf16 = __nv_bfloat16;
    if (keys_bf16) return w_bf16 ? encode_rows_at_kernel<Bf16, Bf16> : encode_rows_at_kernel<Bf16, float>;
    return w_bf16 ? encode_rows_at_kernel<float, Bf16> : encode_rows_at_kernel<float, float>;
}

}  // namespace

cudaError_t launch_encode_append(const void* keys, bool keys_bf16, const float* centre,
                                 const void* W, bool w_bf16, int B, int Hkv, int head_rows, int row0,
                                 int ncap, int n0, int n1, int K, int L, uint32_t* codes,
                                 cudaStream_t st) {
    const int C = K * L;
    if (C == 0 || n1 <= n0) return cudaSuccess;
    if (n1 - n0 > kAppendMaxKeys) return cudaErrorInvalidValue;
    const int cblk = key_blocks(ncap);
    const size_t smem = (static_cast<size_t>(kD) * kAppendPlanes +
                         static_cast<size_t>(n1 - n0) * kD) * sizeof(float);
    const dim3 grid((C + kAppendPlanes - 1) / kAppendPlanes, B * Hkv);
    encode_append_kernel<<<grid, kAppendThreads, smem, st>>>(
        keys, keys_bf16, centre, W, w_bf16, head_rows, row0, n0, n1, C, cblk, codes,
        device_status_ptr());
    return cudaGetLastError();
}

cudaError_t launch_encode_rows_at(const void* keys, bool keys_bf16, const float* centre,
                                  const void* W, bool w_bf16, int B, int Hkv, int m, int ncap,
                                  const int32_t* positions, int C, uint32_t* codes,
                                  cudaStream_t st) {
    AtArgs a;
    a.keys = keys;
    a.W = W;
    a.centre = centre;
    a.positions = positions;
    a.codes = codes;
    a.status = device_status_ptr();
    a.BH = B * Hkv;
    a.Hkv = Hkv;
    a.m = m;
    a.ncap = ncap;
    a.C = C;
    a.cblk = key_blocks(ncap);
    a.heads = std::max(1, kAtRows / m);
    a.wide = C % 4 == 0 && reinterpret_cast<uintptr_t>(W) % (w_bf16 ? 8 : 16) == 0;
    return launch_dependent(pick_at(keys_bf16, w_bf16),
                            dim3((C + kAtThreads - 1) / kAtThreads, (a.BH + a.heads - 1) / a.heads),
                            dim3(kAtThreads), kD * kAtThreads * (w_bf16 ? 2 : 4), st, a);
}

cudaError_t prepare_append() {
    cudaFuncAttributes fa;
    for (int i = 0; i < 4; ++i) {
        const cudaError_t e = cudaFuncSetAttribute(pick_at(i & 1, i & 2),
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   kD * kAtThreads * (i & 2 ? 2 : 4));
        if (e != cudaSuccess) return e;
    }
    return cudaFuncGetAttributes(&fa, encode_append_kernel);
}

}  // namespace mp
