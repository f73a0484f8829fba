// Incremental append of decode tokens: the codes of a short range of keys [n0, n1), written into
// the 32-key words they share with keys already encoded (whose bits are kept).
//
// The pages compute the centre and build the tables once, before decoding ("MagicPIG: LSH
// Sampling for Efficient LLM Generation", method details, data preprocessing and centering), and
// are silent on tokens generated afterwards; each new key is encoded here with the centre of the
// build, bit_{i,j} = [w_j . (k_i - mu) > 0], the same definition as the build.
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
// the kernel above (each over e in order), laid out for many heads with a key or a few each. A lane
// holds one hyperplane's 128 elements in registers, for all the heads its warp takes; keys come from
// shared memory, centred. Each (plane, word) of a head belongs to one lane, so that a word's bits are
// replaced by a plain read and write.
struct AtArgs {
    const void* keys;
    const void* W;
    const float* centre;
    const int32_t* positions;
    uint32_t* codes;
    int* status;
    int keys_bf16, w_bf16, BH, Hkv, m, ncap, C, cblk;
};
constexpr int kAtWarps = 4;                                    // 32 hyperplanes each
constexpr int kAtHeads = 8;                                    // heads a CTA takes one after another

__global__ void __launch_bounds__(32 * kAtWarps) encode_rows_at_kernel(const AtArgs a) {
    __shared__ __align__(16) float kbar[kAppendMaxKeys * kD];
    const int tid = threadIdx.x, lane = tid & 31;
    const int j = (blockIdx.x * kAtWarps + (tid >> 5)) * 32 + lane;
    float w[kD];
#pragma unroll
    for (int e = 0; e < kD; ++e)
        w[e] = j < a.C ? load_elem(a.W, a.w_bf16, static_cast<size_t>(e) * a.C + j) : 0.0f;
    const int bh1 = min(a.BH, static_cast<int>(blockIdx.y + 1) * kAtHeads);
    for (int bh = blockIdx.y * kAtHeads; bh < bh1; ++bh) {
        const int at = a.positions[bh / a.Hkv];
        const float mu = a.centre[static_cast<size_t>(bh) * kD + (tid & (kD - 1))];
        __syncthreads();                                       // the last head's keys are read
        for (int idx = tid; idx < a.m * kD; idx += 32 * kAtWarps)
            kbar[idx] = load_elem(a.keys, a.keys_bf16, static_cast<size_t>(bh) * a.m * kD + idx) - mu;
        __syncthreads();
        // keys [i0, i1) of the m lie inside the capacity
        const int i0 = at < 0 ? static_cast<int>(min(static_cast<long long>(a.m),
                                                     -static_cast<long long>(at))) : 0;
        const int i1 = static_cast<int>(min(static_cast<long long>(a.m),
                                            static_cast<long long>(a.ncap) - at));
        uint32_t range = 0u, bits = 0u;
        for (int i = i0; i < i1; ++i) {
            float sum = 0.0f;
            const float4* k4 = reinterpret_cast<const float4*>(kbar + i * kD);
#pragma unroll
            for (int e = 0; e < kD / 4; ++e) {
                const float4 k = k4[e];
                sum = fmaf(w[4 * e], k.x, sum);
                sum = fmaf(w[4 * e + 1], k.y, sum);
                sum = fmaf(w[4 * e + 2], k.z, sum);
                sum = fmaf(w[4 * e + 3], k.w, sum);
            }
            const int pos = at + i;
            range |= 1u << (pos & 31);
            if (sum > 0.0f) bits |= 1u << (pos & 31);
            if ((pos & 31) == 31 || i + 1 == i1) {             // the word's last key of the range
                const int blk = pos / kKeysPerBlock;
                if (j < a.C && mp_check(a.status, blk, a.cblk, kSiteEncodeCodes)) {
                    uint32_t* dst = a.codes +
                                    ((static_cast<size_t>(bh) * a.cblk + blk) * a.C + j) *
                                        kWordsPerBlock + pos % kKeysPerBlock / 32;
                    *dst = (*dst & ~range) | bits;
                }
                range = bits = 0u;
            }
        }
    }
}

}  // namespace

cudaError_t launch_encode_append(const void* keys, bool keys_bf16, const float* centre,
                                 const void* W, bool w_bf16, int B, int Hkv, int head_rows, int row0,
                                 int ncap, int n0, int n1, int K, int L, uint32_t* codes,
                                 cudaStream_t st) {
    const int C = K * L;
    if (C == 0 || n1 <= n0) return cudaSuccess;
    if (n1 - n0 > kAppendMaxKeys) return cudaErrorInvalidValue;
    const int cblk = (ncap + kKeysPerBlock - 1) / kKeysPerBlock;
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
    a.keys_bf16 = keys_bf16;
    a.w_bf16 = w_bf16;
    a.BH = B * Hkv;
    a.Hkv = Hkv;
    a.m = m;
    a.ncap = ncap;
    a.C = C;
    a.cblk = (ncap + kKeysPerBlock - 1) / kKeysPerBlock;
    const unsigned groups = (a.BH + kAtHeads - 1) / kAtHeads;
    if (groups > 65535u) return cudaErrorInvalidValue;
    encode_rows_at_kernel<<<dim3((C + 32 * kAtWarps - 1) / (32 * kAtWarps), groups), 32 * kAtWarps,
                            0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t prepare_append() {
    cudaFuncAttributes fa;
    const cudaError_t e = cudaFuncGetAttributes(&fa, encode_rows_at_kernel);
    if (e != cudaSuccess) return e;
    return cudaFuncGetAttributes(&fa, encode_append_kernel);
}

}  // namespace mp
