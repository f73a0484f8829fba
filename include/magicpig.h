/*
 * magicpig.h -- C ABI of libmagicpig, LSH-sampled decode attention on one GB300 (sm_103a).
 *
 * The method is MagicPIG's ("MagicPIG: LSH Sampling for Efficient LLM Generation", method
 * details; "MagicPIG: don't pick the tallest", section 5): keys are centred and SimHash-encoded
 * into L tables of K bits; a decode query keeps the keys whose code equals its own in at least
 * two tables, weights each kept key by its closed-form inclusion probability u, and merges that
 * self-normalised importance-sampled attention with exact attention over the sink and local
 * tokens. Everything stays in device memory; every step runs in this library's CUDA kernels.
 *
 * Conventions for every entry point below:
 *   - Pointers to tensors are DEVICE pointers owned by the caller. Nothing here allocates device
 *     memory; scratch comes from a caller-provided workspace whose size a *_workspace_bytes
 *     function returns. Workspace pointers must be 256-byte aligned.
 *   - Tensors are contiguous, row-major:
 *       keys, values  [B][Hkv][n_cap][d]   (MP_BF16 or MP_F32); n_cap = n unless a call takes
 *                                          a capacity (mp_params.n_capacity, or an n_capacity
 *                                          argument): a cache allocated for n_cap tokens per
 *                                          head of which the first n are in use
 *       q             [B][Hq][d]           (MP_BF16 or MP_F32)
 *       out           [B][Hq][d]           float32
 *       centre        [B][Hkv][d]          float32  (mu, the mean key of each head)
 *       W             [d][K*L]             (MP_BF16 or MP_F32); column j = t*K + b is bit b
 *                                          (least significant first) of table t. One W serves
 *                                          every head and layer.
 *   - GQA: query head h reads KV head h / (Hq / Hkv); Hq must be a multiple of Hkv.
 *   - d must be 128. 0 <= K <= 32 and 1 <= L; K == 0 is the degenerate case where every key
 *     collides in every table (u = 1 when L >= 2).
 *   - Packed codes ("codes") are bit-sliced in blocks of 1024 keys: for head (b, g) and block
 *     blk = i / 1024, plane j (= t*K + b) is a row of 32 uint32 words, and bit (i % 32) of word
 *     (i % 1024) / 32 holds the sign bit of key i for hyperplane j. Layout:
 *       codes[((b*Hkv + g)*nblk + blk)*(K*L) + j][w],   nblk = ceil(n_cap / 1024).
 *     Bits of positions i >= n (padding, or capacity not yet in use) are unspecified.
 *   - Calls are asynchronous on `stream`: argument checks run on the host and return an error
 *     before anything is launched; device-side problems (a bounded wait that gave up) set a
 *     device status word that mp_device_status() reads.
 *   - No global mutable state besides that status word; calls on different streams may run
 *     concurrently if their buffers do not overlap.
 */
#ifndef MAGICPIG_H
#define MAGICPIG_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define MP_API __attribute__((visibility("default")))
#else
#define MP_API
#endif

#define MP_ABI_VERSION 9
#define MP_KEYS_PER_BLOCK 1024

typedef enum {
    MP_OK = 0,
    MP_ERR_INVALID_ARG = 1,   /* bad shape, null pointer, misalignment, inconsistent sizes */
    MP_ERR_UNSUPPORTED = 2,   /* a valid request the library does not implement (e.g. d != 128) */
    MP_ERR_CUDA = 3,          /* a CUDA runtime call failed; cudaGetLastError() has the cause */
    MP_ERR_TIMEOUT = 4,       /* a device-side bounded wait gave up (see mp_device_status) */
    MP_ERR_WORKSPACE = 5,     /* the workspace passed is smaller than *_workspace_bytes */
    MP_ERR_BOUNDS = 6         /* an index check of the MP_CHECKS build failed (see
                                 mp_debug_check_report); never raised by the product build */
} mp_status;

typedef enum { MP_F32 = 0, MP_BF16 = 1 } mp_dtype;

/* Decode parameters. K, L: LSH bits per table and tables ("LSH Sampling...", method details,
 * hash-function choice). n_sink, n_local: the exact set T = {0..n_sink-1} u {n-n_local..n-1},
 * attended with u = 1 and never sampled (Algorithm 1's static cache; "don't pick the tallest",
 * section 5). scale: score scale, 0 means 1/sqrt(d). flags: 0, MP_FLAG_MIPS or
 * MP_FLAG_CROSS_POLYTOPE.
 * n_capacity: tokens per head the keys, values and codes are laid out for (0 means n; else
 * n_capacity >= n). A decode cache that grows by appending (mp_encode_keys) keeps one
 * n_capacity for its lifetime and passes the current length as n.
 * n_indexed: keys [0, n_indexed) of each head are in the bucketed tables (0 means n; else
 * n_indexed <= n); only mp_sampled_attention_buckets reads it.
 * radius: with MP_FLAG_MIPS, [B][Hkv] float32 device array from mp_key_radius (the longest
 * centred key of each head); NULL otherwise.
 * logu_table: with MP_FLAG_CROSS_POLYTOPE, the MP_LOGU_TABLE_ENTRIES floats of mp_cp_logu_table
 * for this K and L; NULL otherwise. */
typedef struct {
    int K;
    int L;
    int n_sink;
    int n_local;
    float scale;
    unsigned flags;
    int n_capacity;
    int n_indexed;
    const float* radius;
    const float* logu_table;
} mp_params;

/* MIPS -> cosine variant ("LSH Sampling...", method details, variance reduction with LSH): the
 * query is extended by a 0 and each centred key k - mu by sqrt(r^2 - |k - mu|^2), r the longest
 * centred key, so the collision probability grows with the inner product: p_i = 1 -
 * arccos(q.(k_i - mu) / (|q| r)) / pi replaces the cosine of q and k_i - mu. W then has d + 1
 * rows ([d + 1][K*L]; the query uses the first d), the codes come from mp_encode_keys_mips, and
 * every decode call of the variant sets this flag and mp_params.radius. */
#define MP_FLAG_MIPS 1u

/* Cross-polytope variant (the hash "LSH Sampling..." names in its conclusion as the way to shrink
 * the tables): table t hashes x to the signed index of the largest |coordinate| of G_t x, G_t a
 * d x d matrix of i.i.d. N(0, 1) entries, code = 2 i + (1 if negative), one byte (d = 128); keys
 * are centred, the query is not; one hash per table (K must be 1). W is then G: [L][d][d], row j
 * of G_t at (t * d + j) * d. Codes are bytes [B][Hkv][ceil(n_cap/1024)][L][1024] (mp_cp_codes_bytes,
 * written by mp_encode_keys_cp). p_i is the collision probability of two vectors at the cosine
 * of q and k_i - mu for Gaussian G, p(rho) = 2d int int_{a,b>0} phi_rho(a,b) P[|X|<a, |Y|<b]^(d-1),
 * which has no closed form: the decode reads log u from mp_params.logu_table, built once by
 * mp_cp_logu_table (Gauss-Legendre quadrature; above rho = 0.99 p runs linearly to p(1) = 1).
 * Not with the MIPS variant, the bucketed tables or mp_decode_attention_noalloc
 * (MP_ERR_UNSUPPORTED there), and mp_debug_select gives no collision counts for it. */
#define MP_FLAG_CROSS_POLYTOPE 2u
#define MP_LOGU_TABLE_ENTRIES 4097

/* Human-readable name of a status code (static storage). */
MP_API const char* mp_status_string(mp_status s);

/* MP_ABI_VERSION of the loaded library. */
MP_API int mp_abi_version(void);

/* Bytes of packed codes for B*Hkv heads of n keys: B*Hkv*ceil(n/1024)*K*L*128. */
MP_API size_t mp_codes_bytes(int B, int Hkv, int n, int K, int L);

/* Workspace bytes mp_key_mean needs: fixed-order partial sums plus one counter per head (the
 * call clears the counters itself; the workspace needs no initial contents). */
MP_API size_t mp_key_mean_workspace_bytes(int B, int Hkv, int n, int d);

/* Centre of the cached keys: centre[b][g][:] = (1/n) sum_i keys[b][g][i][:], float32
 * accumulation in a fixed order (run-to-run identical).
 * ("LSH Sampling...", method details, data preprocessing and centering: keys are centred before
 * the tables are built; "don't pick the tallest", section 5.)
 * One kernel: each CTA sums a range of rows (1024, halved down to 64 while the B*Hkv heads
 * would have fewer than 608 ranges, a function of B*Hkv and n only), the last CTA of a head adds
 * the ranges in order. Errors: MP_ERR_INVALID_ARG for n < 1, null pointers; MP_ERR_WORKSPACE if
 * ws_bytes is short. */
MP_API mp_status mp_key_mean(const void* keys, mp_dtype key_dtype, int B, int Hkv, int n, int d,
                             float* centre, void* workspace, size_t ws_bytes,
                             cudaStream_t stream);

/* mp_key_mean over the first n keys of a cache laid out for n_capacity tokens per head
 * (n <= n_capacity); the workspace is mp_key_mean_workspace_bytes(B, Hkv, n, d). */
MP_API mp_status mp_key_mean_cap(const void* keys, mp_dtype key_dtype, int B, int Hkv,
                                 int n_capacity, int n, int d, float* centre, void* workspace,
                                 size_t ws_bytes, cudaStream_t stream);

/* Build the hash tables of one layer: centre each key, project it on the K*L hyperplanes of W,
 * keep the sign (bit = 1 iff w_j.(k_i - mu) > 0), pack into the bit-sliced codes above.
 * ("LSH Sampling...", background, LSH basics: Sign(w^T x); method details, hash-function choice
 * and system co-design item 2: the random projection runs on the GPU.)
 * bf16 keys with a bf16 W run on the tcgen05 tensor cores (exact products, fp32 accumulation);
 * other dtype pairs use an fp32 CUDA-core kernel.
 * codes: mp_codes_bytes(B, Hkv, n, K, L) bytes, 16-byte aligned; may be NULL when K == 0.
 * Errors: MP_ERR_INVALID_ARG (shapes, null, misalignment), MP_ERR_UNSUPPORTED (d != 128). */
MP_API mp_status mp_build_tables(const void* keys, mp_dtype key_dtype, const float* centre,
                                 const void* W, mp_dtype w_dtype, int B, int Hkv, int n, int d,
                                 int K, int L, uint32_t* codes, cudaStream_t stream);

/* Encode keys [n_begin, n_end) of every head of a cache laid out for n_capacity tokens per head
 * into codes laid out for n_capacity (mp_codes_bytes(B, Hkv, n_capacity, K, L) bytes), with a
 * given centre. This is the incremental append of decode tokens: after a build over the prompt
 * (mp_key_mean_cap + mp_encode_keys(0, n)), each new token's key is written to the cache at
 * position n and encoded with mp_encode_keys(n, n + 1); the next decode passes n + 1. The local
 * window of T slides with n, so the key that leaves it joins the sampled keys with the code it
 * got when it was appended. The centre stays the one of the build: the pages compute it once,
 * before the tables are built ("LSH Sampling...", method details, data preprocessing and
 * centering) and say nothing of updates; codes and the weights p_i both use the centre the
 * caller passes, so any fixed centre gives a consistent sampler, and refreshing it means a
 * rebuild (mp_key_mean_cap, then mp_encode_keys over [0, n)).
 * Bits of keys outside [n_begin, n_end) that share a 32-key word with the range are kept. Short
 * ranges (up to 64 keys) run on CUDA cores; longer ones re-encode whole 1024-key blocks (bf16
 * keys and W: tensor cores), which rewrites the blocks' other keys with their own codes again.
 * Errors: MP_ERR_INVALID_ARG (shapes, n_begin < 0, n_end > n_capacity, n_begin > n_end, null,
 * misalignment), MP_ERR_UNSUPPORTED (d != 128). An empty range does nothing. */
MP_API mp_status mp_encode_keys(const void* keys, mp_dtype key_dtype, const float* centre,
                                const void* W, mp_dtype w_dtype, int B, int Hkv, int n_capacity,
                                int n_begin, int n_end, int d, int K, int L, uint32_t* codes,
                                cudaStream_t stream);

/* mp_encode_keys for keys that no cache of full precision holds (a 4-bit cache, mp_kv4 below):
 * keys [B][Hkv][m][d] are the rows that join the context at [n_begin, n_begin + m) of every head.
 * Bits of all other keys are kept; codes as for mp_encode_keys. Up to three launches: the part of a
 * 1024-key block that the range begins in, whole blocks, the part that it ends in.
 * Errors: MP_ERR_INVALID_ARG (shapes, m < 0, n_begin < 0 or n_begin + m > n_capacity, null,
 * misalignment), MP_ERR_UNSUPPORTED (d != 128). m == 0 does nothing. */
MP_API mp_status mp_encode_rows(const void* keys, mp_dtype key_dtype, const float* centre,
                                const void* W, mp_dtype w_dtype, int B, int Hkv, int m,
                                int n_capacity, int n_begin, int d, int K, int L, uint32_t* codes,
                                cudaStream_t stream);

/* mp_encode_rows for sequences of different lengths: keys [B][Hkv][m][d] join the context of sequence
 * b at [positions[b], positions[b] + m) ([B] int32 on the device). A key that falls outside
 * [0, n_capacity) is left out; bits of all other keys are kept. For the few tokens of a decode step:
 * one launch on CUDA cores, with the sums of mp_encode_keys's short ranges (bit for bit).
 * Errors: MP_ERR_INVALID_ARG (shapes, m < 0, B Hkv > 65535, null, misalignment: positions 4 bytes),
 * MP_ERR_UNSUPPORTED (d != 128, m > 64: longer ranges are mp_encode_rows's). m == 0 does nothing. */
MP_API mp_status mp_encode_rows_at(const void* keys, mp_dtype key_dtype, const float* centre,
                                   const void* W, mp_dtype w_dtype, int B, int Hkv, int m,
                                   int n_capacity, const int32_t* positions, int d, int K, int L,
                                   uint32_t* codes, cudaStream_t stream);

/* Workspace bytes mp_decode_attention (and its two halves below) need for these shapes;
 * 0 if the shapes or parameters are invalid. */
MP_API size_t mp_decode_workspace_bytes(int B, int Hq, int Hkv, int n, int d,
                                        const mp_params* prm);

/* One decode step of LSH-sampled attention for B*Hq query rows (Algorithm 1 of "LSH
 * Sampling...", method details, algorithm execution):
 *   q_code = Encode(q, W)                              (q is not centred)
 *   cnt_i  = #{t : code_t(k_i) == code_t(q)}           from the packed codes
 *   S      = {i not in T : cnt_i >= 2}
 *   p_i    = 1 - arccos(q.(k_i - mu) / (|q| |k_i - mu|)) / pi
 *   u_i    = 1 - (1 - p_i^K)^L - L p_i^K (1 - p_i^K)^(L-1)
 *   out    = softmax([s_S - log u_S, s_T]) . [V_S, V_T],   s = scale * q.k_i  (raw keys)
 * log u is a closed form, evaluated in fp32 in the log domain: directly when L p^K >= 0.05, else
 * as the binomial tail series from its second term. The query encoding tabulates it per call at
 * the 4097 cosines -1 + 2 i / 4096; a selected key takes the linear interpolation of that table
 * wherever the chord of its interval lies within 2e-5 of the closed form at the interval's
 * midpoint, and the closed form itself elsewhere (mp_debug_log_inclusion returns exactly this
 * evaluation). The softmax over S and T is computed in pieces of 1024 keys and
 * merged by log-sum-exp (the "recursive attention" merge of the system co-design section). If S
 * and T are both empty the output row is zero. Zero-length q or k - mu gives cosine 0 (p = 1/2).
 * A query row with a NaN or infinite element gets a NaN output row; the other rows are unaffected
 * and the status word is not raised.
 * Errors: MP_ERR_INVALID_ARG (shapes, null, Hq % Hkv, B Hq > 65535, n_sink/n_local < 0, flags other than
 *         MP_FLAG_MIPS or MP_FLAG_CROSS_POLYTOPE, or a flag without its radius / log u table),
 *         MP_ERR_UNSUPPORTED (d != 128, Hq/Hkv not in {1, 2, 4, 8}, or K*L*(Hq/Hkv) so
 *         large that a CTA's query masks no longer fit in shared memory),
 *         MP_ERR_WORKSPACE (ws_bytes < mp_decode_workspace_bytes). */
MP_API mp_status mp_decode_attention(const void* q, mp_dtype q_dtype, const uint32_t* codes,
                                     const float* centre, const void* W, mp_dtype w_dtype,
                                     const void* keys, const void* values, mp_dtype kv_dtype,
                                     int B, int Hq, int Hkv, int n, int d, const mp_params* prm,
                                     float* out, void* workspace, size_t ws_bytes,
                                     cudaStream_t stream);

/* The two halves of mp_decode_attention, for callers that schedule or time them apart. Both
 * take the same workspace; mp_sampled_attention reads what mp_encode_query wrote there for the
 * same q, centre and shapes, so the two must run in that order on the same stream.
 *
 * mp_encode_query: q_code = Encode(q, W), plus |q| and q.mu (Algorithm 1's first step).
 * mp_sampled_attention: collision counts, S, gather of K_S and V_S, importance weights, and the
 * merged softmax with the exact set T (Algorithm 1's remaining steps). It may load codes, q and
 * centre before the work queued ahead of it has ended: they are to be written before
 * mp_encode_query is called, not between the two (keys and values may be).
 * Errors as mp_decode_attention (mp_encode_query takes any B Hq). */
MP_API mp_status mp_encode_query(const void* q, mp_dtype q_dtype, const float* centre,
                                 const void* W, mp_dtype w_dtype, int B, int Hq, int Hkv, int n,
                                 int d, const mp_params* prm, void* workspace, size_t ws_bytes,
                                 cudaStream_t stream);
MP_API mp_status mp_sampled_attention(const void* q, mp_dtype q_dtype, const uint32_t* codes,
                                      const float* centre, const void* keys, const void* values,
                                      mp_dtype kv_dtype, int B, int Hq, int Hkv, int n, int d,
                                      const mp_params* prm, float* out, void* workspace,
                                      size_t ws_bytes, cudaStream_t stream);

/* ---- Bucketed hash tables ---------------------------------------------------------------------
 * The retrieval structure of the pages: per table, the keys of each K-bit code ("LSH Sampling...",
 * system co-design item 3: the query's codes are looked up in L prebuilt hash tables; "don't pick
 * the tallest", section 6: every table stores a pointer to every key, and a query scans about
 * L n / 2^K entries). Layout per (sequence, KV head), 32-bit words: offsets[L][2^K + 1], then
 * members[L][n], then the build's scratch [L][8][2^K]; members[t][offsets[t][c] .. offsets[t][c+1])
 * are the keys with code c in table t. The order inside a bucket is not fixed (a bucket is a set).
 * mp_buckets_bytes: bytes for B*Hkv such tables (L (2^K + 1 + n + 8 * 2^K) words each); 0 if
 * K > 12 or the shapes are invalid. */
MP_API size_t mp_buckets_bytes(int B, int Hkv, int n, int K, int L);

/* Build the bucketed tables from the packed codes of mp_build_tables (same B, Hkv, n, K, L).
 * buckets: caller-owned device memory of mp_buckets_bytes bytes, 4-byte aligned; codes may be
 * NULL when K == 0. Errors: MP_ERR_INVALID_ARG (shapes, null, misalignment), MP_ERR_UNSUPPORTED
 * (K > 12). */
MP_API mp_status mp_build_buckets(const uint32_t* codes, int B, int Hkv, int n, int K, int L,
                                  uint32_t* buckets, cudaStream_t stream);

/* MIPS variant: radius[b][g] = max over keys [0, n) of |k_i - mu| (float32, [B][Hkv], written
 * by this call; fp32 arithmetic). The keys are laid out for n_capacity tokens per head.
 * Errors: MP_ERR_INVALID_ARG (shapes, null, misalignment), MP_ERR_UNSUPPORTED (d != 128). */
MP_API mp_status mp_key_radius(const void* keys, mp_dtype key_dtype, const float* centre,
                               int B, int Hkv, int n_capacity, int n, int d, float* radius,
                               cudaStream_t stream);

/* MIPS variant of mp_encode_keys: codes of keys [n_begin, n_end) from the extended centred keys,
 * bit = [sum_e W[e][j] (k[e] - mu[e]) + W[d][j] sqrt(max(0, r^2 - |k - mu|^2)) > 0].
 * W_aug: [d + 1][K*L]; radius from mp_key_radius (a key longer than r, appended after r was
 * taken, gets 0 in the extra coordinate).
 * norms_scratch: NULL, or caller-owned device memory of B*Hkv*n_capacity floats. With it, bf16
 * keys and W and more than 64 keys, whole 1024-key blocks are re-encoded on the tensor cores
 * (the centred part and the extra coordinate, split exactly into three bf16 terms, both by MMA;
 * the norms of the blocks' keys are written to the scratch first). Otherwise fp32 CUDA cores encode the range
 * itself, keeping the other keys' bits of the words it touches.
 * Errors as mp_encode_keys; MP_ERR_INVALID_ARG also for a NULL radius. */
MP_API mp_status mp_encode_keys_mips(const void* keys, mp_dtype key_dtype, const float* centre,
                                     const void* W_aug, mp_dtype w_dtype, const float* radius,
                                     int B, int Hkv, int n_capacity, int n_begin, int n_end,
                                     int d, int K, int L, uint32_t* codes, float* norms_scratch,
                                     cudaStream_t stream);

/* Cross-polytope variant: bytes of codes for B*Hkv heads of n keys and L tables,
 * B*Hkv*ceil(n/1024)*L*1024; 0 for invalid shapes. */
MP_API size_t mp_cp_codes_bytes(int B, int Hkv, int n, int L);

/* Cross-polytope variant: log u at the MP_LOGU_TABLE_ENTRIES cosines -1 + 2 i / 4096, i.e.
 * log P[Binomial(L, p^K) >= 2] with p the cross-polytope collision probability (d = 128),
 * into the caller's float32 device array `table`, for mp_params.logu_table. One kernel of a few
 * milliseconds; build it once per (K, L). Errors: MP_ERR_INVALID_ARG (K, L < 1, null,
 * misalignment), MP_ERR_UNSUPPORTED (d != 128). */
MP_API mp_status mp_cp_logu_table(int K, int L, int d, float* table, cudaStream_t stream);

/* Cross-polytope variant: codes of keys [n_begin, n_end) of a cache laid out for n_capacity
 * tokens per head, G [L][d][d] (MP_F32 or MP_BF16), ties to the smaller index. With bf16 keys and
 * G and more than 64 keys, whole 1024-key blocks are re-encoded on the tensor cores (the
 * encoder's projections, an argmax instead of the signs); otherwise fp32 CUDA cores encode the
 * range itself and leave other keys' bytes untouched (appends).
 * codes: mp_cp_codes_bytes(B, Hkv, n_capacity, L) bytes, 16-byte aligned.
 * Errors: MP_ERR_INVALID_ARG (shapes, range, null, misalignment), MP_ERR_UNSUPPORTED (d != 128). */
MP_API mp_status mp_encode_keys_cp(const void* keys, mp_dtype key_dtype, const float* centre,
                                   const void* G, mp_dtype g_dtype, int B, int Hkv,
                                   int n_capacity, int n_begin, int n_end, int d, int L,
                                   uint8_t* codes, cudaStream_t stream);

/* mp_build_buckets over keys [0, n) of codes laid out for n_capacity tokens per head (the
 * appendable cache of mp_encode_keys); buckets is mp_buckets_bytes(B, Hkv, n, K, L) bytes. A
 * decode then passes n_indexed = n in mp_params while its own n grows. */
MP_API mp_status mp_build_buckets_cap(const uint32_t* codes, int B, int Hkv, int n_capacity,
                                      int n, int K, int L, uint32_t* buckets,
                                      cudaStream_t stream);

/* mp_sampled_attention with the bucketed tables instead of a scan of the packed codes: each
 * query row reads its bucket in every table and keeps the keys hit by >= 2 tables (the same S as
 * the scan, bit for bit), then the same gather, importance weights and merged softmax. Needs the
 * query encoding of mp_encode_query in the workspace first, like mp_sampled_attention.
 * The tables cover keys [0, prm->n_indexed); keys appended since (up to n) are found by the code
 * scan over the 1024-key blocks from n_indexed / 1024 on, which replaces the lookup's result in
 * those blocks. So codes must be passed too (NULL only when n_indexed == n and n is a multiple
 * of 1024, or K == 0) and the tables must have been built for n_indexed keys.
 * buckets: 16-byte aligned. Errors as mp_sampled_attention; MP_ERR_UNSUPPORTED also for K > 12. */
MP_API mp_status mp_sampled_attention_buckets(const void* q, mp_dtype q_dtype,
                                              const uint32_t* buckets, const uint32_t* codes,
                                              const float* centre,
                                              const void* keys, const void* values,
                                              mp_dtype kv_dtype, int B, int Hq, int Hkv, int n,
                                              int d, const mp_params* prm, float* out,
                                              void* workspace, size_t ws_bytes,
                                              cudaStream_t stream);

/* ---- 4-bit K/V cache ----------------------------------------------------------------------------
 * A cache of n_capacity tokens per (sequence, KV head) in 144 bytes a token and head (bf16: 512).
 * The pages keep K and V at the model's precision; this cache is an addition. Tensors, contiguous
 * and 16-byte aligned, owned by the caller:
 *   k_codes, v_codes  [B][Hkv][n_capacity][64]  uint8; byte i holds dims 2 i (low half) and 2 i + 1
 *   params            [B][Hkv][n_capacity][8]   bf16: s, z of the key's dims 0-63, s, z of its dims
 *                                               64-127, then the same of the value
 * Each group of 64 dims x_e is held by its own minimum and step: z is the largest bf16 with
 * z <= min x, s the smallest bf16 with z + 15 s >= max x, and the code is the integer nearest to
 * (x_e - z) / s (ties to even; 0 where s = 0), so that the value held, z + s code, is within s / 2
 * of x_e. A group with a NaN or an infinity, or whose spread passes bf16's range, is held as NaN
 * in all its 64 dims. Keys are held minus the centre of their head (x = k - mu in float32): the
 * offset that a head's keys share then costs no code, the softmax over one head's keys does not
 * see it, and the cosine of the sampled decode is that of k - mu. */
typedef struct {
    void* k_codes;
    void* v_codes;
    void* params;
    int n_capacity;
} mp_kv4;
#define MP_KV4_GROUP 64          /* dims that share a minimum and a step */
#define MP_KV4_CODE_BYTES 64     /* bytes of a row of k_codes or v_codes */
#define MP_KV4_PARAMS 8          /* bf16 of a row of params */

/* Write m tokens of every head into the cache: keys and values [B][Hkv][m][d] (MP_BF16 or MP_F32)
 * go to rows [n_begin, n_begin + m) of their head, or, with positions ([B] int32 on the device),
 * to rows [positions[b], positions[b] + m) of sequence b (n_begin is then ignored); a row that
 * falls outside [0, n_capacity) is not written. Other rows are left as they were. centre [B][Hkv][d]
 * is subtracted from the keys; NULL subtracts nothing.
 * Errors: MP_ERR_INVALID_ARG (shapes, m < 0, B Hkv m > 2^31 - 1, n_begin < 0 or n_begin + m >
 * n_capacity without positions, null, misalignment: keys and values 16 bytes, centre 16, positions 4),
 * MP_ERR_UNSUPPORTED (d != 128). m == 0 does nothing. */
MP_API mp_status mp_kv4_write(const void* keys, const void* values, mp_dtype kv_dtype,
                              const float* centre, int B, int Hkv, int m, int d, int n_begin,
                              const int32_t* positions, const mp_kv4* cache, cudaStream_t stream);

/* Read m tokens of every head back, from the rows that mp_kv4_write would write: keys and values
 * [B][Hkv][m][d] in kv_dtype, keys with the centre added again (float32 z + s code, rounded once,
 * plus mu, rounded, then the rounding to bf16). A row outside [0, n_capacity) reads as zero, in
 * keys and values both. Errors as mp_kv4_write. */
MP_API mp_status mp_kv4_read(const mp_kv4* cache, const float* centre, int B, int Hkv, int m, int d,
                             int n_begin, const int32_t* positions, void* keys, void* values,
                             mp_dtype kv_dtype, cudaStream_t stream);

/* Workspace bytes of mp_kv4_attention for these shapes and for any smaller n (0 if they are invalid,
 * and where no such call needs one): a decode that grows keeps the workspace of its capacity. The
 * workspace needs no initial contents; two calls that may overlap, captured ones among them, need
 * one each. */
MP_API size_t mp_kv4_attention_workspace_bytes(int B, int Hq, int Hkv, int n, int d);

/* 1 if mp_kv4_attention of exactly these shapes uses its workspace, 0 if NULL does (and for shapes
 * that are invalid). */
MP_API int mp_kv4_attention_uses_workspace(int B, int Hq, int Hkv, int n, int d);

/* Exact attention of one query token per sequence over the cache's first n tokens:
 *   out[b][h] = sum_i w_i v_i / sum_i w_i,   w_i = exp(scale q.k_i),   i < length_b
 * with the values that the cache holds; length_b = n, or lengths[b] ([B] int32 on the device,
 * taken into [0, n]). A sequence of length 0 gets zero rows. The work is laid out for n: where every
 * length is far below it, a smaller n is faster. Any Hq that Hkv divides.
 * scale 0 means 1/sqrt(d). Scores, softmax and sums are float32: codes and the two fp16 halves of a
 * query element or a weight (22 bits) meet in exact tensor-core products. An element of a query
 * enters within 2^-22 of itself and 2^-25 of the largest of its row. Sums over tokens take weights
 * of up to 1 each, before the division: they may overflow where the largest value attended to,
 * whatever its weight, times the tokens passes 2^126; so may scores where a key passes 2^124. A NaN
 * or an infinity in a query gives NaN in its output row (so may an element of 2^121 or more); one
 * that the cache holds gives NaN to the rows that attend to it (in a value: to its 64 dims).
 * Errors: MP_ERR_INVALID_ARG (shapes, n > n_capacity or 2^30, B Hq > 2^22, Hq % Hkv, a scale that is
 * negative, infinite or NaN, null, misalignment: out 16 bytes, lengths 4, workspace 256),
 * MP_ERR_UNSUPPORTED (d != 128), MP_ERR_WORKSPACE. */
MP_API mp_status mp_kv4_attention(const void* q, mp_dtype q_dtype, const mp_kv4* cache, int B, int Hq,
                                  int Hkv, int n, int d, const int32_t* lengths, float scale,
                                  float* out, void* workspace, size_t ws_bytes,
                                  cudaStream_t stream);

/* mp_decode_attention, mp_sampled_attention and mp_sampled_attention_buckets with the keys and
 * values of a 4-bit cache, written with the centre that these calls get: the codes are those of the
 * keys themselves (mp_encode_keys and its variants, before the cache is written), the scores and
 * the cosine of p_i are those of the keys that the cache holds, and log u of the SimHash codes is
 * evaluated for each sampled key (off by about 2^-22 (K + 1) at most). Keys beyond 2^60 and values
 * whose groups span more than 2^110 may overflow on the way. prm->n_capacity is the codes'
 * capacity, cache->n_capacity the cache's own (>= n). Workspaces, the query encoding
 * (mp_encode_query), variants and errors as for those calls. */
MP_API mp_status mp_kv4_decode_attention(const void* q, mp_dtype q_dtype, const uint32_t* codes,
                                         const float* centre, const void* W, mp_dtype w_dtype,
                                         const mp_kv4* cache, int B, int Hq, int Hkv, int n, int d,
                                         const mp_params* prm, float* out, void* workspace,
                                         size_t ws_bytes, cudaStream_t stream);
MP_API mp_status mp_kv4_sampled_attention(const void* q, mp_dtype q_dtype, const uint32_t* codes,
                                          const float* centre, const mp_kv4* cache, int B, int Hq,
                                          int Hkv, int n, int d, const mp_params* prm, float* out,
                                          void* workspace, size_t ws_bytes, cudaStream_t stream);
MP_API mp_status mp_kv4_sampled_attention_buckets(const void* q, mp_dtype q_dtype,
                                                  const uint32_t* buckets, const uint32_t* codes,
                                                  const float* centre, const mp_kv4* cache, int B,
                                                  int Hq, int Hkv, int n, int d,
                                                  const mp_params* prm, float* out,
                                                  void* workspace, size_t ws_bytes,
                                                  cudaStream_t stream);

/* ---- Paged K/V cache ----------------------------------------------------------------------------
 * A pool of pages of page_size tokens of every KV head, keys and values at full precision, and a
 * table that says which pages a sequence's tokens lie in: sequences of any lengths share one pool,
 * grow by a page at a time and may share pages that hold the same tokens. Tensors, owned by the
 * caller:
 *   keys, values  [n_pages][Hkv][page_size][d]   MP_BF16 or MP_F32, contiguous, 16-byte aligned
 *   page_table    [B] rows of n_slots int32, table_stride apart; slot j of row b is the page of
 *                 tokens [j page_size, (j + 1) page_size) of sequence b
 * A slot that holds a number outside [0, n_pages) has no page: its tokens are not written, and
 * attention goes on as if they were not there. Slots behind a call's last token are not looked at.
 * page_size is a multiple of 8. A call may write a token's row once: two sequences that share a page
 * may read it in one call, not write the same rows of it. */
typedef struct {
    void* keys;
    void* values;
    const int32_t* page_table;
    mp_dtype dtype;
    int n_pages;
    int page_size;
    int n_slots;
    int table_stride;
} mp_paged;

/* Rows [B][H][m][d] of a tensor whose first three dims have strides of their own (in elements; a
 * row's d elements follow each other): the queries, keys or values of one fused projection are such
 * rows. data and the strides of dims longer than one are multiples of 16 bytes. */
typedef struct {
    const void* data;
    long long stride_b;
    long long stride_h;
    long long stride_m;
} mp_rows;

/* Append m tokens of every sequence to the cache, with their rotary positions applied on the way.
 * Token i of sequence b stands at p = n_begin + i, or, with positions ([B] int32 on the device), at
 * p = positions[b] + i (n_begin is then ignored). With counts ([B] int32 on the device) only the
 * first counts[b] tokens of a sequence are there (taken into [0, m]); nothing is written for others.
 *   keys, values  [B][Hkv][m][d] of rows_dtype: go to row p of the pages of their sequence, in the
 *                 cache's type; a token whose p has no page is not written
 *   q             [B][Hq][m][d] of rows_dtype: the rotated queries go to q_out, [B][Hq][m][d] of the
 *                 same type, contiguous. NULL where there are none. q_out may be q where q is contiguous.
 *   keys_out      [B][Hkv][m][d] of the cache's type, contiguous, or NULL: the keys as the cache holds
 *                 them, for the calls that encode them (of tokens without a page too)
 * Rotation: the first rotary_dims dims of a row are pairs; pair j = (x, y) becomes
 * (x cos a - y sin a, y cos a + x sin a), a = p inv_freq[j] (float32 on the device, rotary_dims / 2
 * of them), in float32, rounded once to the type it is stored in. Pairs are dims (j, j + rotary_dims /
 * 2), or with interleaved != 0 dims (2 j, 2 j + 1). The angle is reduced in 64-bit fixed point: it is
 * off by less than 2^-61 |p| (1 + |inv_freq[j]|) + 2^-25 radians at any position (2^-23 where rows and
 * cache are both bf16). inv_freq NULL (rotary_dims then ignored) turns nothing. An inv_freq that is
 * infinite or NaN has unspecified results.
 * Errors: MP_ERR_INVALID_ARG (shapes, m < 0, Hq + 2 Hkv > 2^18, B m (Hq + 2 Hkv) > 2^31 - 1, n_begin
 * < 0 or n_begin + m > n_slots page_size without positions, null, misalignment: rows, outputs 16
 * bytes, others 4),
 * MP_ERR_UNSUPPORTED (d != 128, page_size not a multiple of 8, rotary_dims not a multiple of 16 in
 * [16, 128]). m == 0 does nothing. */
MP_API mp_status mp_paged_append(const mp_rows* keys, const mp_rows* values, const mp_rows* q,
                                 mp_dtype rows_dtype, const float* inv_freq, int rotary_dims,
                                 int interleaved, int B, int Hq, int Hkv, int m, int d, int n_begin,
                                 const int32_t* positions, const int32_t* counts,
                                 const mp_paged* cache, void* q_out, void* keys_out,
                                 cudaStream_t stream);

/* Workspace bytes of mp_paged_attention for these shapes, whatever n is (0 if they are invalid). It
 * needs no initial contents; two calls that may overlap, captured ones among them, need one each. */
MP_API size_t mp_paged_attention_workspace_bytes(int B, int Hq, int Hkv, int n, int d);

/* Exact attention of one query token per sequence over the first n tokens of its pages:
 *   out[b][h] = sum_i w_i v_i / sum_i w_i,   w_i = exp(scale q.k_i),   i < length_b
 * length_b = n, or lengths[b] ([B] int32 on the device, taken into [0, n]). The work is shared out by
 * the lengths themselves, on the device: n may be the table's whole capacity. A sequence of length
 * 0, or whose tokens have no page, gets zero rows. Any Hq that Hkv divides. scale 0 means 1/sqrt(d).
 * Scores, softmax and sums are float32: over a bf16 cache the products are tensor-core products of
 * bf16, a float32 query element or a weight being three bf16 terms (24 bits); over a float32 cache with
 * more than four query heads a KV head, of tf32, every number being two terms (22 bits and more). What
 * the pages hold beyond a sequence's length is not looked at, NaN included. A NaN or an infinity in a
 * query, or in a key or value attended to, may give NaN in the rows that it meets, and so may an element
 * past the largest bf16 or tf32 where it is split.
 * Sums over tokens take weights of up to 1 each, before the division: they may overflow where the largest
 * value attended to times the tokens passes 2^127, and so may a score's sum of 128 products.
 * Errors: MP_ERR_INVALID_ARG (shapes, n > n_slots page_size or 2^30, B Hq > 2^22, B Hq n > 2^35, Hq %
 * Hkv, a scale that is negative, NaN, or infinite in float32 once multiplied by log2 e, null, misalignment:
 * out 16 bytes, lengths 4, workspace 256), MP_ERR_UNSUPPORTED (d != 128, page_size not a multiple of 8),
 * MP_ERR_WORKSPACE. */
MP_API mp_status mp_paged_attention(const void* q, mp_dtype q_dtype, const mp_paged* cache, int B,
                                    int Hq, int Hkv, int n, int d, const int32_t* lengths,
                                    float scale, float* out, void* workspace, size_t ws_bytes,
                                    cudaStream_t stream);

/* mp_decode_attention over a paged cache, for sequences of different lengths: keys i < length_b
 * (mp_paged_attention's) of sequence b, T = {0 .. n_sink-1} u {length_b-n_local .. length_b-1}. The
 * codes are contiguous per sequence, as for the other calls, laid out for prm->n_capacity tokens (0
 * means n), and hold the keys' own tokens at their positions (mp_encode_rows, mp_encode_rows_at of
 * the keys that mp_paged_append returns). A token without a page is left out, of T too. log u of the
 * SimHash codes is evaluated for each sampled key. Workspace: mp_decode_workspace_bytes.
 * Errors: those of mp_decode_attention, and MP_ERR_INVALID_ARG (the cache, lengths, n > n_slots
 * page_size or 2^30, an infinite scale), MP_ERR_UNSUPPORTED (page_size not a multiple of 8). */
MP_API mp_status mp_paged_decode_attention(const void* q, mp_dtype q_dtype, const uint32_t* codes,
                                           const float* centre, const void* W, mp_dtype w_dtype,
                                           const mp_paged* cache, int B, int Hq, int Hkv, int n, int d,
                                           const int32_t* lengths, const mp_params* prm, float* out,
                                           void* workspace, size_t ws_bytes, cudaStream_t stream);

/* Workspace bytes mp_debug_select needs. */
MP_API size_t mp_debug_workspace_bytes(int B, int Hq, int Hkv, int n, int d,
                                       const mp_params* prm);

/* mp_decode_attention plus what it decided, for checking against a reference:
 *   q_bits    [B][Hq][ceil(K*L/32)] uint32: bit j%32 of word j/32 is the query's sign bit j
 *   sel_idx   [B][Hq][n] int32: ascending indices of S (the sampled set, T excluded), the first
 *             sel_count[b][h] entries are valid
 *   sel_count [B][Hq] int32
 *   cnt       [B][Hq][n] uint8 collision counts (saturating at 255), or NULL to skip
 * The selection comes from the same kernel mp_decode_attention runs; cnt from a separate
 * counting kernel. Errors as mp_decode_attention. */
MP_API mp_status mp_debug_select(const void* q, mp_dtype q_dtype, const uint32_t* codes,
                                 const float* centre, const void* W, mp_dtype w_dtype,
                                 const void* keys, const void* values, mp_dtype kv_dtype, int B,
                                 int Hq, int Hkv, int n, int d, const mp_params* prm, float* out,
                                 uint32_t* q_bits, int32_t* sel_idx, int32_t* sel_count,
                                 uint8_t* cnt, void* workspace, size_t ws_bytes,
                                 cudaStream_t stream);

/* mp_sampled_attention_buckets plus what it decided, for checking the bucketed retrieval against
 * a reference: the query encoding of mp_encode_query (its sign bits into q_bits), the bucket lookup
 * (and the scan of keys appended since the tables were built), the same attend kernel, and the
 * sampled sets S (T excluded, ascending) into sel_idx / sel_count, laid out as in mp_debug_select.
 * The workspace is mp_debug_workspace_bytes. Errors as mp_sampled_attention_buckets. */
MP_API mp_status mp_debug_select_buckets(const void* q, mp_dtype q_dtype, const uint32_t* buckets,
                                         const uint32_t* codes, const float* centre,
                                         const void* W, mp_dtype w_dtype, const void* keys,
                                         const void* values, mp_dtype kv_dtype, int B, int Hq,
                                         int Hkv, int n, int d, const mp_params* prm, float* out,
                                         uint32_t* q_bits, int32_t* sel_idx, int32_t* sel_count,
                                         void* workspace, size_t ws_bytes, cudaStream_t stream);

/* log u at each of `count` cosines c (float32 device arrays cosines -> out), evaluated as the
 * decode kernels evaluate it for every selected key of the SimHash codes (the per-call table and
 * the closed form where the table is not used, as mp_decode_attention describes): p = 1 -
 * arccos(c) / pi, u = P[Binomial(L, p^K) >= 2] ("LSH Sampling...", method details, the u_i formula),
 * in fp32 in the log domain; p = 0 gives log(FLT_MIN), L = 1 gives -inf. For checking that
 * evaluation against a reference. Errors: MP_ERR_INVALID_ARG (count < 0, K outside [0, 32],
 * L < 1, null or misaligned arrays). */
MP_API mp_status mp_debug_log_inclusion(const float* cosines, int count, int K, int L, float* out,
                                        cudaStream_t stream);

/* Test hook of the failure path: one thread waits, with the bounded wait the tensor-core encoder
 * uses on its pipeline barriers, on an mbarrier that nothing completes (no arrival, copy or MMA is
 * issued), gives up after limit_us microseconds (1 to 100000) and records MP_ERR_TIMEOUT in the
 * device status word, as a stalled encoder would; mp_device_status then returns it once.
 * The paper has no counterpart. Errors: MP_ERR_INVALID_ARG (limit out of range). */
MP_API mp_status mp_debug_wait_expiry(int limit_us, cudaStream_t stream);

/* Unpack codes into one integer per (key, table): table_codes[b][g][i][t] = code_t(k_i) =
 * sum_b bit_{i, t*K+b} << b. Requires K <= 32. */
MP_API mp_status mp_codes_unpack(const uint32_t* codes, int B, int Hkv, int n, int K, int L,
                                 uint32_t* table_codes, cudaStream_t stream);

/* Size of the fixed scratch array mp_decode_attention_noalloc uses (8 MiB). */
#define MP_NOALLOC_SCRATCH_BYTES (8u << 20)

/* mp_decode_attention for callers that cannot allocate device memory. The paper has no
 * counterpart; this entry point exists for callers such as plugins of a runtime that owns all
 * device memory through its own pool, or latency-critical loops where an allocation (which may
 * synchronise the device) is not allowed, or code that holds no allocator at all. It takes the
 * same inputs and output as mp_decode_attention, without a workspace: its scratch is a fixed
 * array of MP_NOALLOC_SCRATCH_BYTES inside the library, resident on every GPU that loads the
 * library until the process exits. It never allocates or frees memory.
 *   - The first call on a device (with that device current) resolves the array's address and
 *     loads the decode kernels; make that first call before any stream capture.
 *   - Shapes that need more scratch than the array holds (mp_decode_workspace_bytes() above
 *     MP_NOALLOC_SCRATCH_BYTES) are rejected with MP_ERR_WORKSPACE before anything is launched.
 *   - Every call on a device shares the one array. The merge counters are reset at the start of
 *     each call and the rest is written before it is read, so sequential calls are independent;
 *     calls whose kernels overlap on the GPU (other streams, unordered threads) race on it.
 * Other errors as mp_decode_attention. */
MP_API mp_status mp_decode_attention_noalloc(const void* q, mp_dtype q_dtype,
                                             const uint32_t* codes, const float* centre,
                                             const void* W, mp_dtype w_dtype, const void* keys,
                                             const void* values, mp_dtype kv_dtype, int B, int Hq,
                                             int Hkv, int n, int d, const mp_params* prm,
                                             float* out, cudaStream_t stream);

/* Synchronise the current device, return its status word (MP_OK, MP_ERR_TIMEOUT, or in the
 * MP_CHECKS build MP_ERR_BOUNDS) through *status and reset it, with the check site beside it, to
 * MP_OK. Returns MP_ERR_CUDA if the device cannot be reached. */
MP_API mp_status mp_device_status(int* status);

/* The MP_CHECKS build (the library compiled with -DMP_CHECKS=1, libmagicpig_checks.so): every
 * kernel of the decode path, the bucketed lookup, the tensor-core encoder, the CUDA-core encoders
 * of mp_encode_keys, mp_encode_rows and mp_encode_rows_at, the 4-bit cache and the paged cache check
 * the indices of their global accesses (code blocks, selection words, K/V rows, partial states, bucket
 * ranges and members, code words written) and skip an access that is out of range instead of making
 * it, raising MP_ERR_BOUNDS in the status word. A stand-in for a memory checker: the paper has no
 * counterpart.
 * Synchronises the device and returns through *enabled 1 in that build, 0 in the product build, and
 * through *site the site of the first failed check since the status word was last reset (0 if
 * none): 1 query encoding stores, 2 scanned code block, 3 selection words written, 4 K/V row
 * copied, 5 partial state or output written, 6 selection words read, 7 bucket range beyond the
 * table's keys, 8 bucket member beyond n_indexed, 9 code words written by the encoders, 10 a row of
 * the 4-bit cache, 11 rows read back from it, partial states and output rows of its attention, 12 a
 * key row that a CUDA-core encoder reads, 13 the list of an attend CTA's selected keys, 14 a row of the
 * paged cache or a slot of its page table (the boxes that the bf16 attention copies by TMA are checked
 * by that unit, against the pool), 15 rows returned by an append to it, and of its attention output
 * rows, partial states and what says where they begin, against the workspace's size. Neither word is reset. Errors: MP_ERR_INVALID_ARG (null), MP_ERR_CUDA. */
MP_API mp_status mp_debug_check_report(int* enabled, int* site);

#ifdef __cplusplus
}
#endif
#endif /* MAGICPIG_H */
