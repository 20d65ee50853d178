/*
 * mnb.h -- block-quantized INT4 (MatMulNBits) products on one GB300 GPU (sm_103a).
 *
 * The library computes Y[M,N] = A[M,K] . dequant(B)^T for weights stored in the
 * ONNX com.microsoft::MatMulNBits layout, as spelled out in
 *   onnx-runtime-ep-cuda 0.1.0-dev.6, src/kernels/marlin_gemm.rs, module doc,
 *   section "ONNX MatMulNBits int4 format", and
 *   onnx-runtime-ep-cuda 0.1.0-dev.3, src/kernels/matmul_nbits.rs, kernel
 *   matmul_nbits_dequant_f32:
 *
 *   packed       uint8 [N, k_blocks, bs/2], k_blocks = K/bs. The nibble for (n, k) is in
 *                byte (n*k_blocks + k/bs)*(bs/2) + (k%bs)/2: low nibble for even k,
 *                high nibble for odd k. code in 0..15. (With K % bs == 0 every row is
 *                simply K/2 consecutive bytes.)
 *   scales       [N, k_blocks], fp16 or fp32.
 *   zero_points  optional uint8 [N, ceil(k_blocks/2)]: the nibble for (n, g) is in byte
 *                n*ceil(k_blocks/2) + g/2, low nibble for even g. NULL means zp = 8.
 *   dequant(B)[n, k] = (code[n, k] - zp[n, k/bs]) * scale[n, k/bs].
 *
 * Conventions shared by every entry point
 *   - Every pointer argument is device memory owned by the caller (except where an
 *     argument is marked HOST); the library keeps no reference after the call returns
 *     and allocates nothing.
 *   - A and Y are fp16 (IEEE binary16, passed as raw 16-bit storage), row-major, except
 *     in mnb_gemm_f32, where they are fp32.
 *   - Every device pointer must be non-NULL (except zero_points, workspace when
 *     ws_bytes is 0, and repacked where stated) and 16-byte aligned:
 *     otherwise MNB_ERR_INVALID_ARG / MNB_ERR_MISALIGNED.
 *   - block_size must be 16, 32, 64 or 128 and K a multiple of it; K, N, M >= 1 and
 *     K, N <= 2^24, M <= 2^20. Otherwise MNB_ERR_INVALID_ARG or MNB_ERR_UNSUPPORTED.
 *   - Work is enqueued on `stream` (a cudaStream_t; NULL is the legacy default stream)
 *     and runs asynchronously: the call neither synchronises nor copies to the host,
 *     so every compute call may be captured into a CUDA graph. Launch geometry depends
 *     only on the shape arguments and the device.
 *   - Errors never throw. A non-MNB_OK status leaves a message for mnb_last_error()
 *     (per host thread). MNB_ERR_CUDA carries the CUDA error string.
 *   - Results are deterministic: the same inputs give the same bits on every run.
 */
#ifndef MNB_H_
#define MNB_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define MNB_API __attribute__((visibility("default")))
#else
#define MNB_API
#endif

struct CUstream_st; /* cudaStream_t is `struct CUstream_st *` */
typedef struct CUstream_st *mnb_stream;

typedef enum {
    MNB_OK = 0,
    MNB_ERR_INVALID_ARG = 1,  /* bad shape, block size, NULL pointer, or dtype */
    MNB_ERR_UNSUPPORTED = 2,  /* valid for the format, but not handled by this build */
    MNB_ERR_MISALIGNED = 3,   /* a pointer is not 16-byte aligned */
    MNB_ERR_CAPTURE = 4,      /* the call is refused while `stream` is being captured */
    MNB_ERR_CUDA = 5,         /* a CUDA runtime call or launch failed */
    MNB_ERR_TIMEOUT = 6       /* a bounded device-side wait gave up (kernel status word) */
} mnb_status;

typedef enum { MNB_F16 = 0, MNB_F32 = 1 } mnb_dtype;

/* One quantised weight: the MatMulNBits tuple (packed, scales, zero_points). */
typedef struct {
    const uint8_t *packed;      /* [N, K/2] bytes                                   */
    const void *scales;         /* [N, K/bs] of fp16 or fp32 (scales_dtype)          */
    int32_t scales_dtype;       /* MNB_F16 or MNB_F32                                */
    const uint8_t *zero_points; /* [N, ceil(K/bs/2)] nibbles, or NULL for zp = 8      */
} mnb_weight;

/*
 * Dequantise to fp32 [K, N] (row k, column n at out_kn[k*N + n]).
 * Follows matmul_nbits_dequant_f32 (matmul_nbits.rs): element (code - zp) * scale.
 * The product is rounded once to fp32 (round to nearest even); it is exact for fp16
 * scales. out_kn holds K*N floats.
 */
MNB_API mnb_status mnb_dequant(mnb_weight w, int K, int N, int block_size, float *out_kn,
                       mnb_stream stream);

/*
 * Size in bytes of the repacked tensor-core operand for a K x N weight:
 * ceil(N/128)*128 * ceil(K/64)*64 / 2. Returns 0 for invalid arguments.
 */
MNB_API size_t mnb_repacked_bytes(int K, int N, int block_size);

/*
 * Reorder `packed` into this library's tensor-core operand layout (a bijection on the
 * codes; scales and zero points keep their MatMulNBits indexing). The pages repack
 * once for their mma.sync kernel (marlin_gemm.rs, "Repacked weight layout"); the layout
 * here is new, built for 1-D bulk copies and shared-memory dequantisation:
 *   tile t (128 rows) and k-block b (64 k) form one 4096-byte block at
 *   (t * ceil(K/64) + b) * 4096; in it the 16 bytes at q*2048 + r*16 (q in 0..1,
 *   r in 0..127) hold the codes of row n = 128t + r for k = 64b + 32q + i, i in 0..31,
 *   as four little-endian 32-bit words; word j = i/8 keeps i at nibble p (bits 4p..4p+3)
 *   where i = 8j + 2(p%4) + p/4. Codes outside the K x N weight are 0.
 * `out` holds mnb_repacked_bytes(K, N, block_size) bytes. Runs once per weight, so it is
 * refused with MNB_ERR_CAPTURE while `stream` is capturing (a repack inside a graph
 * would be replayed on every launch).
 */
MNB_API mnb_status mnb_repack(const uint8_t *packed, int K, int N, int block_size, uint8_t *out,
                      mnb_stream stream);

/*
 * Decode GEMV, M = 1: Y[n] = sum_k A[k] * dequant(B)[n, k], stored as fp16 (round to
 * nearest even from the fp32 accumulator). A is fp16 [K], Y is fp16 [N].
 * The per-group partial dot of (code - zp) and A is scaled after it is formed
 * (matmul_nbits.rs, matmul_nbits_gemv_f16; marlin_gemm.rs, "Per-group scale applied
 * after the tensor-core accumulate"). |Y - exact| <= 2e-3 * sum_k |a_k w_nk| + 1e-5.
 */
MNB_API mnb_status mnb_gemv(const void *A, mnb_weight w, int K, int N, int block_size, void *Y,
                    mnb_stream stream);

/*
 * Scratch bytes for mnb_gemm (and mnb_gemm_bias) at this shape (0 when none): fp32
 * partials ([slices, M, N]) of a K split, summed in slice order, so results stay
 * deterministic.
 *   2 <= M <= 16: required when K is too large for one shared-memory pass of the small-M
 *   kernel; the size is an upper bound over the scale dtype and zero points.
 *   M > 16: optional; with it, outputs with fewer 128 x 256 tiles than half the SMs split
 *   K (whole quant groups) over the SMs, without it they run unsplit. The size covers
 *   GPUs of up to 160 SMs.
 * The caller allocates it once and passes it to every call of that shape; its contents
 * need no initialisation, each call overwrites them, so calls sharing one workspace must
 * be ordered on one stream.
 */
MNB_API size_t mnb_workspace_bytes(int M, int K, int N, int block_size);

/*
 * Y[M, N] = A[M, K] . dequant(B)^T, fp16 in and out, fp32 accumulation.
 * M = 1 runs the GEMV. 2 <= M <= 16 (speculative verify) streams the MatMulNBits
 * storage directly; `repacked` may be NULL and is not read. M > 16 needs the repacked
 * operand from mnb_repack (`repacked` NULL gives MNB_ERR_INVALID_ARG) and runs on the
 * tcgen05 tensor cores,
 * the group scale applied to each group's partial accumulator (marlin_gemm.rs,
 * matmul_nbits_marlin_gemm_f16). `workspace`/`ws_bytes`: see mnb_workspace_bytes;
 * for 2 <= M <= 16 a smaller workspace gives MNB_ERR_INVALID_ARG.
 */
MNB_API mnb_status mnb_gemm(const void *A, int M, mnb_weight w, const uint8_t *repacked, int K, int N,
                    int block_size, void *workspace, size_t ws_bytes, void *Y,
                    mnb_stream stream);

/* Bias epilogue modes for mnb_gemm_bias. */
typedef enum {
    MNB_BIAS_NONE = 0,         /* Y = fp16(acc)                                          */
    MNB_BIAS_FUSED = 1,        /* Y = fp16(acc + b), one rounding (a fused MatMul+bias)   */
    MNB_BIAS_AFTER_ROUND = 2   /* Y = fp16(fp16(acc) + b), bit-identical to mnb_gemm
                                  followed by a separate fp16 add                          */
} mnb_bias_mode;

/*
 * mnb_gemm with a bias [N] (fp16, one value per output column) added in the epilogue,
 * in either of the two rounding orders of the pages' fp16 bias epilogue (matmul_nbits.rs,
 * fold_bias_f16; marlin_gemm.rs, fold_bias): MNB_BIAS_FUSED adds b to the fp32
 * accumulator and rounds once, MNB_BIAS_AFTER_ROUND rounds the accumulator to fp16 first
 * and then rounds fp32(that) + b. `bias` may be NULL only with MNB_BIAS_NONE.
 */
MNB_API mnb_status mnb_gemm_bias(const void *A, int M, mnb_weight w, const uint8_t *repacked, int K,
                                 int N, int block_size, const void *bias, int bias_mode,
                                 void *workspace, size_t ws_bytes, void *Y, mnb_stream stream);

/*
 * Paired gate/up projection with the SwiGLU epilogue (matmul_nbits.rs,
 * matmul_nbits_gemv_f16_gate_up_swiglu): g = A . gate^T, u = A . up^T (both M = 1,
 * same K, N, block_size), out[n] = silu(g[n]) * u[n] with silu(x) = x / (1 + e^-x),
 * computed in fp32 from the fp32 accumulators and stored as fp16. A is fp16 [K],
 * out is fp16 [N]. Each weight may use its own scale dtype and zero points.
 */
MNB_API mnb_status mnb_gemv_gate_up_swiglu(const void *A, mnb_weight gate, mnb_weight up, int K, int N,
                                   int block_size, void *out, mnb_stream stream);

/*
 * ---- fp32 activations ----
 *
 * The operator's fp32 path (matmul_nbits.rs, MatMulNBitsKernel::run with a Float32 A:
 * matmul_nbits_gemv_f32 for M = 1, dequantise-then-GEMM otherwise): A [M, K], Y [M, N]
 * and the optional bias [N] are fp32 (row-major, 16-byte aligned), Y = A . dequant(B)^T
 * + bias with no fp16 rounding anywhere. M = 1 multiplies fp32 activations directly. For
 * M >= 2 every row of A is scaled by a power of two and split into two fp16 rows (high
 * and low part, together within 2^-22 of the row) that the fp16 tensor-core kernels
 * multiply; their two accumulators are added and scaled back in fp32. Either way the
 * weights are exact and the accumulation is fp32, so |Y - exact| <= 2e-3 * sum_k |a_k
 * w_nk| + 1e-5 holds with a wide margin. A row holding inf or NaN gives non-finite
 * outputs in that row.
 */

/*
 * Workspace bytes for mnb_gemm_f32: 0 for M = 1, else 4*M*K (the split activation) +
 * 4*M rounded up to 16 (row exponents) + mnb_workspace_bytes(2*M, K, N, block_size)
 * (the K-slice partials of the 2*M split rows: required for M <= 8, optional above, as
 * in mnb_gemm).
 */
MNB_API size_t mnb_workspace_bytes_f32(int M, int K, int N, int block_size);

/*
 * fp32 Y[M, N] = A[M, K] . dequant(B)^T (+ bias[n] when bias is not NULL). Weight
 * arguments as mnb_gemm; `repacked` (mnb_repack) is required when M > 8, because the
 * split activation then has more than 16 rows and runs on the tcgen05 kernel. The
 * workspace holds the split activation, the row exponents and any K-slice partials; its contents need no
 * initialisation and are overwritten by each call, so calls sharing one workspace must
 * be ordered on one stream.
 */
MNB_API mnb_status mnb_gemm_f32(const float *A, int M, mnb_weight w, const uint8_t *repacked, int K, int N,
                                int block_size, const float *bias, void *workspace, size_t ws_bytes, float *Y,
                                mnb_stream stream);

/*
 * ---- Act-order weights (g_idx) ----
 *
 * MatMulNBits takes an optional int32 group index g_idx[K] (matmul_nbits.rs,
 * MatMulNBitsKernel::run, input 4; kernel matmul_nbits_dequant_f32): the scale and zero
 * point of column k are those of group g_idx[k] instead of group k / bs, while the code
 * still sits in block k / bs:
 *   dequant(B)[n, k] = (code[n, k] - zp[n, g_idx[k]]) * scale[n, g_idx[k]].
 * The pages check every entry with a device-to-host copy on each call. Here the check
 * happens once, on the host, when the weight is prepared (mnb_act_order_plan), and the
 * weight is rewritten into an equivalent plain block weight of K' columns
 * (mnb_act_order_prepare): k sorted by group, ascending k inside a group, each group's
 * run padded with empty slots to whole blocks. Each call then gathers the activation
 * into the same order and runs the ordinary kernels, so every per-call entry point
 * below is capture-safe. With g_idx[k] = k / bs the prepared weight is the original.
 */

/*
 * Dequantise with a group index per k to fp32 [K, N] (out_kn[k*N + n]), as
 * matmul_nbits_dequant_f32 does when given group indices: element
 * (code[n, k] - zp[n, g]) * scale[n, g], g = g_idx[k], rounded once to fp32. g_idx is
 * device int32 [K]. An entry outside 0..K/bs-1 writes 0 for that k (the pages' kernel
 * rule) and sets the index bit of the device status word, which mnb_check_device_status
 * reports as MNB_ERR_INVALID_ARG.
 */
MNB_API mnb_status mnb_dequant_gidx(mnb_weight w, const int32_t *g_idx, int K, int N, int block_size,
                                    float *out_kn, mnb_stream stream);

/*
 * Host-only planning step (no GPU work). g_idx is HOST int32 [K]; every entry must lie
 * in 0..K/bs-1, else MNB_ERR_INVALID_ARG names the first bad entry (the operator's own
 * check, matmul_nbits.rs). Writes *K_prepared = K' = bs * sum_g ceil(count_g / bs), with
 * K <= K' <= 2K (K' = K when every group has exactly bs members, the act-order
 * quantisation case). If perm is not NULL it receives K' entries (host int32): perm[k']
 * = the source column of prepared column k', or -1 for an empty slot. If block_group is
 * not NULL it receives K'/bs entries: the group of each prepared block. Call once with
 * NULL arrays to learn K', or size both for the 2K worst case.
 */
MNB_API mnb_status mnb_act_order_plan(const int32_t *g_idx, int K, int block_size, int32_t *K_prepared,
                                      int32_t *perm, int32_t *block_group);

/*
 * Write the prepared weight (device buffers owned by the caller, same block_size, K'
 * columns): packed_out [N, K'/2] bytes with codes code[n, perm[k']] (the block's zero
 * point at an empty slot, so its weight is 0); scales_out [N, K'/bs] of w.scales_dtype,
 * scales_out[n, j] = scales[n, block_group[j]]; zero_points_out [N, ceil(K'/bs/2)] bytes
 * (nibbles as in MatMulNBits, the unused high nibble of an odd count 0), required when w
 * has zero points and ignored otherwise (the prepared weight then has none either).
 * perm [K'] and block_group [K'/bs] are device copies of mnb_act_order_plan's output.
 * For M > 16 repack packed_out with mnb_repack(packed_out, K', N, block_size, ...).
 * Runs once per weight, so it is refused with MNB_ERR_CAPTURE while `stream` captures.
 */
MNB_API mnb_status mnb_act_order_prepare(mnb_weight w, int K, int N, int block_size, const int32_t *perm,
                                         const int32_t *block_group, int K_prepared, uint8_t *packed_out,
                                         void *scales_out, uint8_t *zero_points_out, mnb_stream stream);

/*
 * A_out[m, k'] = A[m, perm[k']] for m < M, k' < K', and +0 where perm[k'] = -1 (fp16,
 * row-major; A is [M, K], A_out is [M, K']). perm is device int32 [K'] and K' a
 * multiple of 8 no larger than 2K. Any other perm entry writes 0 and sets the index
 * bit of the device status word.
 */
MNB_API mnb_status mnb_act_order_gather(const void *A, int M, int K, const int32_t *perm, int K_prepared,
                                        void *A_out, mnb_stream stream);

/* Workspace bytes mnb_gemm_act_order needs: M * K' * 2 (the gathered activation). */
MNB_API size_t mnb_act_order_workspace_bytes(int M, int K_prepared);

/*
 * Y[M, N] = A[M, K] . dequant_g_idx(B)^T for an act-order weight, with the bias modes of
 * mnb_gemm_bias. `w` and `repacked` are the PREPARED weight (K' columns; `repacked`
 * needed for M > 16 as in mnb_gemm); perm is the device copy of the plan's perm. The call
 * gathers A into `workspace` (at least mnb_act_order_workspace_bytes(M, K') bytes,
 * contents need no initialisation, overwritten by each call) and then runs mnb_gemm's
 * kernel for (M, K', N) on it. A workspace larger by at least
 * mnb_workspace_bytes(M, K', N, block_size), placed after the gathered activation rounded
 * up to 16 bytes, lets 2 <= M <= 16 with K' beyond one shared-memory pass run on the
 * small-M kernel's K slices (without it those calls take the generic kernel). Calls that
 * share one workspace must be ordered on one stream. Tolerance as mnb_gemm, with the bound
 * taken over the g_idx weights.
 */
MNB_API mnb_status mnb_gemm_act_order(const void *A, int M, mnb_weight w, const uint8_t *repacked,
                                      const int32_t *perm, int K, int K_prepared, int N, int block_size,
                                      const void *bias, int bias_mode, void *workspace, size_t ws_bytes,
                                      void *Y, mnb_stream stream);

/*
 * mnb_gemm_act_order without a workspace, for callers that cannot allocate device
 * memory (a plugin inside a host framework that owns all device memory and hands it no
 * workspace, or a loop where cudaMalloc's implicit synchronisation is not allowed). The
 * published MatMulNBits descriptions have no counterpart: this entry point is this
 * library's own.
 * Same arguments and result as mnb_gemm_act_order minus workspace/ws_bytes. The
 * gathered activation (M * K' * 2 bytes) lives in a static device array of 8 MiB
 * (8388608 bytes) inside the library, held on every GPU that loads the library until
 * the process exits; a larger M * K' gives MNB_ERR_UNSUPPORTED. The call allocates
 * nothing. Its first call on a device looks up the array's device address
 * (cudaGetSymbolAddress, with that device current); make that first call before any
 * stream capture. All calls share the one array and it keeps the last call's contents
 * (each call overwrites everything it reads, so nothing needs clearing): calls that
 * may overlap on the GPU (different streams, or threads without ordering) race on it,
 * so order them on one stream.
 */
MNB_API mnb_status mnb_gemm_act_order_noalloc(const void *A, int M, mnb_weight w, const uint8_t *repacked,
                                              const int32_t *perm, int K, int K_prepared, int N,
                                              int block_size, const void *bias, int bias_mode, void *Y,
                                              mnb_stream stream);

/*
 * ---- Paged 4-bit key/value cache and attention ----
 *
 * What a decoder layer needs between its qkv product and its output product, with the
 * cache held in 4 bits as the weights are. The pages have no counterpart: formats and
 * entry points are this library's own.
 *
 * Cache: `pages` holds num_pages x kv_heads records; a record holds the page_size tokens
 * of one page and one key/value head as page_size / 16 blocks of 16 tokens. With
 * D = head_dim (64, 128 or 256), ng = D / group_size (group_size 32, 64 or 128, at most D)
 * a block is 16 D + 128 ng bytes:
 *   K codes  16 rows of D/2 bytes; row r is 32-bit words in the order (t, w), t in 0..3, w in
 *            0..D/32-1; nibble n (bits 4n..4n+3) of word (t, w) is element 32 w + 8 t + n. For
 *            D = 256 the word is stored at w ^ 4 in odd rows.
 *   V codes  words in the order (g, r', w), g in 0..7, r' in 0..15, w in 0..D/64-1; nibble
 *            4 h + n (h in 0..1, n in 0..3) of word (g, r', w) is element 64 w + 32 h + 4 g + n
 *            of row r' ^ x(g), x(g) = 8 (g/2 % 2) for D = 64, 8 (g % 2) for 128, g % 2 for 256.
 *   K, then V parameters: fp16 pairs (scale, offset) in the order (group, row).
 * An element is offset + code * scale (fp32, one rounding). Slot s is row s % 16 of block
 * (s % page_size) / 16 of page s / page_size. The orders are those in which the attention
 * kernel's lanes read a block: whole vectors, no bank conflicts, one bulk copy per block.
 */
typedef struct {
    uint8_t *pages;     /* num_pages * kv_heads * (page_size / 16) blocks, 16-byte aligned   */
    int32_t num_pages;  /* >= 1, and fewer than 2^32 - 1 blocks in all                       */
    int32_t page_size;  /* tokens in a page: a multiple of 16, at most 4096                  */
    int32_t kv_heads;   /* 1 .. 1024                                                         */
    int32_t head_dim;   /* 64, 128 or 256                                                    */
    int32_t group_size; /* 32, 64 or 128, at most head_dim                                   */
} mnb_kv4_cache;

/* Rotation tables: cos and sin are fp32 [rows, rot_dim / 2]; rot_dim is 0 (no rotation, the
 * pointers are not read) or a multiple of 16 up to head_dim: the first rot_dim elements of
 * each head turn, the others stay. Pair i is the elements (i, i + rot_dim / 2), or (2i, 2i + 1)
 * when `interleaved` is not 0. */
typedef struct {
    const float *cos;
    const float *sin;
    int32_t rows;
    int32_t rot_dim;
    int32_t interleaved;
} mnb_rope;

/* Bytes of a cache's `pages` (0 for arguments outside the ranges above). */
MNB_API size_t mnb_kv4_cache_bytes(int num_pages, int page_size, int kv_heads, int head_dim, int group_size);

/*
 * Append T tokens: rotate q and k by their positions, quantise k and v, store them at their
 * slots, write the rotated q.
 * q [T, q_heads, D], k and v [T, kv_heads, D] are of `dtype` (MNB_F16 or MNB_F32); a token's
 * heads lie one after the other and tokens are *_stride elements apart (views of one fused
 * qkv product do), each stride a multiple of 16 bytes (else MNB_ERR_MISALIGNED). q may be
 * NULL (q_heads 0): then q_out is not written. q_out is [T, q_heads, D] of `dtype`, contiguous,
 * and may be q itself where q is contiguous. positions is int32 [T] (not read when rot_dim is 0), slots
 * int64 [T]; the non-negative slots of a call are distinct.
 * Arithmetic, fp32, each operation rounded once and none fused:
 *   a' = a cos - b sin, b' = b cos + a sin; q_out rounds them to dtype, k goes on unrounded.
 *   A group with least element lo and largest hi: offset = fp16(lo) and scale =
 *   fp16((hi - lo) * fp32(1/15)), both held within +-65504; code = rint((x - offset) * (1 / scale)) within
 *   0..15, and 0 where scale is 0. A group with an inf or NaN element holds NaN.
 * A negative slot: the token is not stored (padding), its q is still written. A slot beyond
 * the cache: not stored. A position outside 0..rows-1: not stored, and its q_out row is 0.
 * The last two set the index bit of the device status word. T = 0 is valid and does nothing.
 */
MNB_API mnb_status mnb_kv4_append(const void *q, const void *k, const void *v, int dtype, int T, int q_heads,
                                  int64_t q_stride, int64_t k_stride, int64_t v_stride, const int32_t *positions,
                                  mnb_rope rope, const int64_t *slots, mnb_kv4_cache cache, void *q_out,
                                  mnb_stream stream);

/*
 * The values that T slots hold: k_out and v_out [T, kv_heads, D] of `dtype`, element
 * offset + code * scale in fp32, rounded once more for MNB_F16. A negative slot reads as
 * zeros; one beyond the cache too, and it sets the index bit of the device status word.
 */
MNB_API mnb_status mnb_kv4_read(mnb_kv4_cache cache, const int64_t *slots, int T, int dtype, void *k_out,
                                void *v_out, mnb_stream stream);

/*
 * Scratch bytes of mnb_kv4_attention for these shapes (0 for arguments outside its ranges).
 * The size covers GPUs of up to 160 SMs; contents need no initialisation, each call
 * overwrites them, so calls sharing one workspace must be ordered on one stream (from any host
 * threads: a call's launches are issued together).
 */
MNB_API size_t mnb_kv4_attention_workspace_bytes(int T, int batch, int q_heads, int kv_heads, int head_dim,
                                                 int dtype);

/*
 * Attention of T query tokens of `batch` sequences over the cache, one token a sequence
 * (decode), a few (speculative verify) or many (prefill). Sequence b has the query tokens
 * q_start[b] .. q_start[b+1]-1 (int32 [batch + 1], not decreasing, from 0 to T) and kv_len[b]
 * keys (int32 [batch], its query tokens' own included): key j is in page
 * page_table[b * table_stride + j / page_size] (int32). Query token i of n is at position
 * kv_len[b] - n + i; it sees the keys j of 0..kv_len[b]-1 with, if `causal`, j <= its position
 * and, if window > 0, j > its position - window. Query head h reads key/value head
 * h / (q_heads / kv_heads); q_heads is a multiple of kv_heads.
 *   out[i, h] = sum_j softmax_j(scale * q[i, h] . k_j) v_j;  lse[i, h] = log sum_j e^(scale * q . k_j)
 * (natural log; lse may be NULL). A token that sees no key gets out = 0 and lse = -inf.
 * q [T, q_heads, D] of `dtype`, tokens q_stride elements apart (a multiple of 16 bytes); out
 * [T, q_heads, D] of `dtype`, contiguous; lse fp32 [T, q_heads]. Sums and softmax statistics are fp32.
 * MNB_F16: the probabilities, and with many rows the held keys and values too, enter the products rounded to fp16 (error, as
 * a norm, 2.4e-4 to 4.4e-4, of which the result's own rounding is 2.1e-4); MNB_F32: to 22 bits (3e-7).
 * A page index outside the cache: its keys are left out; a kv_len beyond
 * table_stride * page_size: cut to it. Both set the index bit of the device status word.
 * Rows of q_start's range are clamped to 0..T. Launch geometry depends on the shape
 * arguments alone: the lengths are read on the device, so a captured call follows them.
 */
MNB_API mnb_status mnb_kv4_attention(const void *q, int dtype, int T, int q_heads, int64_t q_stride,
                                     mnb_kv4_cache cache, const int32_t *q_start, const int32_t *kv_len,
                                     const int32_t *page_table, int batch, int table_stride, float scale,
                                     int causal, int window, void *workspace, size_t ws_bytes, void *out,
                                     float *lse, mnb_stream stream);

/*
 * ---- What each request of a shared step has of its own ----
 *
 * Requests that share the 4-bit products of a decode, verify or prefill step may each have a low-rank adapter, a
 * temperature and drafted tokens. The pages have no counterpart: these entry points are this library's own.
 */

/* Low-rank adapters of one layer, in one pool: adapter i is down[i] (fp16 [max_rank, K]) and up[i] (fp16 [N, max_rank]), of
 * which the first ranks[i] rows of down and columns of up count (the rest is not used, whatever it holds). */
typedef struct {
    const void *down;      /* fp16 [count, max_rank, K]                                  */
    const void *up;        /* fp16 [count, N, max_rank]                                  */
    const int32_t *ranks;  /* int32 [count], held to 0..max_rank; NULL: all max_rank      */
    const float *scales;   /* fp32 [count]; NULL: 1                                      */
    int32_t count;         /* 1 .. 2^20                                                  */
    int32_t max_rank;      /* a multiple of 8 in 8 .. 128                                */
} mnb_lora_pool;

/*
 * out[m] = base[m] + scales[a] * up[a] . (down[a] . x[m]), a = adapter[m], for M rows of any adapters in any order (rows of one
 * adapter that lie near each other share its loads). Beside a product of this section's kind, base is that product's Y.
 * x [M, K], base and out [M, N] are of `dtype` (MNB_F16 or MNB_F32), rows *_stride elements apart (views of one fused
 * product do); x_stride is a multiple of 16 bytes (else MNB_ERR_MISALIGNED), K of 16 elements. base may be out
 * (with the same stride; neither it nor x may overlap out otherwise) or NULL, which counts as zeros. adapter is int32 [M]: a
 * negative one leaves out[m] = base[m], and so does one beyond the pool, which sets the index bit of the device status word.
 * Products and sums are fp32. down . x enters the second product with 22 bits, relative to the row's largest, and with MNB_F32 x the
 * first one, relative to the largest of 32 neighbours. A row of x with inf or NaN gives non-finite outputs in that row.
 * `workspace` holds mnb_lora_workspace_bytes(M) bytes (0 up to 256 rows); its contents need no initialisation and are overwritten by
 * each call, so calls sharing one workspace must be ordered on one stream (from any host threads). M = 0 is valid and does
 * nothing.
 */
MNB_API size_t mnb_lora_workspace_bytes(int M);
MNB_API mnb_status mnb_lora(const void *x, int dtype, int M, int K, int64_t x_stride, mnb_lora_pool pool,
                            const int32_t *adapter, const void *base, int64_t base_stride, int N, void *workspace,
                            size_t ws_bytes, void *out, int64_t out_stride, mnb_stream stream);

/*
 * Probabilities: out[r, j] = e^((x[r, j] - max_j x) / temperature[r]) / sum_j, fp32 [rows, V], contiguous. logits x [rows, V]
 * are of `dtype` (MNB_F16 or MNB_F32), rows `stride` elements apart; out may be logits (MNB_F32, stride V), and may not overlap
 * them otherwise. temperature is fp32 [rows], NULL for 1; a row of
 * temperature 0 gets 1 at its largest logit (the first of equal ones) and 0 elsewhere, one of an infinite temperature the same for all finite ones. Masked logits are -inf: a row of
 * nothing else gets zeros. A NaN or (unless the temperature is 0) +inf logit, and a temperature that is negative or NaN, make the row
 * NaN. `workspace` holds mnb_softmax_workspace_bytes(rows, V) bytes (0 for V up to 16377, and for few
 * rows), under the rules of mnb_lora's; more than 2^42 elements give MNB_ERR_UNSUPPORTED. rows = 0 is valid and does nothing.
 */
MNB_API size_t mnb_softmax_workspace_bytes(int rows, int V);
MNB_API mnb_status mnb_softmax(const void *logits, int dtype, int rows, int V, int64_t stride, const float *temperature,
                               void *workspace, size_t ws_bytes, float *out, mnb_stream stream);

/*
 * Verification of drafted tokens from given random numbers (speculative sampling). Sequence b of `batch` has the drafted tokens
 * draft_start[b] .. draft_start[b+1]-1 of draft_tokens (int32 [drafted]; draft_start int32 [batch + 1], not decreasing,
 * from 0 to drafted or, where a batch is padded, below it; there may be none). target holds drafted + batch rows of V fp32
 * probabilities, rows target_stride elements apart: token i of sequence b has row draft_start[b] + b + i, and one more row
 * follows after the sequence's last; what lies behind the last sequence is neither used nor written. draft holds `drafted` rows, those that the tokens were drawn from; NULL: each is 1 at its token.
 *   Token d_i is accepted while u_accept[.] * q_i(d_i) < p_i(d_i). The token after the last accepted one is the first j with
 *   sum_{k <= j} w_k > u_next[b] * sum_k w_k, w = max(p - q, 0) at the rejected token's rows, w = p of the last row
 *   when all are accepted. Where nothing is left of p - q it is drawn from p; where p is all 0, it is -1.
 * u_accept fp32 [drafted], u_next fp32 [batch], in [0, 1) (others are held to 0 .. 1 - 2^-24, NaN counts as 0). tokens int32 [drafted + batch], laid out as
 * target's rows: a sequence's accepted tokens, the next one, then -1. accepted int32 [batch]: how many were accepted.
 * Arithmetic is exact: probabilities are held to 0..1 (NaN counts as 0) and rounded to whole numbers of 2^-60, in which weights and
 * sums are taken (a row adds up to less than 16). A drafted token outside 0..V-1 is rejected and sets the index bit of the
 * device status word. No output may overlap an input.
 * `workspace` holds mnb_verify_workspace_bytes(batch, V) bytes (0 for few sequences), under the rules of mnb_lora's; more than
 * 2^42 elements in the batch's rows give MNB_ERR_UNSUPPORTED. batch = 0 is valid and does nothing.
 */
MNB_API size_t mnb_verify_workspace_bytes(int batch, int V);
MNB_API mnb_status mnb_verify(const float *target, int64_t target_stride, const float *draft, int64_t draft_stride,
                              const int32_t *draft_tokens, const int32_t *draft_start, const float *u_accept,
                              const float *u_next, int batch, int drafted, int V, void *workspace, size_t ws_bytes,
                              int32_t *tokens, int32_t *accepted, mnb_stream stream);

/*
 * Programmatic dependent launch. With `enable` != 0, later calls on this host thread
 * launch their kernels with programmatic stream serialisation: a kernel may start while
 * the previous kernel on the stream is still running, and it streams its weight, scale
 * and zero-point buffers (and an act-order perm) before waiting for that kernel to
 * finish; it reads A and writes Y only after the wait. Enable it only when no earlier
 * work on the stream writes those buffers (weights that stay constant during
 * inference). Default: off.
 */
MNB_API void mnb_set_programmatic_launch(int enable);

/*
 * Reads and clears the device status word. Kernels that wait on shared-memory barriers
 * bound every wait; one that gives up sets a bit in this word, writes NaN outputs and
 * returns instead of hanging. The act-order, key/value cache, adapter and verification kernels set another bit for
 * an index input out of range. Returns MNB_ERR_TIMEOUT (with the bits in the message) if a wait gave
 * up, MNB_ERR_INVALID_ARG if only the index bit is set, else MNB_OK. Synchronises the
 * current device, so it must not be called while a stream is being captured.
 */
MNB_API mnb_status mnb_check_device_status(void);

/*
 * Self-test of the failure path above (no counterpart on the pages; the bounded waits are
 * this library's own): launches one kernel on `stream` whose bounded wait on a
 * shared-memory barrier that nothing ever arrives on gives up after `limit_us`
 * microseconds (1 .. 1000000, else MNB_ERR_INVALID_ARG), sets the wait bit of the device
 * status word and returns. Nothing faults and the context stays usable; the next
 * mnb_check_device_status returns MNB_ERR_TIMEOUT and clears the word. For tests.
 */
MNB_API mnb_status mnb_selftest_wait_timeout(unsigned int limit_us, mnb_stream stream);

/* Message of the last failed call on this host thread ("" if none). */
MNB_API const char *mnb_last_error(void);

/* Name of the kernel variant the last successful call on this host thread launched. */
MNB_API const char *mnb_last_variant(void);

/* Library version string. */
MNB_API const char *mnb_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MNB_H_ */
