// Host-side declarations shared by the mnb translation units (not part of the C ABI).
#pragma once

#include <cuda_runtime.h>
#include <atomic>
#include <stddef.h>
#include <stdint.h>

namespace mnb {

struct QWeight {
  const uint8_t* packed;
  const void* scales;
  const uint8_t* zp;
  int scales_f16;  // 1: fp16 scales, 0: fp32
};

struct LaunchCtx {
  cudaStream_t stream;
  bool pdl;         // launch with programmatic stream serialisation
  int num_sms;
  int device = 0;
  uint32_t* status = nullptr;     // device status word for bounded waits
  const void* bias = nullptr;     // fp16 [N] or null
  int bias_mode = 0;              // 0 none, 1 fp16(acc + b), 2 fp16(fp16(acc) + b)
  const char* variant = nullptr;  // set by the launcher that ran
};

// Each launcher returns cudaSuccess or the launch error.  Shapes are validated by the
// caller (api.cu).
cudaError_t launch_dequant(LaunchCtx& ctx, const QWeight& w, int K, int N, int bs, float* out);
cudaError_t launch_repack(LaunchCtx& ctx, const uint8_t* packed, int K, int N, uint8_t* out);
// Act-order (g_idx): per-k-group dequant, one-time preparation, per-call activation gather.
cudaError_t launch_dequant_gidx(LaunchCtx& ctx, const QWeight& w, const int32_t* gidx, int K, int N, int bs,
                                float* out);
cudaError_t launch_act_order_prepare(LaunchCtx& ctx, const QWeight& w, int K, int N, int bs, const int32_t* perm,
                                     const int32_t* bgroup, int Kp, uint8_t* packed_out, void* scales_out,
                                     uint8_t* zp_out);
cudaError_t launch_act_order_gather(LaunchCtx& ctx, const void* A, int M, int K, const int32_t* perm, int Kp,
                                    void* out);
// M = 1 act-order GEMV with the gather fused into the activation load (one chunk per lane:
// K' <= 8192); cudaErrorNotSupported otherwise.
cudaError_t launch_gemv_tma_gather(LaunchCtx& ctx, const void* A, const int32_t* perm, int Ka, const QWeight& w,
                                   int Kp, int N, int bs, void* Y);
// The driver's cuTensorMapEncodeTiled (CUDA 12 ABI), or null when unavailable.
void* tensor_map_encode_fn();
// Bulk-copy ring GEMV (M = 1); cudaErrorNotSupported when rows are not 16-byte multiples.
cudaError_t launch_gemv_tma(LaunchCtx& ctx, const void* A, const QWeight& w, int K, int N, int bs,
                            void* Y);
cudaError_t launch_gemv_pair_swiglu_tma(LaunchCtx& ctx, const void* A, const QWeight& gate,
                                        const QWeight& up, int K, int N, int bs, void* out);
// M = 1 GEMV with the multiply-accumulate on mma.sync tensor cores (K % 256 == 0, block
// size 32/64/128); cudaErrorNotSupported for other shapes.
cudaError_t launch_gemv_mma(LaunchCtx& ctx, const void* A, const QWeight& w, int K, int N, int bs, void* Y);
cudaError_t launch_gemv_pair_swiglu_mma(LaunchCtx& ctx, const void* A, const QWeight& gate, const QWeight& up,
                                        int K, int N, int bs, void* out);
// 2 <= M <= 2 * (bs / 32) (block sizes 32 and 64, K % 256 == 0, M * K * 2 <= 32 KB) on the
// M = 1 kernel's machinery with the row mapping; cudaErrorNotSupported otherwise.
cudaError_t launch_gemm_rows_mma(LaunchCtx& ctx, const void* A, int M, const QWeight& w, int K, int N, int bs,
                                 void* Y);
// One-thread kernel whose bounded wait on a never-armed mbarrier gives up after limit_ns.
cudaError_t launch_wait_selftest(LaunchCtx& ctx, uint64_t limit_ns);
// Register-pipelined M = 1 GEMV; cudaErrorNotSupported when the shape has no variant.
cudaError_t launch_gemv(LaunchCtx& ctx, const void* A, const QWeight& w, int K, int N, int bs,
                        void* Y);
cudaError_t launch_gemv_pair_swiglu(LaunchCtx& ctx, const void* A, const QWeight& gate,
                                    const QWeight& up, int K, int N, int bs, void* out);
// 2 <= M <= 16 (block size >= 32): weights streamed once, mma.sync over M rows.  For K
// beyond one shared-memory pass the K range is split into slices whose fp32 partials go to
// `workspace` (smallm_workspace_bytes of it) and are summed in slice order.
cudaError_t launch_gemm_smallm(LaunchCtx& ctx, const void* A, int M, const QWeight& w, int K, int N, int bs,
                               void* Y, void* workspace, size_t ws_bytes);
int smallm_kslice(int M, int K, int bs, int ssz, bool zp);
size_t smallm_workspace_bytes(int M, int K, int N, int bs);
// M > 16 on the tcgen05 tensor cores, reading the repacked operand.  With a workspace of
// at least gemm_tc_workspace_bytes (the sizing for up to 160 SMs), shapes with fewer
// output tiles than half the SMs split K into slices of whole quant groups and sum their
// fp32 partials in slice order; without one they run unsplit.
cudaError_t launch_gemm_tc(LaunchCtx& ctx, const void* A, int M, const QWeight& w,
                           const uint8_t* repacked, int K, int N, int bs, void* Y, void* workspace = nullptr,
                           size_t ws_bytes = 0);
size_t gemm_tc_workspace_bytes(int M_rows, int K, int N, int bs);
// fp32 activations.  M = 1: bulk-copy GEMV with fp32 activations (K <= 16384).  M >= 2:
// rows split into fp16 hi/lo pairs (A2 holds 2M rows, rexp M exponents), then the small-M
// kernel (2M <= 16) or the tcgen05 kernel with the pair-summing fp32 epilogue.  The generic
// fp32 kernel takes any shape.
cudaError_t launch_gemv_f32_tma(LaunchCtx& ctx, const float* A, const QWeight& w, int K, int N, int bs,
                                float* Y, const float* bias);
cudaError_t launch_split_f32(LaunchCtx& ctx, const float* A, int M, int K, void* A2, int* rexp);
// Fixed-order sums of K-slice partials part[slice][rows][N]: fp16 Y with ctx's bias mode,
// or fp32 Yf from hi/lo row pairs with their exponents (split fp32 activations).
cudaError_t launch_combine_slices(LaunchCtx& ctx, const float* part, int nslices, int M, int N, void* Y);
cudaError_t launch_combine_slices_f32(LaunchCtx& ctx, const float* part, int nslices, int Mout, int N, float* Yf,
                                      const float* biasf, const int* rexp);
cudaError_t launch_gemm_smallm_f32split(LaunchCtx& ctx, const void* A2, int M, const QWeight& w, int K, int N,
                                        int bs, float* Y, const float* bias, const int* rexp,
                                        void* workspace = nullptr, size_t ws_bytes = 0);
cudaError_t launch_gemm_tc_f32split(LaunchCtx& ctx, const void* A2, int M, const QWeight& w,
                                    const uint8_t* repacked, int K, int N, int bs, float* Y, const float* bias,
                                    const int* rexp, void* workspace = nullptr, size_t ws_bytes = 0);
cudaError_t launch_generic_f32(LaunchCtx& ctx, const float* A, int M, const QWeight& w, int K, int N, int bs,
                               float* Y, const float* bias);
// Any M, any K % 16 == 0: CUDA-core kernel, fp32 arithmetic.
cudaError_t launch_generic(LaunchCtx& ctx, const void* A, int M, const QWeight& w, int K, int N,
                           int bs, void* Y);
cudaError_t launch_generic_pair_swiglu(LaunchCtx& ctx, const void* A, const QWeight& gate,
                                       const QWeight& up, int K, int N, int bs, void* out);

// Paged 4-bit key/value cache (mnb.h): geometry of a cache and of its 16-token blocks.
struct Kv4Cache {
  uint8_t* pages;
  int num_pages, page_size, kv_heads, head_dim, group;
  // derived once on the host: kernels would divide for them
  int groups, block_size, page_blocks;
  Kv4Cache() = default;
  Kv4Cache(uint8_t* pages_, int num_pages_, int page_size_, int kv_heads_, int head_dim_, int group_)
      : pages(pages_), num_pages(num_pages_), page_size(page_size_), kv_heads(kv_heads_), head_dim(head_dim_), group(group_),
        groups(head_dim_ / group_), block_size(16 * head_dim_ + 128 * (head_dim_ / group_)), page_blocks(page_size_ / 16) {}
  __host__ __device__ int ng() const { return groups; }
  __host__ __device__ int block_bytes() const { return block_size; }
  __host__ __device__ int64_t head_bytes() const { return (int64_t)page_blocks * block_size; }  // of a page's key head
};
struct Kv4Append {
  const void *q, *k, *v;
  int f32, T, q_heads;
  int64_t q_stride, k_stride, v_stride;
  const int32_t* positions;
  const float *cos, *sin;
  int rows, rot, interleaved;
  const int64_t* slots;
  void* q_out;
};
struct Kv4Attention {
  const void* q;
  int f32, T, q_heads;
  int64_t q_stride;
  const int32_t *q_start, *kv_len, *page_table;
  int batch, table_stride;
  float scale;
  int causal, window;
  void* workspace;
  size_t ws_bytes;
  void* out;
  float* lse;
};
cudaError_t launch_kv4_append(LaunchCtx& ctx, const Kv4Cache& c, const Kv4Append& a);
cudaError_t launch_kv4_read(LaunchCtx& ctx, const Kv4Cache& c, const int64_t* slots, int T, int f32, void* k_out,
                            void* v_out);
cudaError_t launch_kv4_attention(LaunchCtx& ctx, const Kv4Cache& c, const Kv4Attention& a);
size_t kv4_attention_workspace_bytes(int T, int batch, int q_heads, int kv_heads, int head_dim, int f32);

// Low-rank adapters beside a product (mnb.h).
struct Lora {
  const void* x;
  int f32, M, K;
  int64_t x_stride;
  const void *down, *up;
  const int32_t* ranks;
  const float* scales;
  int count, max_rank;
  const int32_t* adapter;
  const void* base;
  int64_t base_stride;
  int N;
  void* out;
  int64_t out_stride;
  void* workspace;
};
cudaError_t launch_lora(LaunchCtx& ctx, const Lora& a);
size_t lora_workspace_bytes(int M);

// Probabilities and verification of drafted tokens (mnb.h).
struct Softmax {
  const void* logits;
  int f32, rows, V;
  int64_t stride;
  const float* temperature;
  float* out;
  void* workspace;
};
struct Verify {
  const float* target;
  int64_t target_stride;
  const float* draft;
  int64_t draft_stride;
  const int32_t *tokens, *start;
  const float *u_accept, *u_next;
  int batch, drafted, V;
  int32_t *out, *accepted;
  void* workspace;
};
cudaError_t launch_softmax(LaunchCtx& ctx, const Softmax& a);
cudaError_t launch_verify(LaunchCtx& ctx, const Verify& a);
size_t softmax_workspace_bytes(int rows, int V);
size_t verify_workspace_bytes(int batch, int V);

// cudaFuncSetAttribute(MaxDynamicSharedMemorySize) once per kernel and device: `done` is a static of the caller,
// a bit for each device.
template <typename Kern>
cudaError_t allow_smem(Kern kernel, int bytes, int device, std::atomic<uint64_t>& done) {
  const uint64_t bit = device < 64 ? 1ull << device : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Launch helper: cudaLaunchKernelEx with the programmatic-serialisation attribute when
// ctx.pdl is set.
template <typename Kern, typename... Args>
cudaError_t launch_kernel(LaunchCtx& ctx, Kern kernel, dim3 grid, dim3 block, size_t smem,
                          Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = ctx.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctx.pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The same for a grid of thread-block clusters of `cluster` CTAs.  Sizes above 8 need the kernel's
// NonPortableClusterSizeAllowed attribute (allow_wide_clusters).
template <typename Kern, typename... Args>
cudaError_t launch_clusters(LaunchCtx& ctx, Kern kernel, int cluster, dim3 grid, dim3 block, size_t smem, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = ctx.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctx.pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename Kern>
cudaError_t allow_wide_clusters(Kern kernel, int device, std::atomic<uint64_t>& done) {
  const uint64_t bit = device < 64 ? 1ull << device : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Clusters of this kernel that the GPU holds at a time, asked for once a device: `known` is a static of the caller. 0: it holds none, or
// could not tell, which is asked again and leaves no error behind for the launches that follow.
template <typename Kern>
int clusters_held(const LaunchCtx& ctx, Kern kernel, int cluster, int threads, size_t smem, std::atomic<int> (&known)[64]) {
  int n = ctx.device < 64 ? known[ctx.device].load(std::memory_order_relaxed) : 0;
  if (n != 0) return n - 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cluster);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
    (void)cudaGetLastError();
    return 0;
  }
  if (ctx.device < 64) known[ctx.device].store(n + 1, std::memory_order_relaxed);
  return n;
}

}  // namespace mnb
