// From logits to verified tokens: probabilities at each row's temperature, and the verification of drafted tokens from
// given random numbers.
#include <float.h>

#include "cluster.cuh"
#include "mnb_device.cuh"
#include "mnb_internal.h"

namespace mnb {
namespace {

// ---------------------------------------------------------------------------------
// Softmax: p = e^((x - max) / temperature) / sum.  A cluster has a row, its CTAs a part each.
// ---------------------------------------------------------------------------------
constexpr int kSoftThreads = 512;

struct MaxSum {
  float m, s;
};

template <bool F32>
__device__ __forceinline__ float logit(const void* row, int j) {
  if constexpr (F32) return static_cast<const float*>(row)[j];
  else return __half2float(static_cast<const __half*>(row)[j]);
}

__device__ __forceinline__ float nan_max(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <bool F32>
__global__ void __launch_bounds__(kSoftThreads) softmax_kernel(const Softmax a, int cluster) {
  __shared__ float red[kSoftThreads / 32];
  __shared__ int red_at[kSoftThreads / 32];
  __shared__ float2 mine;
  __shared__ int mine_at;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int part = cluster_ctarank(), r = blockIdx.x / cluster;
  pdl_launch_dependents();
  pdl_wait();
  const void* row = static_cast<const uint8_t*>(a.logits) + (int64_t)r * a.stride * (F32 ? 4 : 2);
  float* out = a.out + (int64_t)r * a.V;
  const int j0 = (int)((int64_t)a.V * part / cluster), j1 = (int)((int64_t)a.V * (part + 1) / cluster);
  const float temp = a.temperature ? a.temperature[r] : 1.0f;
  // ---- the largest, and the first place that has it ----
  float m = -INFINITY;
  int at = 0x7fffffff;
  for (int j = j0 + tid; j < j1; j += kSoftThreads) {
    const float x = logit<F32>(row, j);
    if (x > m) at = j;
    m = nan_max(m, x);
  }
  float top = m;
  for (int o = 16; o; o >>= 1) top = nan_max(top, __shfl_xor_sync(kFull, top, o));
  if (m != top) at = 0x7fffffff;
  for (int o = 16; o; o >>= 1) at = min(at, __shfl_xor_sync(kFull, at, o));
  if (lane == 0) red[warp] = top, red_at[warp] = at;
  __syncthreads();
  top = red[0];
  for (int w = 1; w < kSoftThreads / 32; ++w) top = nan_max(top, red[w]);
  at = 0x7fffffff;
  for (int w = 0; w < kSoftThreads / 32; ++w)
    if (red[w] == top) at = min(at, red_at[w]);
  __syncthreads();
  const float inv_t = temp > 0.0f ? fminf(1.0f / temp, FLT_MAX) : temp == 0.0f ? 1.0f : NAN;
  float sum = 0.0f;
  if (top != -INFINITY)
    for (int j = j0 + tid; j < j1; j += kSoftThreads) sum += expf((logit<F32>(row, j) - top) * inv_t);
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  if (lane == 0) red[warp] = sum;
  __syncthreads();
  if (tid == 0) {
    sum = 0.0f;
    for (int w = 0; w < kSoftThreads / 32; ++w) sum += red[w];
    mine = make_float2(top, sum);
    mine_at = at;
  }
  // ---- over the cluster ----
  cluster_arrive();
  cluster_wait();
  float all_top = -INFINITY;
  for (int c = 0; c < cluster; ++c) all_top = nan_max(all_top, cluster_ld_f2(cluster_map(smem_u32(&mine), c)).x);
  float all = 0.0f;
  int first = 0x7fffffff;
  for (int c = 0; c < cluster; ++c) {
    const float2 v = cluster_ld_f2(cluster_map(smem_u32(&mine), c));
    if (v.x != -INFINITY) all += v.y * expf((v.x - all_top) * inv_t);
    int f;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(f) : "r"(cluster_map(smem_u32(&mine_at), c)));
    if (v.x == all_top) first = min(first, f);
  }
  cluster_arrive();
  const bool none = all_top == -INFINITY;  // no logit above -inf
  const float inv = none ? 0.0f : 1.0f / all;
  for (int j = j0 + tid; j < j1; j += kSoftThreads) {
    float p;
    if (temp == 0.0f) p = all_top != all_top ? NAN : j == first ? 1.0f : 0.0f;
    else p = none ? 0.0f : expf((logit<F32>(row, j) - all_top) * inv_t) * inv;
    out[j] = p;
  }
  cluster_wait();
}

// ---------------------------------------------------------------------------------
// Verification.  A cluster has a sequence.  Every warp finds the first rejected token by itself; then the warps of the
// cluster share the row to draw from.
//
// Weights are whole numbers of 2^-60 (probabilities are held to 0..1; what is below 2^-60 counts as 0): sums are exact in any
// order, and the drawn token does not hang on how the row was cut. A row may add up to just below 16.
// ---------------------------------------------------------------------------------
constexpr int kVerifyWarps = 8;

__device__ __forceinline__ uint64_t fixed60(float p) {
  const uint32_t b = __float_as_uint(__saturatef(p));  // NaN: 0
  const uint64_t m = (uint64_t)((b & 0x7fffffu) | 0x800000u) << 37;
  uint64_t r;
  asm("shr.u64 %0, %1, %2;" : "=l"(r) : "l"(m), "r"(127u - (b >> 23)));  // shifts of 64 and more give 0
  return r;
}
__device__ __forceinline__ uint64_t sub_clamped(uint64_t a, uint64_t b) { return a > b ? a - b : 0; }

// floor(total * u), u in [0, 1)
__device__ __forceinline__ uint64_t scaled(uint64_t total, float u) {
  const uint32_t b = min(__float_as_uint(__saturatef(u)), 0x3f7fffffu);
  const uint64_t m = b >> 23 ? (b & 0x7fffffu) | 0x800000u : b & 0x7fffffu;
  const int s = 150 - (int)max(b >> 23, 1u);  // u = m * 2^-s, s >= 24
  const uint64_t hi = __umul64hi(total, m), lo = total * m;
  return s < 64 ? hi << (64 - s) | lo >> s : s < 128 ? hi >> (s - 64) : 0;
}

__device__ __forceinline__ uint64_t shfl_up_u64(uint64_t v, int o) { return __shfl_up_sync(kFull, (unsigned long long)v, o); }
__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, (unsigned long long)v, o);
  return v;
}

__global__ void __launch_bounds__(kVerifyWarps * 32) verify_kernel(const Verify a, int cluster, uint32_t* status) {
  __shared__ uint64_t sums[2][kVerifyWarps];
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int part = cluster_ctarank(), b = blockIdx.x / cluster;
  pdl_launch_dependents();
  pdl_wait();
  const int s0 = min(max(a.start[b], 0), a.drafted), s1 = min(max(a.start[b + 1], s0), a.drafted), n = s1 - s0;
  // ---- the first rejected token ----
  int accepted = n;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int i = i0 + lane;
    bool bad = false;
    if (i < n) {
      const int tok = a.tokens[s0 + i];
      bad = true;
      if (tok >= 0 && tok < a.V) {
        const float pt = __saturatef(a.target[(int64_t)(s0 + b + i) * a.target_stride + tok]);
        const float qt = a.draft ? __saturatef(a.draft[(int64_t)(s0 + i) * a.draft_stride + tok]) : 1.0f;
        bad = !((double)__saturatef(a.u_accept[s0 + i]) * (double)qt < (double)pt);
      } else if (part == 0 && warp == 0) {
        report_status(status, kStatusBadIndex);
      }
    }
    const uint32_t vote = __ballot_sync(kFull, bad);
    if (vote) {
      accepted = i0 + __ffs(vote) - 1;
      break;
    }
  }
  const bool rejected = accepted < n;
  const float* p = a.target + (int64_t)(s0 + b + accepted) * a.target_stride;
  const float* q = rejected && a.draft ? a.draft + (int64_t)(s0 + accepted) * a.draft_stride : nullptr;
  const int not_this = rejected && !a.draft ? a.tokens[s0 + accepted] : -1;
  // ---- sums of this warp's part of the row ----
  const int parts = cluster * kVerifyWarps, own = part * kVerifyWarps + warp;
  const int len = ((a.V + parts - 1) / parts + 127) / 128 * 128;
  const int j0 = (int)min((int64_t)own * len, (int64_t)a.V), j1 = min(j0 + len, a.V);
  auto weight = [&](int j, bool residual) -> uint64_t {
    const uint64_t f = fixed60(p[j]);
    if (!residual) return f;
    if (q) return sub_clamped(f, fixed60(q[j]));
    return j == not_this ? 0 : f;
  };
  uint64_t sum_w = 0, sum_p = 0;
  for (int j = j0 + lane; j < j1; j += 32) {
    sum_p += weight(j, false);
    if (rejected) sum_w += weight(j, true);
  }
  sum_p = warp_sum(sum_p), sum_w = warp_sum(sum_w);
  if (lane == 0) sums[0][warp] = sum_w, sums[1][warp] = sum_p;
  cluster_arrive();
  cluster_wait();
  // ---- all parts' sums; the part that the drawn one is in ----
  uint64_t total[2] = {0, 0}, before[2] = {0, 0};
  for (int i = lane; i < parts; i += 32) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint64_t v = cluster_ld_u64(cluster_map(smem_u32(&sums[k][i % kVerifyWarps]), i / kVerifyWarps));
      total[k] += v;
      if (i < own) before[k] += v;
    }
  }
  cluster_arrive();
#pragma unroll
  for (int k = 0; k < 2; ++k) total[k] = warp_sum(total[k]), before[k] = warp_sum(before[k]);
  const bool residual = rejected && total[0] > 0;  // nothing left of p - q: drawn from p
  const uint64_t all = residual ? total[0] : total[1], head = residual ? before[0] : before[1];
  const uint64_t here = residual ? sum_w : sum_p;
  const uint64_t limit = scaled(all, a.u_next[b]);
  const int64_t at = (int64_t)s0 + b;
  if (all > 0 && head <= limit && head + here > limit) {
    uint64_t run = head;
    for (int j = j0; j < j1; j += 32) {
      const uint64_t w = j + lane < j1 ? weight(j + lane, residual) : 0;
      uint64_t inc = w;
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t v = shfl_up_u64(inc, o);
        if (lane >= o) inc += v;
      }
      const uint32_t past = __ballot_sync(kFull, run + inc > limit);
      if (past) {
        if (lane == 0) a.out[at + accepted] = j + __ffs(past) - 1;
        break;
      }
      run += __shfl_sync(kFull, (unsigned long long)inc, 31);
    }
  }
  if (own == 0) {
    if (lane == 0) {
      a.accepted[b] = accepted;
      if (all == 0) a.out[at + accepted] = -1;
    }
    for (int i = lane; i <= n; i += 32)
      if (i != accepted) a.out[at + i] = i < accepted ? a.tokens[s0 + i] : -1;
  }
  cluster_wait();
}

// CTAs of a cluster: enough of them for every SM, parts of at least `least` elements.
int cluster_for(int rows, int V, int least, int num_sms) {
  int c = 16;
  while (c > 1 && ((int64_t)rows * (c / 2) >= 2 * num_sms || V / c < least)) c /= 2;
  return c;
}

}  // namespace

cudaError_t launch_softmax(LaunchCtx& ctx, const Softmax& a) {
  const int c = cluster_for(a.rows, a.V, 2048, ctx.num_sms);
  ctx.variant = a.f32 ? "softmax_f32" : "softmax_f16";
  auto go = [&](auto kern, std::atomic<uint64_t>& wide) {
    const cudaError_t e = c > 8 ? allow_wide_clusters(kern, ctx.device, wide) : cudaSuccess;
    return e != cudaSuccess ? e : launch_clusters(ctx, kern, c, dim3((unsigned)a.rows * c), dim3(kSoftThreads), 0, a, c);
  };
  static std::atomic<uint64_t> wide[2];
  return a.f32 ? go(softmax_kernel<true>, wide[1]) : go(softmax_kernel<false>, wide[0]);
}

cudaError_t launch_verify(LaunchCtx& ctx, const Verify& a) {
  const int c = cluster_for(a.batch, a.V, 1024, ctx.num_sms);
  ctx.variant = "verify";
  static std::atomic<uint64_t> wide{0};
  const cudaError_t e = c > 8 ? allow_wide_clusters(verify_kernel, ctx.device, wide) : cudaSuccess;
  if (e != cudaSuccess) return e;
  return launch_clusters(ctx, verify_kernel, c, dim3((unsigned)a.batch * c), dim3(kVerifyWarps * 32), 0, a, c, ctx.status);
}

}  // namespace mnb
