// From logits to verified tokens: probabilities at each row's temperature, and the verification of drafted tokens from
// given random numbers.
#include <float.h>

#include "cluster.cuh"
#include "mnb_device.cuh"
#include "mnb_internal.h"

namespace mnb {
namespace {

// ---------------------------------------------------------------------------------
// Softmax: p = e^((x - max) / temperature) / sum.  A cluster has a row, its CTAs a part each: read once, kept in registers
// (parts of up to 32 elements a thread; of rows beyond 16 such parts, read three times), largest and sum of the parts exchanged once.
// Elements go in chunks of 8 that begin at 16-byte boundaries of the logits, whatever the row's own start.
// ---------------------------------------------------------------------------------
constexpr int kHeld = 4;  // chunks that a thread keeps

__device__ __forceinline__ float nan_max(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float2 half2_floats(uint32_t u) { return __half22float2(*reinterpret_cast<const __half2*>(&u)); }

template <bool F32, int kThreads, bool kHold>
__global__ void __launch_bounds__(kThreads) softmax_kernel(const Softmax a, int cluster) {
  constexpr int kWarps = kThreads / 32, kNone = 0x7fffffff;
  __shared__ float red[2][kWarps];
  __shared__ int red_at[kWarps];
  __shared__ float2 mine;
  __shared__ int mine_at;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int part = cluster_ctarank(), r = blockIdx.x / cluster;
  pdl_launch_dependents();
  pdl_wait();
  const int64_t in_at = (int64_t)r * a.stride, out_at = (int64_t)r * a.V;
  const int skew = (int)(in_at % (F32 ? 4 : 8));  // chunk i is the elements 8 i - skew ..
  const int chunks = (a.V + skew + 7) / 8;
  const int c0 = (int)((int64_t)chunks * part / cluster), c1 = (int)((int64_t)chunks * (part + 1) / cluster);
  const bool out_vec = ((out_at - skew) & 3) == 0;
  const float temp = a.temperature ? a.temperature[r] : 1.0f;
  auto load = [&](int c, float (&v)[8]) {
    const int j = 8 * c - skew;
    if (j >= 0 && j + 8 <= a.V) {
      if constexpr (F32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.logits) + in_at + j);
        const float4 x = __ldg(p), y = __ldg(p + 1);
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
      } else {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(static_cast<const __half*>(a.logits) + in_at + j));
        const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = half2_floats(u[i]);
          v[2 * i] = f.x, v[2 * i + 1] = f.y;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = -INFINITY;
        if (j + i >= 0 && j + i < a.V) {
          if constexpr (F32) v[i] = static_cast<const float*>(a.logits)[in_at + j + i];
          else v[i] = __half2float(static_cast<const __half*>(a.logits)[in_at + j + i]);
        }
      }
    }
  };
  float held[kHold ? kHeld : 1][8];
  // f(first element, values) of each of this thread's chunks
  auto each = [&](auto f) {
    if constexpr (kHold) {
#pragma unroll
      for (int i = 0; i < kHeld; ++i)
        if (c0 + tid + i * kThreads < c1) f(8 * (c0 + tid + i * kThreads) - skew, held[i]);
    } else {
      for (int c = c0 + tid; c < c1; c += kThreads) {
        load(c, held[0]);
        f(8 * c - skew, held[0]);
      }
    }
  };
  if constexpr (kHold) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (c0 + tid + i * kThreads < c1) load(c0 + tid + i * kThreads, held[i]);
  }
  float top = -INFINITY;
  each([&](int, const float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) top = nan_max(top, v[i]);
  });
  for (int o = 16; o; o >>= 1) top = nan_max(top, __shfl_xor_sync(kFull, top, o));
  if (lane == 0) red[0][warp] = top;
  __syncthreads();
  top = red[0][lane % kWarps];
  for (int o = kWarps / 2; o; o >>= 1) top = nan_max(top, __shfl_xor_sync(kFull, top, o));
  const float c = temp > 0.0f ? fmaxf(fminf(1.4426950408889634f / temp, FLT_MAX), FLT_MIN) : temp == 0.0f ? 1.0f : NAN;
  const float ref = top == -INFINITY ? 0.0f : top;
  float sum = 0.0f;
  int at = kNone;
  if (temp == 0.0f) {
    each([&](int j, const float (&v)[8]) {
#pragma unroll
      for (int i = 7; i >= 0; --i)
        if (v[i] == top) at = min(at, j + i);
    });
    at = __reduce_min_sync(kFull, at);
    if (lane == 0) red_at[warp] = at;
  } else {
    each([&](int, float (&v)[8]) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float e = ex2((v[i] - ref) * c);
        if constexpr (kHold) v[i] = e;
        sum += e;
      }
    });
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    if (lane == 0) red[1][warp] = sum;
  }
  __syncthreads();
  if (warp == 0) {
    sum = red[1][lane % kWarps];
    for (int o = kWarps / 2; o; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    at = __reduce_min_sync(kFull, red_at[lane % kWarps]);
    if (lane == 0) mine = make_float2(top, sum), mine_at = top == -INFINITY ? kNone : at;
  }
  // ---- over the cluster: lane i reads part i ----
  cluster_arrive();
  cluster_wait();
  float2 other = make_float2(-INFINITY, 0.0f);
  int first = kNone;
  if (lane < cluster) {
    other = cluster_ld_f2(cluster_map(smem_u32(&mine), lane));
    if (temp == 0.0f) first = cluster_ld_s32(cluster_map(smem_u32(&mine_at), lane));
  }
  cluster_arrive();
  float all_top = other.x;
  for (int o = 8; o; o >>= 1) all_top = nan_max(all_top, __shfl_xor_sync(kFull, all_top, o));
  all_top = __shfl_sync(kFull, all_top, 0);
  float all = other.x == -INFINITY ? 0.0f : other.y * ex2((other.x - all_top) * c);
  for (int o = 8; o; o >>= 1) all += __shfl_xor_sync(kFull, all, o);
  all = __shfl_sync(kFull, all, 0);
  first = __reduce_min_sync(kFull, other.x == all_top ? first : kNone);
  const bool none = all_top == -INFINITY;  // no logit above -inf
  const float all_ref = none ? 0.0f : all_top;
  // what a held exponential is off by, and 1 / sum
  const float factor = none ? 0.0f : kHold ? ex2((top - all_top) * c) / all : 1.0f / all;
  each([&](int j, const float (&v)[8]) {
    float p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (temp == 0.0f) p[i] = all_top != all_top ? NAN : j + i == first ? 1.0f : 0.0f;
      else p[i] = (kHold ? v[i] : ex2((v[i] - all_ref) * c)) * factor;
    }
    float* out = a.out + out_at + j;
    if (out_vec && j >= 0 && j + 8 <= a.V) {
      *reinterpret_cast<float4*>(out) = make_float4(p[0], p[1], p[2], p[3]);
      *reinterpret_cast<float4*>(out + 4) = make_float4(p[4], p[5], p[6], p[7]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (j + i >= 0 && j + i < a.V) out[i] = p[i];
    }
  });
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
  // Chunks of 4 elements that begin at 16-byte boundaries of p (and of q, where its row lies alike).
  const int skew = (int)((int64_t)(s0 + b + accepted) * a.target_stride & 3);
  const bool alike = q && ((int64_t)(s0 + accepted) * a.draft_stride & 3) == skew;
  const int chunks = (a.V + skew + 3) / 4;
  const int parts = cluster * kVerifyWarps, own = part * kVerifyWarps + warp;
  const int each = ((chunks + parts - 1) / parts + 31) / 32 * 32;
  const int c0 = (int)min((int64_t)own * each, (int64_t)chunks), c1 = min(c0 + each, chunks);
  auto load = [&](const float* row, int c, bool whole, float (&v)[4]) {
    const int j = 4 * c - skew;
    if (whole && j >= 0 && j + 4 <= a.V) {
      const float4 x = __ldg(reinterpret_cast<const float4*>(row + j));
      v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = j + i >= 0 && j + i < a.V ? __ldg(row + j + i) : 0.0f;
    }
  };
  auto weight = [&](float pj, float qj, int j, bool residual) -> uint64_t {
    const uint64_t f = fixed60(pj);
    if (!residual) return f;
    if (q) return sub_clamped(f, fixed60(qj));
    return j == not_this ? 0 : f;
  };
  constexpr int kFlight = 4;
  uint64_t sum_w = 0, sum_p = 0;
  for (int c = c0 + lane; c < c1; c += 32 * kFlight) {
    float pv[kFlight][4], qv[kFlight][4];
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
#pragma unroll
      for (int i = 0; i < 4; ++i) pv[k][i] = qv[k][i] = 0.0f;
      if (c + 32 * k < c1) {
        load(p, c + 32 * k, true, pv[k]);
        if (q) load(q, c + 32 * k, alike, qv[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < kFlight; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t f = fixed60(pv[k][i]);
        sum_p += f;
        if (q) sum_w += sub_clamped(f, fixed60(qv[k][i]));
        else if (4 * (c + 32 * k) - skew + i != not_this) sum_w += f;
      }
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
    for (int c = c0; c < c1; c += 32) {
      float pv[4] = {}, qv[4] = {};
      uint64_t w[4], inc = 0;
      if (c + lane < c1) {
        load(p, c + lane, true, pv);
        if (q) load(q, c + lane, alike, qv);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[i] = weight(pv[i], qv[i], 4 * (c + lane) - skew + i, residual);
        inc += w[i];
      }
      const uint64_t mine = inc;
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t v = shfl_up_u64(inc, o);
        if (lane >= o) inc += v;
      }
      const uint32_t past = __ballot_sync(kFull, run + inc > limit);
      if (past) {
        if (lane == __ffs(past) - 1) {
          uint64_t s = run + inc - mine;
          int i = 0;
          for (; i < 3; ++i) {
            s += w[i];
            if (s > limit) break;
          }
          a.out[at + accepted] = 4 * (c + lane) - skew + i;
        }
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
  int c = cluster_for(a.rows, a.V, 2048, ctx.num_sms);
  while (c < 16 && a.V + 7 > c * 512 * kHeld * 8) c *= 2;
  const bool hold = a.V + 7 <= c * 512 * kHeld * 8, few = (a.V + 7) / 8 <= c * 128 * kHeld - c;
  ctx.variant = a.f32 ? "softmax_f32" : "softmax_f16";
  auto go = [&](auto kern, int threads, std::atomic<uint64_t>& wide) {
    const cudaError_t e = c > 8 ? allow_wide_clusters(kern, ctx.device, wide) : cudaSuccess;
    return e != cudaSuccess ? e : launch_clusters(ctx, kern, c, dim3((unsigned)a.rows * c), dim3(threads), 0, a, c);
  };
  static std::atomic<uint64_t> wide[6];
  if (!hold) return a.f32 ? go(softmax_kernel<true, 512, false>, 512, wide[0]) : go(softmax_kernel<false, 512, false>, 512, wide[1]);
  if (few) return a.f32 ? go(softmax_kernel<true, 128, true>, 128, wide[2]) : go(softmax_kernel<false, 128, true>, 128, wide[3]);
  return a.f32 ? go(softmax_kernel<true, 512, true>, 512, wide[4]) : go(softmax_kernel<false, 512, true>, 512, wide[5]);
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
