// From logits to verified tokens: probabilities at each row's temperature, and the verification of drafted tokens from
// given random numbers.  Rows that one CTA would be long at are cut into segments: a first launch takes every segment's
// numbers, a second one, which depends on it, joins them.  (A cluster for each row in one launch was slower beyond a few rows: 16 CTAs that have to
// start and meet together; 320 rows of 128256 took 67 us at its best size, one row the same.)
#include <float.h>

#include "mnb_device.cuh"
#include "mnb_internal.h"

namespace mnb {
namespace {

// ---------------------------------------------------------------------------------
// Softmax: p = e^((x - max) / temperature) / sum.  Elements go in chunks of 8 that begin at 16-byte boundaries of the logits,
// whatever the row's own start; a thread keeps its chunks in registers.
// ---------------------------------------------------------------------------------
constexpr int kHeld = 4;           // chunks of a thread
constexpr int kSegThreads = 256;   // of a segment: 8192 elements
constexpr int kNone = 0x7fffffff;

struct SoftPart {  // of a segment: largest, sum of the exponentials relative to it, first place of the largest
  float m, s;
  int at, pad;
};

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

// One row's place, temperature and chunks.
template <bool F32>
struct SoftRow {
  const Softmax& a;
  int64_t in_at, out_at;
  int skew, chunks;  // chunk i is the elements 8 i - skew ..
  __device__ __forceinline__ SoftRow(const Softmax& a_, int r) : a(a_), in_at((int64_t)r * a_.stride), out_at((int64_t)r * a_.V) {
    skew = (int)(in_at % (F32 ? 4 : 8));
    chunks = (a.V + skew + 7) / 8;
  }
  __device__ __forceinline__ void load(int c, float (&v)[8]) const {
    const int j = 8 * c - skew;
    if (j >= 0 && j + 8 <= a.V) {
      if constexpr (F32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.logits) + in_at + j);
        const float4 x = __ldcg(p), y = __ldcg(p + 1);
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
      } else {
        const uint4 x = __ldcg(reinterpret_cast<const uint4*>(static_cast<const __half*>(a.logits) + in_at + j));
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
          if constexpr (F32) v[i] = __ldcg(static_cast<const float*>(a.logits) + in_at + j + i);
          else v[i] = __half2float(__ldcg(static_cast<const __half*>(a.logits) + in_at + j + i));
        }
      }
    }
  }
  __device__ __forceinline__ void store(int c, const float (&p)[8]) const {
    const int j = 8 * c - skew;
    float* out = a.out + out_at + j;
    if (((out_at - skew) & 3) == 0 && j >= 0 && j + 8 <= a.V) {
      *reinterpret_cast<float4*>(out) = make_float4(p[0], p[1], p[2], p[3]);
      *reinterpret_cast<float4*>(out + 4) = make_float4(p[4], p[5], p[6], p[7]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (j + i >= 0 && j + i < a.V) out[i] = p[i];
    }
  }
};

// 1 / temperature in powers of two, within what keeps 0 * it at 0 and -inf * it at -inf; NaN for what is no temperature.
__device__ __forceinline__ float cold_factor(float temp) {
  return temp > 0.0f ? fmaxf(fminf(1.4426950408889634f / temp, FLT_MAX), FLT_MIN) : temp == 0.0f ? 1.0f : NAN;
}

// Largest, its first place (temperature 0) or the sum of exponentials (else) of a CTA's chunks, for all its threads; the
// exponentials replace the values.
template <int kThreads>
__device__ __forceinline__ SoftPart soft_part(float (&v)[kHeld][8], int n, int first, float temp, float c) {
  constexpr int kWarps = kThreads / 32;
  __shared__ float red[2][kWarps];
  __shared__ int red_at[kWarps];
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  SoftPart r = {-INFINITY, 0.0f, kNone, 0};
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (tid + i * kThreads < n)
#pragma unroll
      for (int k = 0; k < 8; ++k) r.m = nan_max(r.m, v[i][k]);
#pragma unroll
  for (int o = 16; o; o >>= 1) r.m = nan_max(r.m, __shfl_xor_sync(kFull, r.m, o));
  if (lane == 0) red[0][warp] = r.m;
  __syncthreads();
  r.m = red[0][lane % kWarps];
#pragma unroll
  for (int o = kWarps / 2; o; o >>= 1) r.m = nan_max(r.m, __shfl_xor_sync(kFull, r.m, o));
  if (temp == 0.0f) {
#pragma unroll
    for (int i = kHeld - 1; i >= 0; --i)
      if (tid + i * kThreads < n)
#pragma unroll
        for (int k = 7; k >= 0; --k)
          if (v[i][k] == r.m) r.at = first + 8 * (tid + i * kThreads) + k;
    r.at = __reduce_min_sync(kFull, r.at);
    if (lane == 0) red_at[warp] = r.at;
    __syncthreads();
    r.at = r.m == -INFINITY ? kNone : __reduce_min_sync(kFull, red_at[lane % kWarps]);
  } else {
    const float ref = r.m == -INFINITY ? 0.0f : r.m;
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (tid + i * kThreads < n)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          v[i][k] = ex2((v[i][k] - ref) * c);
          r.s += v[i][k];
        }
#pragma unroll
    for (int o = 16; o; o >>= 1) r.s += __shfl_xor_sync(kFull, r.s, o);
    if (lane == 0) red[1][warp] = r.s;
    __syncthreads();
    r.s = red[1][lane % kWarps];
#pragma unroll
    for (int o = kWarps / 2; o; o >>= 1) r.s += __shfl_xor_sync(kFull, r.s, o);
  }
  return r;
}

// Rows of up to kThreads * kHeld chunks: a CTA has one, and reads it once.
template <bool F32, int kThreads>
__global__ void __launch_bounds__(kThreads) softmax_row_kernel(const Softmax a) {
  pdl_launch_dependents();
  pdl_wait();
  const SoftRow<F32> row(a, blockIdx.x);
  const float temp = a.temperature ? a.temperature[blockIdx.x] : 1.0f;
  float v[kHeld][8];
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if ((int)threadIdx.x + i * kThreads < row.chunks) row.load(threadIdx.x + i * kThreads, v[i]);
  const SoftPart all = soft_part<kThreads>(v, row.chunks, -row.skew, temp, cold_factor(temp));
  const float inv = all.m == -INFINITY ? 0.0f : 1.0f / all.s;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int c = threadIdx.x + i * kThreads;
    if (c < row.chunks) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (temp == 0.0f) v[i][k] = all.m != all.m ? NAN : 8 * c - row.skew + k == all.at ? 1.0f : 0.0f;
        else v[i][k] *= inv;
      }
      row.store(c, v[i]);
    }
  }
}

// Longer rows: a CTA has a segment, in both launches.
template <bool F32>
__global__ void __launch_bounds__(kSegThreads) softmax_part_kernel(const Softmax a, int segs) {
  pdl_wait();
  pdl_launch_dependents();  // behind the wait: the next launch reads logits (past L1) before its own
  const int r = blockIdx.x / segs, seg = blockIdx.x % segs;
  const SoftRow<F32> row(a, r);
  const float temp = a.temperature ? a.temperature[r] : 1.0f;
  const int c0 = (int)((int64_t)row.chunks * seg / segs), n = (int)((int64_t)row.chunks * (seg + 1) / segs) - c0;
  float v[kHeld][8];
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if ((int)threadIdx.x + i * kSegThreads < n) row.load(c0 + threadIdx.x + i * kSegThreads, v[i]);
  const SoftPart part = soft_part<kSegThreads>(v, n, 8 * c0 - row.skew, temp, cold_factor(temp));
  if (threadIdx.x == 0) static_cast<SoftPart*>(a.workspace)[blockIdx.x] = part;
}

template <bool F32>
__global__ void __launch_bounds__(kSegThreads) softmax_join_kernel(const Softmax a, int segs) {
  pdl_launch_dependents();
  const int r = blockIdx.x / segs, seg = blockIdx.x % segs, lane = threadIdx.x % 32;
  const SoftRow<F32> row(a, r);
  const float temp = a.temperature ? a.temperature[r] : 1.0f, c = cold_factor(temp);
  const int c0 = (int)((int64_t)row.chunks * seg / segs), n = (int)((int64_t)row.chunks * (seg + 1) / segs) - c0;
  float v[kHeld][8];
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if ((int)threadIdx.x + i * kSegThreads < n) row.load(c0 + threadIdx.x + i * kSegThreads, v[i]);
  pdl_wait();
  const SoftPart* parts = static_cast<const SoftPart*>(a.workspace) + (int64_t)r * segs;
  SoftPart all = {-INFINITY, 0.0f, kNone, 0};
  for (int s = lane; s < segs; s += 32) {
    const int4 u = *reinterpret_cast<const int4*>(parts + s);
    const float m = __int_as_float(u.x), top = nan_max(all.m, m), ref = top == -INFINITY ? 0.0f : top;
    if (m > all.m) all.at = u.z;
    all.s = all.s * ex2((all.m - ref) * c) + __int_as_float(u.y) * ex2((m - ref) * c);
    all.m = top;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float m = __shfl_xor_sync(kFull, all.m, o), s = __shfl_xor_sync(kFull, all.s, o);
    const int at = __shfl_xor_sync(kFull, all.at, o);
    const float top = nan_max(all.m, m), ref = top == -INFINITY ? 0.0f : top;
    all.at = m > all.m ? at : m == all.m ? min(all.at, at) : all.at;
    all.s = all.s * ex2((all.m - ref) * c) + s * ex2((m - ref) * c);
    all.m = top;
  }
  const float ref = all.m == -INFINITY ? 0.0f : all.m, inv = all.m == -INFINITY ? 0.0f : 1.0f / all.s;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int k0 = threadIdx.x + i * kSegThreads;
    if (k0 < n) {
      const int ch = c0 + k0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (temp == 0.0f) v[i][k] = all.m != all.m ? NAN : 8 * ch - row.skew + k == all.at ? 1.0f : 0.0f;
        else v[i][k] = ex2((v[i][k] - ref) * c) * inv;
      }
      row.store(ch, v[i]);
    }
  }
}

// Chunks of a row that one CTA takes, and segments of longer rows (0: one CTA).
int soft_segments(int V) {
  const int chunks = (V + 14) / 8;
  return chunks <= 512 * kHeld ? 0 : (chunks + kSegThreads * kHeld - 1) / (kSegThreads * kHeld);
}

// ---------------------------------------------------------------------------------
// Verification.  Every CTA of a sequence's segments finds the first rejected token by itself and sums its segment of the
// row to draw from; the second launch has a CTA for each sequence, which finds the segment, then the element.
//
// Weights are whole numbers of 2^-60 (probabilities are held to 0..1; what is below 2^-60 counts as 0): sums are exact in any
// order, and the drawn token does not hang on how the row was cut. A row may add up to just below 16.
// ---------------------------------------------------------------------------------
constexpr int kVerifyWarps = 8, kVerifyThreads = kVerifyWarps * 32;
constexpr int kRun = 4;                                // chunks of 4 elements of a thread
constexpr int kSegChunks = kVerifyThreads * kRun;      // of a segment: 4096 elements

struct VerifyPart {  // of a segment: sums of max(p - q, 0) and of p
  uint64_t w, p;
};

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

__device__ __forceinline__ uint64_t shfl_u64(uint64_t v, int from) { return __shfl_sync(kFull, (unsigned long long)v, from); }
__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, (unsigned long long)v, o);
  return v;
}
__device__ __forceinline__ uint64_t warp_scan(uint64_t v, int lane) {  // of the lanes up to this one
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t u = __shfl_up_sync(kFull, (unsigned long long)v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// The row to draw from, in chunks of 4 elements that begin at 16-byte boundaries of p (and of q, where its row lies alike).
struct DrawRow {
  const float *p, *q;  // q: null when all were accepted, or without draft rows
  int V, not_this;     // not_this: the rejected token without draft rows, -1 else
  int skew, chunks;
  bool rejected, alike;
  __device__ __forceinline__ DrawRow(const Verify& a, int b, int s0, int n, int accepted) : V(a.V) {
    rejected = accepted < n;
    const int64_t p_at = (int64_t)(s0 + b + accepted) * a.target_stride, q_at = (int64_t)(s0 + accepted) * a.draft_stride;
    p = a.target + p_at;
    q = rejected && a.draft ? a.draft + q_at : nullptr;
    not_this = rejected && !a.draft ? a.tokens[s0 + accepted] : -1;
    skew = (int)(p_at & 3);
    alike = (q_at & 3) == skew;
    chunks = (V + skew + 3) / 4;
  }
  __device__ __forceinline__ void load4(const float* row, int c, bool whole, float (&v)[4]) const {
    const int j = 4 * c - skew;
    if (whole && j >= 0 && j + 4 <= V) {
      const float4 x = __ldg(reinterpret_cast<const float4*>(row + j));
      v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = j + i >= 0 && j + i < V ? __ldg(row + j + i) : 0.0f;
    }
  }
};

__device__ __forceinline__ void sequence(const Verify& a, int b, int& s0, int& n) {
  s0 = min(max(a.start[b], 0), a.drafted);
  n = min(max(a.start[b + 1], s0), a.drafted) - s0;
}

__global__ void __launch_bounds__(kVerifyThreads) verify_part_kernel(const Verify a, int segs, uint32_t* status) {
  __shared__ uint64_t sums[2][kVerifyWarps];
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int b = blockIdx.x / segs, seg = blockIdx.x % segs;
  pdl_launch_dependents();
  pdl_wait();
  int s0, n;
  sequence(a, b, s0, n);
  // ---- the first rejected token ----
  int accepted = n;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int i = i0 + lane;
    bool bad = false;
    if (i < n) {
      const int tok = a.tokens[s0 + i];
      const float u = __saturatef(a.u_accept[s0 + i]);
      bad = true;
      if (tok >= 0 && tok < a.V) {
        const float pt = __saturatef(a.target[(int64_t)(s0 + b + i) * a.target_stride + tok]);
        const float qt = a.draft ? __saturatef(a.draft[(int64_t)(s0 + i) * a.draft_stride + tok]) : 1.0f;
        bad = !((double)u * (double)qt < (double)pt);
      } else if (seg == 0 && warp == 0) {
        report_status(status, kStatusBadIndex);
      }
    }
    const uint32_t vote = __ballot_sync(kFull, bad);
    if (vote) {
      accepted = i0 + __ffs(vote) - 1;
      break;
    }
  }
  // ---- sums of this segment ----
  const DrawRow row(a, b, s0, n, accepted);
  const int c0 = seg * kSegChunks + tid;
  float pv[kRun][4], qv[kRun][4];
#pragma unroll
  for (int k = 0; k < kRun; ++k) {
    const int c = c0 + k * kVerifyThreads;
#pragma unroll
    for (int i = 0; i < 4; ++i) pv[k][i] = qv[k][i] = 0.0f;
    if (c < row.chunks) {
      row.load4(row.p, c, true, pv[k]);
      if (row.q) row.load4(row.q, c, row.alike, qv[k]);
    }
  }
  uint64_t sum_w = 0, sum_p = 0;
#pragma unroll
  for (int k = 0; k < kRun; ++k)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t f = fixed60(pv[k][i]);
      sum_p += f;
      if (row.q) sum_w += sub_clamped(f, fixed60(qv[k][i]));
      else if (4 * (c0 + k * kVerifyThreads) - row.skew + i != row.not_this) sum_w += f;
    }
  sum_w = warp_sum(sum_w), sum_p = warp_sum(sum_p);
  if (lane == 0) sums[0][warp] = sum_w, sums[1][warp] = sum_p;
  __syncthreads();
  if (tid == 0) {
    VerifyPart r = {0, 0};
    for (int w = 0; w < kVerifyWarps; ++w) r.w += sums[0][w], r.p += sums[1][w];
    static_cast<VerifyPart*>(a.workspace)[blockIdx.x] = r;
    if (seg == 0) a.accepted[b] = accepted;
  }
}

__global__ void __launch_bounds__(kVerifyThreads) verify_draw_kernel(const Verify a, int segs) {
  __shared__ uint64_t runs[kVerifyWarps];
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, b = blockIdx.x;
  pdl_launch_dependents();
  pdl_wait();
  int s0, n;
  sequence(a, b, s0, n);
  const int accepted = min(max(a.accepted[b], 0), n);  // the first launch's: in range unless the caller's buffers overlap
  const float u = a.u_next[b];
  const VerifyPart* parts = static_cast<const VerifyPart*>(a.workspace) + (int64_t)b * segs;
  int32_t* out = a.out + s0 + b;
  // ---- the row's total, then the segment that the drawn one is in; every warp finds it by itself ----
  VerifyPart total = {0, 0}, first = {0, 0};
  for (int s = lane; s < segs; s += 32) {
    const VerifyPart v = parts[s];
    if (s == lane) first = v;
    total.w += v.w, total.p += v.p;
  }
  const DrawRow row(a, b, s0, n, accepted);
  total.w = row.rejected ? warp_sum(total.w) : 0;
  const bool residual = total.w > 0;  // nothing left of p - q: drawn from p
  const uint64_t all = residual ? total.w : warp_sum(total.p);
  const uint64_t limit = scaled(all, u);
  uint64_t head = 0;
  int seg = -1;
  for (int i = 0; i < segs; i += 32) {
    VerifyPart v = first;
    if (i > 0 && i + lane < segs) v = parts[i + lane];
    const uint64_t x = i + lane < segs ? residual ? v.w : v.p : 0, to = head + warp_scan(x, lane);
    const uint32_t past = __ballot_sync(kFull, to > limit);
    if (past) {
      seg = i + __ffs(past) - 1;
      head = shfl_u64(to - x, __ffs(past) - 1);
      break;
    }
    head = shfl_u64(to, 31);
  }
  for (int i = tid; i <= n; i += kVerifyThreads)
    if (i != accepted || all == 0) out[i] = i < accepted ? a.tokens[s0 + i] : -1;
  if (seg < 0) return;
  // ---- the element: each warp a run of the segment ----
  const int c0 = seg * kSegChunks + warp * (32 * kRun);
  uint64_t w[kRun][4], sum[kRun], mine = 0;
  float pv[kRun][4], qv[kRun][4];
#pragma unroll
  for (int k = 0; k < kRun; ++k) {
    const int c = c0 + 32 * k + lane;
#pragma unroll
    for (int i = 0; i < 4; ++i) pv[k][i] = qv[k][i] = 0.0f;
    if (c < row.chunks) {
      row.load4(row.p, c, true, pv[k]);
      if (row.q && residual) row.load4(row.q, c, row.alike, qv[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < kRun; ++k) {
    sum[k] = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[k][i] = fixed60(pv[k][i]);
      if (residual && row.q) w[k][i] = sub_clamped(w[k][i], fixed60(qv[k][i]));
      if (residual && 4 * (c0 + 32 * k + lane) - row.skew + i == row.not_this) w[k][i] = 0;
      sum[k] += w[k][i];
    }
    mine += sum[k];
  }
  mine = warp_sum(mine);
  if (lane == 0) runs[warp] = mine;
  __syncthreads();
  for (int i = 0; i < warp; ++i) head += runs[i];
  if (head <= limit && head + mine > limit) {
    bool done = false;
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
      if (!done) {
        const uint64_t to = head + warp_scan(sum[k], lane);
        const uint32_t past = __ballot_sync(kFull, to > limit);
        if (past) {
          done = true;
          if (lane == __ffs(past) - 1) {
            uint64_t s = to - sum[k];
            int at = 3;
#pragma unroll
            for (int i = 2; i >= 0; --i) {
              uint64_t upto = s;
#pragma unroll
              for (int j = 0; j <= i; ++j) upto += w[k][j];
              if (upto > limit) at = i;
            }
            out[accepted] = 4 * (c0 + 32 * k + lane) - row.skew + at;
          }
        }
        head = shfl_u64(to, 31);
      }
    }
  }
}

int verify_segments(int V) { return ((V + 6) / 4 + kSegChunks - 1) / kSegChunks; }

}  // namespace

size_t softmax_workspace_bytes(int rows, int V) { return (size_t)rows * soft_segments(V) * sizeof(SoftPart); }
size_t verify_workspace_bytes(int batch, int V) { return (size_t)batch * verify_segments(V) * sizeof(VerifyPart); }

cudaError_t launch_softmax(LaunchCtx& ctx, const Softmax& a) {
  ctx.variant = a.f32 ? "softmax_f32" : "softmax_f16";
  const int segs = soft_segments(a.V);
  if (segs == 0) {
    const bool few = (a.V + 14) / 8 <= 128 * kHeld;
    auto go = [&](auto kern, int threads) { return launch_kernel(ctx, kern, dim3(a.rows), dim3(threads), 0, a); };
    if (few) return a.f32 ? go(softmax_row_kernel<true, 128>, 128) : go(softmax_row_kernel<false, 128>, 128);
    return a.f32 ? go(softmax_row_kernel<true, 512>, 512) : go(softmax_row_kernel<false, 512>, 512);
  }
  const dim3 grid((unsigned)a.rows * segs);
  cudaError_t e = a.f32 ? launch_kernel(ctx, softmax_part_kernel<true>, grid, dim3(kSegThreads), 0, a, segs)
                        : launch_kernel(ctx, softmax_part_kernel<false>, grid, dim3(kSegThreads), 0, a, segs);
  if (e != cudaSuccess) return e;
  const bool pdl = ctx.pdl;
  ctx.pdl = true;  // the second launch waits for the first one on the device
  e = a.f32 ? launch_kernel(ctx, softmax_join_kernel<true>, grid, dim3(kSegThreads), 0, a, segs)
            : launch_kernel(ctx, softmax_join_kernel<false>, grid, dim3(kSegThreads), 0, a, segs);
  ctx.pdl = pdl;
  return e;
}

cudaError_t launch_verify(LaunchCtx& ctx, const Verify& a) {
  ctx.variant = "verify";
  const int segs = verify_segments(a.V);
  cudaError_t e = launch_kernel(ctx, verify_part_kernel, dim3((unsigned)a.batch * segs), dim3(kVerifyThreads), 0, a, segs, ctx.status);
  if (e != cudaSuccess) return e;
  const bool pdl = ctx.pdl;
  ctx.pdl = true;
  e = launch_kernel(ctx, verify_draw_kernel, dim3(a.batch), dim3(kVerifyThreads), 0, a, segs);
  ctx.pdl = pdl;
  return e;
}

}  // namespace mnb
