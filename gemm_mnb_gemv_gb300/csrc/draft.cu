// From logits to verified tokens: probabilities at each row's temperature, and the verification of drafted tokens from
// given random numbers.
//
// Rows that one CTA would be long at are cut into segments.  A few of them have a cluster of CTAs each, which hand each other their
// segments' numbers; many go through two launches, the second of which depends on the first. (Clusters have to start and meet together: 320
// rows of 128256 took 67 us with them at their best size, in two launches 50.)
// Softmax, bound: 320 x 128256 fp16 with temperatures, 50 us (36 at the copy rate). The first launch takes 16 us, most of it
// arithmetic (70% of the issue slots); the second reads the logits again, about half of them from L2, and writes at the memory's rate (7 TB/s).
// One row: 4.8 us, launch and cluster.
// Verification, bound: 64 x 4 drafted tokens x 128256, 15.0 us (8.9): three loads that follow each other to the accepted length, then one row
// of p and q at half the copy rate, the cluster, the element. One sequence: 6.2 us. Where nothing is left of p - q, one CTA reads the row again: 21 us
// for one sequence, 50 for 64 that all do.
#include <float.h>

#include "cluster.cuh"
#include "mnb_device.cuh"
#include "mnb_internal.h"

namespace mnb {
namespace {

// CTAs that share a row of `chunks`: four an SM together where that is possible, so that none waits for another's end, each with
// `smallest` to `largest` chunks.
int row_parts(int rows, int chunks, int smallest, int largest) {
  const int most = (chunks + smallest - 1) / smallest, least = (chunks + largest - 1) / largest, want = 4 * 152 / rows;
  return want < least ? least : want > most ? most : want;
}

// ---------------------------------------------------------------------------------
// Softmax: p = e^((x - max) / temperature) / sum.  Elements go in chunks of 8 that begin at 16-byte boundaries of the logits,
// whatever the row's own start.
// ---------------------------------------------------------------------------------
constexpr int kBatch = 4;          // chunks of a thread in flight
constexpr int kPartThreads = 256;  // of a row's part
constexpr int kNone = 0x7fffffff;
constexpr int kMostCluster = 16, kClusterThreads = 512;
constexpr float kLeastC = 1.0f / (1ull << 63) / (1ull << 63) / (1 << 23);  // 2^-149: logits differ by less than 2^129, so this is no temperature at all

struct SoftPart {  // of a part: largest, sum of the exponentials relative to it, first place of the largest
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
__device__ __forceinline__ float some(float m) { return m == -INFINITY ? 0.0f : m; }  // what logits are taken relative to
// The factor that brings sums relative to m to `ref`; halves, as the difference of two finite ones may be none.
__device__ __forceinline__ float rescale(float m, float ref, float c) { return ex2((0.5f * m - 0.5f * ref) * c * 2.0f); }
struct Base;

// Eight logits as they lie.
template <bool F32>
struct Chunk {
  uint32_t u[F32 ? 8 : 4];
  __device__ __forceinline__ float2 pair(int i) const {
    if constexpr (F32) return make_float2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
    else return half2_floats(u[i]);
  }
  __device__ __forceinline__ float largest() const {
    if constexpr (F32) {
      float m = __uint_as_float(u[0]);
#pragma unroll
      for (int i = 1; i < 8; ++i) m = nan_max(m, __uint_as_float(u[i]));
      return m;
    } else {
      uint32_t m = u[0];
#pragma unroll
      for (int i = 1; i < 4; ++i) asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(u[i]));
      const float2 f = half2_floats(m);
      return nan_max(f.x, f.y);
    }
  }
  // e^((x - m) c) / base.factor
  template <bool kPlain>
  __device__ __forceinline__ void exps(const Base& base, float (&e)[8]) const;
};

// The exponent (x - m) c as one operation, x c - rc, where rc = m c is moderate: rc's rounding is the same for all and goes into
// `factor` = 2^(rc - m c), by its series (ex2's own error, 2^-22, would be every probability's). Else as two (infinite logits, large
// ones, temperatures near 0).
struct Base {
  float m, c, rc, factor;
  bool plain;
  __device__ __forceinline__ Base(float m_, float c_) : m(some(m_)), c(c_) {
    rc = m * c;
    plain = fabsf(rc) < 65536.0f;  // its rounding moves the exponent by 2^-9 at most: the series' third term is below 2^-28
    const float y = plain ? -0.693147181f * fmaf(m, c, -rc) : 0.0f;
    factor = fmaf(y, fmaf(y, 0.5f, 1.0f), 1.0f);
  }
  template <bool kPlain>
  __device__ __forceinline__ float exponent(float x) const {
    return kPlain ? fmaf(x, c, -rc) : (x - m) * c;
  }
};
template <bool F32>
template <bool kPlain>
__device__ __forceinline__ void Chunk<F32>::exps(const Base& base, float (&e)[8]) const {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = pair(i);
    e[2 * i] = ex2(base.exponent<kPlain>(f.x)), e[2 * i + 1] = ex2(base.exponent<kPlain>(f.y));
  }
}

template <bool F32>
struct SoftRow {
  const Softmax& a;
  int64_t in_at, out_at;
  int skew, chunks;  // chunk i is the elements 8 i - skew ..
  float temp, c;     // c: 1 / temperature in powers of two, within what keeps 0 * c at 0 and -inf * c at -inf (subnormal for the largest
                     // temperatures, the smallest one for an infinite one); NaN for no temperature
  __device__ __forceinline__ SoftRow(const Softmax& a_, int r) : a(a_), in_at((int64_t)r * a_.stride), out_at((int64_t)r * a_.V) {
    skew = (int)(in_at % 8);
    chunks = (a.V + skew + 7) / 8;
    temp = a.temperature ? __ldcg(a.temperature + r) : 1.0f;
    c = temp > 0.0f ? fmaxf(fminf(1.4426950408889634f / temp, FLT_MAX), kLeastC) : temp == 0.0f ? 1.0f : NAN;
  }
  // Whether chunks i0 .. i1 - 1 lie within the row, and its probabilities at 32 bytes.
  __device__ __forceinline__ bool whole(int i0, int i1) const {
    return 8 * i0 - skew >= 0 && 8 * i1 - skew <= a.V && ((reinterpret_cast<uintptr_t>(a.out + out_at) >> 2) - skew) % 8 == 0;
  }
  // Chunk i when `live`, past L1; -inf beyond the row and when not.
  template <bool kWhole>
  __device__ __forceinline__ void load(int i, bool live, Chunk<F32>& v) const {
    constexpr int kWords = F32 ? 8 : 4;
    const int j = 8 * i - skew;
#pragma unroll
    for (int k = 0; k < kWords; ++k) v.u[k] = F32 ? 0xff800000u : 0xfc00fc00u;
    if (!live) return;
    if (kWhole || (j >= 0 && j + 8 <= a.V)) {
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.logits) + (in_at + j) * (F32 ? 4 : 2));
#pragma unroll
      for (int k = 0; k < kWords / 4; ++k) {
        const uint4 x = __ldcg(p + k);
        v.u[4 * k] = x.x, v.u[4 * k + 1] = x.y, v.u[4 * k + 2] = x.z, v.u[4 * k + 3] = x.w;
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (j + k >= 0 && j + k < a.V) {
          if constexpr (F32) v.u[k] = __ldcg(static_cast<const uint32_t*>(a.logits) + in_at + j + k);
          else v.u[k / 2] = __byte_perm(v.u[k / 2], __ldcg(static_cast<const unsigned short*>(a.logits) + in_at + j + k), k & 1 ? 0x5410 : 0x3254);
        }
    }
  }
  // 32 bytes in one store (two of 16 would write every sector twice), streaming: the logits are to stay in L2
  template <bool kWhole>
  __device__ __forceinline__ void store(int i, const float (&p)[8]) const {
    const int j = 8 * i - skew;
    float* out = a.out + out_at + j;
    if (kWhole) {
      asm volatile("st.global.cs.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(out), "f"(p[0]), "f"(p[1]), "f"(p[2]),
                   "f"(p[3]), "f"(p[4]), "f"(p[5]), "f"(p[6]), "f"(p[7])
                   : "memory");
    } else if ((reinterpret_cast<uintptr_t>(out) & 15) == 0 && j >= 0 && j + 8 <= a.V) {
      __stcs(reinterpret_cast<float4*>(out), make_float4(p[0], p[1], p[2], p[3]));
      __stcs(reinterpret_cast<float4*>(out + 4), make_float4(p[4], p[5], p[6], p[7]));
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (j + k >= 0 && j + k < a.V) out[k] = p[k];
    }
  }
  __device__ __forceinline__ int find(int i, const Chunk<F32>& v, float m) const {  // first place of m in the chunk
    int at = kNone;
#pragma unroll
    for (int k = 7; k >= 0; --k) {
      const float2 f = v.pair(k / 2);
      if ((k & 1 ? f.y : f.x) == m) at = 8 * i - skew + k;
    }
    return at;
  }
  template <bool kWhole>
  __device__ __forceinline__ void one_hot(int i, const SoftPart& all) const {  // temperature 0
    const float zero = all.m != all.m ? NAN : 0.0f;
    const int at = all.at - (8 * i - skew);
    float p[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) p[k] = at == k ? zero + 1.0f : zero;
    store<kWhole>(i, p);
  }
};

// a and b together
__device__ __forceinline__ SoftPart join(const SoftPart& a, const SoftPart& b, float c) {
  SoftPart r = {nan_max(a.m, b.m), 0.0f, kNone, 0};
  const float ref = some(r.m);
  r.s = a.s * rescale(a.m, ref, c) + b.s * rescale(b.m, ref, c);
  r.at = a.m > b.m ? a.at : b.m > a.m ? b.at : min(a.at, b.at);
  return r;
}
__device__ __forceinline__ SoftPart warp_join(SoftPart r, float c) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const SoftPart v = {__shfl_xor_sync(kFull, r.m, o), __shfl_xor_sync(kFull, r.s, o), __shfl_xor_sync(kFull, r.at, o), 0};
    r = join(r, v, c);
  }
  return r;
}
// Of the CTA's threads, for all of them: the largest first, so that a thread's sum is brought to it once.
template <int kThreads>
__device__ __forceinline__ SoftPart cta_join(SoftPart r, float temp, float c) {
  constexpr int kWarps = kThreads / 32;
  __shared__ float m[kWarps], s[kWarps];
  __shared__ int at[kWarps];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  float top = r.m;
#pragma unroll
  for (int o = 16; o; o >>= 1) top = nan_max(top, __shfl_xor_sync(kFull, top, o));
  if (temp == 0.0f) {
    r.at = __reduce_min_sync(kFull, r.m == top ? r.at : kNone);
  } else {
    r.s *= rescale(r.m, some(top), c);
#pragma unroll
    for (int o = 16; o; o >>= 1) r.s += __shfl_xor_sync(kFull, r.s, o);
  }
  if (lane == 0) m[warp] = top, s[warp] = r.s, at[warp] = r.at;
  __syncthreads();
  r.m = m[lane % kWarps];
  top = r.m;
#pragma unroll
  for (int o = kWarps / 2; o; o >>= 1) top = nan_max(top, __shfl_xor_sync(kFull, top, o));
  if (temp == 0.0f) {
    r.at = __reduce_min_sync(kFull, r.m == top ? at[lane % kWarps] : kNone);
  } else {
    r.s = s[lane % kWarps] * rescale(r.m, some(top), c);
#pragma unroll
    for (int o = kWarps / 2; o; o >>= 1) r.s += __shfl_xor_sync(kFull, r.s, o);
  }
  r.m = top;
  return r;
}

// A batch joins r: chunks i, i + kThreads .. (-inf where there are none).
template <bool F32, int kThreads, bool kPlain>
__device__ __forceinline__ float batch_sum(const Chunk<F32> (&v)[kBatch], const Base& base) {
  float sum[4] = {}, e[8];
#pragma unroll
  for (int k = 0; k < kBatch; ++k) {
    v[k].template exps<kPlain>(base, e);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[j % 4] += e[j];
  }
  return ((sum[0] + sum[1]) + (sum[2] + sum[3])) * base.factor;
}
template <bool F32, int kThreads>
__device__ __forceinline__ void take(const SoftRow<F32>& row, const Chunk<F32> (&v)[kBatch], int i, SoftPart& r) {
  float m = r.m;
#pragma unroll
  for (int k = 0; k < kBatch; ++k) m = nan_max(m, v[k].largest());
  if (row.temp == 0.0f) {
    if (m > r.m) {
      r.at = kNone;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) r.at = min(r.at, row.find(i + k * kThreads, v[k], m));
    }
  } else {
    const Base base(m, row.c);
    const float sum = base.plain ? batch_sum<F32, kThreads, true>(v, base) : batch_sum<F32, kThreads, false>(v, base);
    r.s = r.s * rescale(r.m, base.m, row.c) + sum;
  }
  r.m = m;
}
template <bool F32, int kThreads, bool kWhole>
__device__ __forceinline__ void load_batch(const SoftRow<F32>& row, int i, int end, Chunk<F32> (&v)[kBatch]) {
#pragma unroll
  for (int k = 0; k < kBatch; ++k) row.template load<kWhole>(i + k * kThreads, i + k * kThreads < end, v[k]);
}
template <bool F32, int kThreads, bool kWhole, bool kPlain>
__device__ __forceinline__ void store_batch(const SoftRow<F32>& row, int i, int end, const Chunk<F32> (&v)[kBatch], const Base& base, float inv) {
#pragma unroll
  for (int k = 0; k < kBatch; ++k) {
    float e[8];
    v[k].template exps<kPlain>(base, e);
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] *= inv;
    if (i + k * kThreads < end) row.template store<kWhole>(i + k * kThreads, e);
  }
}

// Rows of up to kThreads * kBatch chunks: a CTA has one, and reads it once.
template <bool F32, int kThreads>
__global__ void __launch_bounds__(kThreads) softmax_row_kernel(const Softmax a) {
  pdl_launch_dependents();
  pdl_wait();
  const SoftRow<F32> row(a, blockIdx.x);
  const int tid = threadIdx.x, end = row.chunks;
  Chunk<F32> v[kBatch];
  const bool whole = row.whole(0, end);
  if (whole) load_batch<F32, kThreads, true>(row, tid, end, v);
  else load_batch<F32, kThreads, false>(row, tid, end, v);
  SoftPart all = {-INFINITY, 0.0f, kNone, 0};
  take<F32, kThreads>(row, v, tid, all);
  all = cta_join<kThreads>(all, row.temp, row.c);
  if (row.temp == 0.0f) {
    for (int i = tid; i < end; i += kThreads) row.template one_hot<false>(i, all);
    return;
  }
  const Base base(all.m, row.c);
  const float inv = all.m == -INFINITY ? 0.0f : base.factor / all.s;
  if (whole && base.plain) store_batch<F32, kThreads, true, true>(row, tid, end, v, base, inv);
  else if (base.plain) store_batch<F32, kThreads, false, true>(row, tid, end, v, base, inv);
  else store_batch<F32, kThreads, false, false>(row, tid, end, v, base, inv);
}

// A few longer rows: a cluster of `cluster` CTAs has one, in registers.
template <bool F32>
__global__ void __launch_bounds__(kClusterThreads) softmax_cluster_kernel(const Softmax a, int cluster) {
  __shared__ __align__(16) SoftPart parts[kMostCluster];
  cluster_arrive();
  pdl_launch_dependents();
  pdl_wait();
  const int r = blockIdx.x / cluster, part = cluster_ctarank(), tid = threadIdx.x, lane = tid % 32;
  const SoftRow<F32> row(a, r);
  const int i0 = (int)((int64_t)row.chunks * part / cluster), i1 = (int)((int64_t)row.chunks * (part + 1) / cluster);
  Chunk<F32> v[kBatch];
  const bool whole = row.whole(i0, i1);
  if (whole) load_batch<F32, kClusterThreads, true>(row, i0 + tid, i1, v);
  else load_batch<F32, kClusterThreads, false>(row, i0 + tid, i1, v);
  SoftPart all = {-INFINITY, 0.0f, kNone, 0};
  take<F32, kClusterThreads>(row, v, i0 + tid, all);
  all = cta_join<kClusterThreads>(all, row.temp, row.c);
  cluster_wait();  // the others have started
  if (tid < cluster) {
    const uint32_t to = cluster_map(smem_u32(&parts[part]), tid);
    cluster_st_u64(to, __float_as_uint(all.m), __float_as_uint(all.s));
    cluster_st_u64(to + 8, (uint32_t)all.at, 0u);
  }
  __syncwarp();
  cluster_arrive();
  cluster_wait();
  all = {-INFINITY, 0.0f, kNone, 0};
  if (lane < cluster) all = parts[lane];
  all = warp_join(all, row.c);
  if (row.temp == 0.0f) {
    for (int i = i0 + tid; i < i1; i += kClusterThreads) row.template one_hot<false>(i, all);
    return;
  }
  const Base base(all.m, row.c);
  const float inv = all.m == -INFINITY ? 0.0f : base.factor / all.s;
  if (whole && base.plain) store_batch<F32, kClusterThreads, true, true>(row, i0 + tid, i1, v, base, inv);
  else if (base.plain) store_batch<F32, kClusterThreads, false, true>(row, i0 + tid, i1, v, base, inv);
  else store_batch<F32, kClusterThreads, false, false>(row, i0 + tid, i1, v, base, inv);
}

// Longer rows: a CTA has a part, the same one in both launches.
template <bool F32, bool kWhole>
__device__ __forceinline__ SoftPart part_of(const SoftRow<F32>& row, int i0, int i1) {
  SoftPart mine = {-INFINITY, 0.0f, kNone, 0};
  for (int i = i0 + threadIdx.x; i < i1; i += kPartThreads * kBatch) {
    Chunk<F32> v[kBatch];
    load_batch<F32, kPartThreads, kWhole>(row, i, i1, v);
    take<F32, kPartThreads>(row, v, i, mine);
  }
  return mine;
}
template <bool F32>
__global__ void __launch_bounds__(kPartThreads) softmax_part_kernel(const Softmax a, int parts) {
  pdl_wait();
  pdl_launch_dependents();  // behind the wait: the next launch reads logits (past L1) before its own
  const int r = blockIdx.x / parts, part = blockIdx.x % parts;
  const SoftRow<F32> row(a, r);
  const int i0 = (int)((int64_t)row.chunks * part / parts), i1 = (int)((int64_t)row.chunks * (part + 1) / parts);
  SoftPart mine = row.whole(i0, i1) ? part_of<F32, true>(row, i0, i1) : part_of<F32, false>(row, i0, i1);
  mine = cta_join<kPartThreads>(mine, row.temp, row.c);
  if (threadIdx.x == 0) static_cast<SoftPart*>(a.workspace)[blockIdx.x] = mine;
}

// v: the first batch.
template <bool F32, bool kWhole, bool kPlain>
__device__ __forceinline__ void put(const SoftRow<F32>& row, int i0, int i1, Chunk<F32> (&v)[kBatch], const Base& base, float inv) {
  for (int i = i0 + threadIdx.x; i < i1; i += kPartThreads * kBatch) {
    store_batch<F32, kPartThreads, kWhole, kPlain>(row, i, i1, v, base, inv);
    load_batch<F32, kPartThreads, kWhole>(row, i + kPartThreads * kBatch, i1, v);
  }
}
template <bool F32>
__global__ void __launch_bounds__(kPartThreads) softmax_join_kernel(const Softmax a, int parts) {
  __shared__ SoftPart joined;
  pdl_launch_dependents();
  // From the last part to the first: what the first launch read last is in L2.
  const int id = gridDim.x - 1 - blockIdx.x, r = id / parts, part = id % parts, lane = threadIdx.x % 32;
  const SoftRow<F32> row(a, r);
  const int i0 = (int)((int64_t)row.chunks * part / parts), i1 = (int)((int64_t)row.chunks * (part + 1) / parts);
  const bool whole = row.whole(i0, i1);
  Chunk<F32> v[kBatch];
  if (row.temp != 0.0f) {
    if (whole) load_batch<F32, kPartThreads, true>(row, i0 + threadIdx.x, i1, v);
    else load_batch<F32, kPartThreads, false>(row, i0 + threadIdx.x, i1, v);
  }
  pdl_wait();
  if (threadIdx.x < 32) {
    const int4* of = static_cast<const int4*>(a.workspace) + (int64_t)r * parts;
    SoftPart all = {-INFINITY, 0.0f, kNone, 0};
    for (int p = lane; p < parts; p += 32) {
      const int4 u = of[p];
      all = join(all, {__int_as_float(u.x), __int_as_float(u.y), u.z, 0}, row.c);
    }
    all = warp_join(all, row.c);
    if (lane == 0) joined = all;
  }
  __syncthreads();
  const SoftPart all = joined;
  const Base base(all.m, row.c);
  const float inv = all.m == -INFINITY ? 0.0f : base.factor / all.s;
  if (row.temp == 0.0f) {
    for (int i = i0 + threadIdx.x; i < i1; i += kPartThreads)
      if (whole) row.template one_hot<true>(i, all);
      else row.template one_hot<false>(i, all);
  } else if (whole && base.plain) {
    put<F32, true, true>(row, i0, i1, v, base, inv);
  } else if (base.plain) {
    put<F32, false, true>(row, i0, i1, v, base, inv);
  } else {
    put<F32, false, false>(row, i0, i1, v, base, inv);
  }
}

// CTAs of a cluster that has a row in registers, 0: no clusters. One launch saves 3 us of host time, and up to 256 CTAs GPU time too; more
// clusters than the GPU starts at once do not, nor (up to 100 rows) pairs that are more than one CTA an SM. Fewer CTAs a row where they are more than
// 128. fp16, us with clusters / in two launches: 128256 logits a row: 1 row 4.7 / 4.5, 4 rows 4.7 / 5.2, 8 rows 5.4 / 6.5, 32 rows 7.4 / 7.8, 40 rows
// 9.9 / 9.4; 65000 logits: 32 rows 5.6 / 6.6, 64 rows 7.1 / 8.2, 85 rows 10.1 / 10.0; 32003 logits: 32 rows 5.5 / 6.4, 64 rows 6.6 / 7.4, 85 rows (pairs)
// 8.7 / 8.3 and in fp32 9.3 / 7.9, 128 rows 9.0 / 11.2 and in fp32 9.7 / 10.9 (not taken: 152 CTAs are the border). Clusters of 16 / of 8: 4 rows of
// 128256 4.7 / 5.3, 8 rows 6.0 / 5.4.
int soft_cluster(int rows, int V) {
  const int chunks = (V + 14) / 8;
  auto fits = [&](int cluster) { return chunks <= cluster * kClusterThreads * kBatch; };
  if (fits(1)) return 0;
  int c = rows <= 4 ? 16 : 8;
  while (c > 2 && c * rows > 128 && fits(c / 2)) c /= 2;
  if (!fits(c) && rows <= 8) c = 16;
  return fits(c) && (int64_t)c * rows <= (c == 2 ? 152 : 256) ? c : 0;
}

// Parts of a row, 0: one CTA or one cluster has a whole one.
int soft_parts(int rows, int V) {
  const int chunks = (V + 14) / 8;
  if (soft_cluster(rows, V)) return 0;
  return chunks <= 512 * kBatch ? 0 : row_parts(rows, chunks, 256, 2048);
}

// ---------------------------------------------------------------------------------
// Verification.  Every CTA of a sequence finds the first rejected token by itself and sums its part of the row to draw
// from, each warp a run of it; the second launch has a CTA for each sequence, which finds the run, then the element.
//
// Probabilities are whole numbers of 2^-60 (held to 0..1, rounded to nearest): sums are exact in any order, and the drawn
// token does not hang on how the row was cut. A row may add up to just below 16. A number is taken apart by fp32
// additions: x + 8 has its last place at 2^-20, and what that leaves of x goes on to 1.5 * 2^-17 (2^-40) and 1.5 * 2^-37 (2^-60);
// the sums' bits, less those of the constants, count the places. (Shifts of the mantissa take half as many instructions again.)
// ---------------------------------------------------------------------------------
constexpr int kVerifyWarps = 8, kVerifyThreads = kVerifyWarps * 32;
constexpr int kMostSteps = 16;  // of 32 chunks, in the longest run

struct Places {  // bits of the three sums
  uint32_t at[3];
};
__device__ __forceinline__ Places places(float v) {
  const float c[3] = {8.0f, 1.5f / 131072.0f, 1.5f / 137438953472.0f};
  Places r;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const float s = v + c[i];
    r.at[i] = __float_as_uint(s);
    v -= s - c[i];
  }
  return r;
}
__device__ __forceinline__ Places zero_places() {
  return {{__float_as_uint(8.0f), __float_as_uint(1.5f / 131072.0f), __float_as_uint(1.5f / 137438953472.0f)}};
}
// The number that counts of the three places stand for (the constants' bits taken off, or cancelled).
__device__ __forceinline__ int64_t placed(int32_t a, int32_t b, int32_t c) {
  return ((int64_t)a << 40) + ((int64_t)b << 20) + (int64_t)c;
}

// A random number, held to [0, 1): the largest is 1 - 2^-24.
__device__ __forceinline__ float unit(float u) { return fminf(__saturatef(u), 0.99999994f); }

// floor(total * u), u in [0, 1)
__device__ __forceinline__ uint64_t scaled(uint64_t total, float u) {
  const uint32_t b = __float_as_uint(unit(u));
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
  int V, not_this;     // not_this: the rejected token without draft rows, else no element
  int skew, chunks;
  bool rejected, alike;
  __device__ __forceinline__ DrawRow(const Verify& a, int b, int s0, int n, int accepted) : V(a.V) {
    rejected = accepted < n;
    const int64_t p_at = (int64_t)(s0 + b + accepted) * a.target_stride, q_at = (int64_t)(s0 + accepted) * a.draft_stride;
    p = a.target + p_at;
    q = rejected && a.draft ? a.draft + q_at : nullptr;
    not_this = rejected && !a.draft ? a.tokens[s0 + accepted] : -100;
    skew = (int)(p_at & 3);
    alike = (q_at & 3) == skew;
    chunks = (V + skew + 3) / 4;
  }
  __device__ __forceinline__ void without_draft() { q = nullptr, not_this = -100; }
  __device__ __forceinline__ void load4(const float* row, int c, bool whole, float (&v)[4]) const {
    const int j = 4 * c - skew;
    if (whole && j >= 0 && j + 4 <= V) {
      const float4 x = __ldcg(reinterpret_cast<const float4*>(row + j));
      v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = j + i >= 0 && j + i < V ? __ldcg(row + j + i) : 0.0f;
    }
  }
  // p and q of chunk c, zeros when not `live`. kAny: any row; kPair: the chunk lies within the row, and q alike; kAlone: the same,
  // without q.
  enum Mode { kAny, kPair, kAlone };
  template <int kMode>
  __device__ __forceinline__ void load(int c, bool live, float (&pv)[4], float (&qv)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) pv[i] = qv[i] = 0.0f;
    if (!live) return;
    if constexpr (kMode != kAny) {
      const float4 x = __ldcg(reinterpret_cast<const float4*>(p + 4 * c - skew));
      pv[0] = x.x, pv[1] = x.y, pv[2] = x.z, pv[3] = x.w;
      if constexpr (kMode == kPair) {
        const float4 y = __ldcg(reinterpret_cast<const float4*>(q + 4 * c - skew));
        qv[0] = y.x, qv[1] = y.y, qv[2] = y.z, qv[3] = y.w;
      }
    } else {
      load4(p, c, true, pv);
      if (q) load4(q, c, alike, qv);
    }
  }
  // s += the places of max(p - q, 0): those of p less those of q, or of 0, where p is the larger
  template <int kMode>
  static __device__ __forceinline__ void add(float pj, float qj, uint32_t (&s)[3]) {
    pj = __saturatef(pj);  // NaN: 0
    const Places x = places(pj), y = kMode == kAlone ? zero_places() : places(fminf(pj, __saturatef(qj)));
#pragma unroll
    for (int j = 0; j < 3; ++j) s[j] += x.at[j] - y.at[j];
  }
  __device__ __forceinline__ uint64_t weight64(int c, int i, float pj, float qj) const {
    uint32_t s[3] = {0, 0, 0};
    if (4 * c - skew + i != not_this) add<kAny>(pj, qj, s);
    return (uint64_t)placed((int32_t)s[0], (int32_t)s[1], (int32_t)s[2]);
  }
};

__device__ __forceinline__ void sequence(const Verify& a, int b, int& s0, int& n) {
  s0 = min(max(a.start[b], 0), a.drafted);
  n = min(max(a.start[b + 1], s0), a.drafted) - s0;
}

// Chunks of a warp's run of a part.
__host__ __device__ __forceinline__ int run_chunks(int chunks, int parts) {
  const int each = (chunks + parts - 1) / parts;
  return (each + kVerifyWarps * 32 - 1) / (kVerifyWarps * 32) * 32;
}

// This warp's sum of the run c0 .. c1 - 1, in all lanes.
template <int kMode>
__device__ __forceinline__ uint64_t run_sum_of(const DrawRow& row, int c0, int c1) {
  int64_t sum = 0;
  for (int c = c0 + threadIdx.x % 32; c < c1; c += 32 * 4) {
    float pv[4][4], qv[4][4];
#pragma unroll
    for (int k = 0; k < 4; ++k) row.load<kMode>(c + k * 32, c + k * 32 < c1, pv[k], qv[k]);
    uint32_t s[3] = {0, 0, 0};  // 16 numbers of up to 2^20 places
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) DrawRow::add<kMode>(pv[k][i], qv[k][i], s);
    sum += placed((int32_t)s[0], (int32_t)s[1], (int32_t)s[2]);
  }
  return warp_sum((uint64_t)sum);
}
__device__ __forceinline__ uint64_t run_sum(const DrawRow& row, int c0, int c1) {
  const bool whole = 4 * c0 - row.skew >= 0 && 4 * c1 - row.skew <= row.V;
  uint64_t sum = whole && !row.q      ? run_sum_of<DrawRow::kAlone>(row, c0, c1)
                 : whole && row.alike ? run_sum_of<DrawRow::kPair>(row, c0, c1)
                                      : run_sum_of<DrawRow::kAny>(row, c0, c1);
  // the rejected token without draft rows
  const int c = (row.not_this + row.skew) / 4, i = (row.not_this + row.skew) % 4;
  if (row.not_this >= 0 && row.not_this < row.V && c >= c0 && c < c1) {
    DrawRow all = row;
    all.without_draft();
    sum -= all.weight64(c, i, __ldcg(row.p + row.not_this), 0.0f);
  }
  return sum;
}

// How many of a sequence's tokens are accepted; a warp each finds it by itself.
__device__ __forceinline__ int count_accepted(const Verify& a, int b, int s0, int n, bool report, uint32_t* status) {
  const int lane = threadIdx.x % 32;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int i = i0 + lane;
    bool bad = false;
    if (i < n) {
      const int tok = a.tokens[s0 + i];
      const float u = unit(a.u_accept[s0 + i]);
      bad = true;
      if (tok >= 0 && tok < a.V) {
        const float pt = __saturatef(a.target[(int64_t)(s0 + b + i) * a.target_stride + tok]);
        const float qt = a.draft ? __saturatef(a.draft[(int64_t)(s0 + i) * a.draft_stride + tok]) : 1.0f;
        bad = !((double)u * (double)qt < (double)pt);
      } else if (report) {
        report_status(status, kStatusBadIndex);
      }
    }
    const uint32_t vote = __ballot_sync(kFull, bad);
    if (vote) return i0 + __ffs(vote) - 1;
  }
  return n;
}

__global__ void __launch_bounds__(kVerifyThreads) verify_part_kernel(const Verify a, int parts, int run, uint32_t* status) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, b = blockIdx.x / parts, part = blockIdx.x % parts;
  pdl_launch_dependents();
  pdl_wait();
  int s0, n;
  sequence(a, b, s0, n);
  const int accepted = count_accepted(a, b, s0, n, part == 0 && warp == 0, status);
  // ---- the sum of this warp's run ----
  const DrawRow row(a, b, s0, n, accepted);
  const int c0 = (part * kVerifyWarps + warp) * run;
  const uint64_t sum = run_sum(row, c0, min(c0 + run, row.chunks));
  if (lane == 0) static_cast<uint64_t*>(a.workspace)[blockIdx.x * kVerifyWarps + warp] = sum;
  if (part == 0 && threadIdx.x == 0) a.accepted[b] = accepted;
}

// The drawn element, from the sums of `runs` runs, and the sequence's tokens. `cta` of the CTAs that call this has the runs `cta` *
// kVerifyWarps .. when `share` is set (all of them do the same up to there), else the only one has all. `sums` are this CTA's alone.
__device__ __forceinline__ void draw(const Verify& a, int b, int s0, int n, int accepted, uint64_t* sums, int runs, int run, int cta, bool share,
                                     float u) {
  __shared__ uint64_t of_step[kMostSteps];
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, per = (runs + 31) / 32;
  int32_t* out = a.out + s0 + b;
  // ---- the row's total, then the run that the drawn one is in: a lane has `per` neighbouring ones. Every warp finds it by itself ----
  uint64_t mine = 0;
#pragma unroll 16
  for (int i = 0; i < per; ++i) mine += lane * per + i < runs ? sums[lane * per + i] : 0;
  DrawRow row(a, b, s0, n, accepted);
  uint64_t to = warp_scan(mine, lane), all = shfl_u64(to, 31), limit = scaled(all, u), head = 0;
  int found = -1;
  auto find = [&](int first, int end) {  // among these runs, of which `head` is the sum before
    for (int i = first; i < end && found < 0; i += 32) {
      const uint64_t x = i + lane < end ? sums[i + lane] : 0;
      to = head + warp_scan(x, lane);
      const uint32_t past = __ballot_sync(kFull, to > limit);
      if (past) {
        found = i + __ffs(past) - 1;
        head = shfl_u64(to - x, __ffs(past) - 1);
      } else {
        head = shfl_u64(to, 31);
      }
    }
  };
  if (all > 0) {
    const int from = __ffs(__ballot_sync(kFull, to > limit)) - 1;  // there is one: limit < all
    head = shfl_u64(to - mine, from);
    find(from * per, min((from + 1) * per, runs));
  } else if (row.rejected) {  // nothing left of p - q: drawn from p, whose sums one CTA takes here
    if (cta != 0) return;
    share = false;
    row.without_draft();
    __syncthreads();  // every warp has read the sums, which are 0
    for (int i = warp; i < runs; i += kVerifyWarps) {
      const uint64_t x = run_sum(row, i * run, min((i + 1) * run, row.chunks));
      if (lane == 0) sums[i] = x;
    }
    __syncthreads();
    for (int i = lane; i < runs; i += 32) all += sums[i];
    all = warp_sum(all);
    limit = scaled(all, u);
    if (all > 0) find(0, runs);
  }
  if (cta == 0)
    for (int i = tid; i <= n; i += kVerifyThreads)
      if (i != accepted || found < 0) out[i] = i < accepted ? a.tokens[s0 + i] : -1;
  if (found < 0 || (share && found / kVerifyWarps != cta)) return;
  // ---- the element: the warps take the run's steps of 32 chunks in turn ----
  constexpr int kMine = kMostSteps / kVerifyWarps;
  const int steps = run / 32;
  float pv[kMine][4], qv[kMine][4];
  uint64_t sum[kMine];
#pragma unroll
  for (int k = 0; k < kMine; ++k) {
    const int s = k * kVerifyWarps + warp, c = found * run + 32 * s + lane;
    row.load<DrawRow::kAny>(c, s < steps && c < row.chunks, pv[k], qv[k]);
  }
#pragma unroll
  for (int k = 0; k < kMine; ++k) {
    const int s = k * kVerifyWarps + warp, c = found * run + 32 * s + lane;
    sum[k] = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[k] += row.weight64(c, i, pv[k][i], qv[k][i]);
    const uint64_t total = warp_sum(sum[k]);
    if (lane == 0) of_step[s] = total;
  }
  __syncthreads();
  const uint64_t x = lane < kMostSteps ? of_step[lane] : 0;
  to = head + warp_scan(x, lane);
  const int step = __ffs(__ballot_sync(kFull, to > limit)) - 1;
  head = shfl_u64(to - x, max(step, 0));
#pragma unroll
  for (int k = 0; k < kMine; ++k) {
    if (step == k * kVerifyWarps + warp) {
      const int c = found * run + 32 * step + lane;
      to = head + warp_scan(sum[k], lane);
      const uint32_t past = __ballot_sync(kFull, to > limit);
      if (past && lane == __ffs(past) - 1) {
        uint64_t s = to - sum[k];
        int at = -1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s += row.weight64(c, i, pv[k][i], qv[k][i]);
          if (at < 0 && s > limit) at = i;
        }
        out[accepted] = 4 * c - row.skew + at;
      }
    }
  }
}

__global__ void __launch_bounds__(kVerifyThreads) verify_draw_kernel(const Verify a, int parts, int run) {
  const int b = blockIdx.x, runs = parts * kVerifyWarps;
  pdl_launch_dependents();
  pdl_wait();
  int s0, n;
  sequence(a, b, s0, n);
  const int accepted = min(max(a.accepted[b], 0), n);  // the first launch's: in range unless the caller's buffers overlap
  draw(a, b, s0, n, accepted, static_cast<uint64_t*>(a.workspace) + (int64_t)b * runs, runs, run, 0, false, a.u_next[b]);
}

// Few sequences: a cluster of CTAs has one, whose sums they hand to each other.
__global__ void __launch_bounds__(kVerifyThreads) verify_cluster_kernel(const Verify a, int cluster, int run, uint32_t* status) {
  __shared__ __align__(16) uint64_t sums[kMostCluster * kVerifyWarps];
  cluster_arrive();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, b = blockIdx.x / cluster, cta = cluster_ctarank();
  pdl_launch_dependents();
  pdl_wait();
  int s0, n;
  sequence(a, b, s0, n);
  const float u = a.u_next[b];
  const int accepted = count_accepted(a, b, s0, n, cta == 0 && warp == 0, status);
  const DrawRow row(a, b, s0, n, accepted);
  const int at = cta * kVerifyWarps + warp, c0 = at * run;
  const uint64_t sum = run_sum(row, c0, min(c0 + run, row.chunks));
  __syncwarp();
  cluster_wait();  // the others have started
  if (lane < cluster) cluster_st_u64(cluster_map(smem_u32(&sums[at]), lane), (uint32_t)sum, (uint32_t)(sum >> 32));
  if (cta == 0 && threadIdx.x == 0) a.accepted[b] = accepted;
  __syncwarp();
  cluster_arrive();
  cluster_wait();
  draw(a, b, s0, n, accepted, sums, cluster * kVerifyWarps, run, cta, true, u);
}

// CTAs of a cluster that has a sequence, 0: two launches. As many as give a warp a run of 64 chunks; fewer, with runs of up to 256, where
// that is more than a CTA for each SM, and of up to 512 where it is more than 512 in all. us with clusters / in two launches, 4 drafted tokens a
// sequence, all accepted (a call takes 4 us less of host time besides): V 128256: 1 sequence 6.0 / 7.7, 8 7.1 / 9.6, 32 9.3 / 9.3, 64 11.1 / 11.3, 76 (608
// CTAs) 14.3 / 11.3, 100 16.7 / 14.3; V 151936, whose runs fit clusters of 16 alone: 8 7.7 / 8.6, 32 10.2 / 9.3; V 32003: 1 5.3 / 6.5, 64 7.8 / 8.4, 100 8.8 /
// 9.7, 200 11.4 / 11.7. With rows of q to subtract: V 128256: 64 14.0 / 14.4, 72 14.1 / 15.5, 80 16.8 / 16.7, 96 20.5 / 18.3.
int verify_cluster(int batch, int V) {
  const int chunks = (V + 6) / 4;
  int c = kMostCluster;
  while (c > 1 && c * kVerifyWarps * 64 > chunks) c /= 2;
  while (c > 1 && c * batch > 152 && run_chunks(chunks, c / 2) <= 256) c /= 2;
  while (c > 1 && c * batch > 512 && run_chunks(chunks, c / 2) <= 32 * kMostSteps) c /= 2;
  return run_chunks(chunks, c) <= 32 * kMostSteps && (int64_t)c * batch <= 512 ? c : 0;
}
int verify_parts(int batch, int V) {
  return verify_cluster(batch, V) ? 0 : row_parts(batch, (V + 6) / 4, 512, kVerifyThreads * kMostSteps);
}

}  // namespace

size_t softmax_workspace_bytes(int rows, int V) { return (size_t)rows * soft_parts(rows, V) * sizeof(SoftPart); }
size_t verify_workspace_bytes(int batch, int V) { return (size_t)batch * verify_parts(batch, V) * kVerifyWarps * sizeof(uint64_t); }

cudaError_t launch_softmax(LaunchCtx& ctx, const Softmax& a) {
  ctx.variant = a.f32 ? "softmax_f32" : "softmax_f16";
  const int parts = soft_parts(a.rows, a.V);
  if (const int cluster = soft_cluster(a.rows, a.V)) {
    auto go = [&](auto kern, std::atomic<uint64_t>& wide) {
      const cudaError_t e = cluster > 8 ? allow_wide_clusters(kern, ctx.device, wide) : cudaSuccess;
      return e != cudaSuccess ? e : launch_clusters(ctx, kern, cluster, dim3((unsigned)(a.rows * cluster)), dim3(kClusterThreads), 0, a, cluster);
    };
    static std::atomic<uint64_t> wide[2] = {};
    return a.f32 ? go(softmax_cluster_kernel<true>, wide[1]) : go(softmax_cluster_kernel<false>, wide[0]);
  }
  if (parts == 0) {
    const bool few = (a.V + 14) / 8 <= 128 * kBatch;
    auto go = [&](auto kern, int threads) { return launch_kernel(ctx, kern, dim3(a.rows), dim3(threads), 0, a); };
    if (few) return a.f32 ? go(softmax_row_kernel<true, 128>, 128) : go(softmax_row_kernel<false, 128>, 128);
    return a.f32 ? go(softmax_row_kernel<true, 512>, 512) : go(softmax_row_kernel<false, 512>, 512);
  }
  const dim3 grid((unsigned)a.rows * parts);
  cudaError_t e = a.f32 ? launch_kernel(ctx, softmax_part_kernel<true>, grid, dim3(kPartThreads), 0, a, parts)
                        : launch_kernel(ctx, softmax_part_kernel<false>, grid, dim3(kPartThreads), 0, a, parts);
  if (e != cudaSuccess) return e;
  const bool pdl = ctx.pdl;
  ctx.pdl = true;  // the second launch waits for the first one on the device
  e = a.f32 ? launch_kernel(ctx, softmax_join_kernel<true>, grid, dim3(kPartThreads), 0, a, parts)
            : launch_kernel(ctx, softmax_join_kernel<false>, grid, dim3(kPartThreads), 0, a, parts);
  ctx.pdl = pdl;
  return e;
}

cudaError_t launch_verify(LaunchCtx& ctx, const Verify& a) {
  ctx.variant = "verify";
  if (const int cluster = verify_cluster(a.batch, a.V)) {
    static std::atomic<uint64_t> wide{0};
    const cudaError_t e = cluster > 8 ? allow_wide_clusters(verify_cluster_kernel, ctx.device, wide) : cudaSuccess;
    return e != cudaSuccess ? e
                            : launch_clusters(ctx, verify_cluster_kernel, cluster, dim3((unsigned)(a.batch * cluster)), dim3(kVerifyThreads), 0,
                                              a, cluster, run_chunks((a.V + 6) / 4, cluster), ctx.status);
  }
  const int parts = verify_parts(a.batch, a.V), run = run_chunks((a.V + 6) / 4, parts);
  cudaError_t e = launch_kernel(ctx, verify_part_kernel, dim3((unsigned)a.batch * parts), dim3(kVerifyThreads), 0, a, parts, run,
                                ctx.status);
  if (e != cudaSuccess) return e;
  const bool pdl = ctx.pdl;
  ctx.pdl = true;
  e = launch_kernel(ctx, verify_draw_kernel, dim3(a.batch), dim3(kVerifyThreads), 0, a, parts, run);
  ctx.pdl = pdl;
  return e;
}

}  // namespace mnb
