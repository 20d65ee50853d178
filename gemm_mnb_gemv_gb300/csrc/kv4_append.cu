// Append to, and read back from, the paged 4-bit key/value cache.
//
// Append: y = R(pos) x for q and k (pairs (a, b) -> (a c - b s, b c + a s)), then per group of
// K and V: offset = fp16(min), scale = fp16((max - min) / 15), code = rint((x - offset) / scale).
// A block takes one token in passes over its heads: q with 16 elements a lane, both sides of eight
// pairs, so that each element is converted and each table entry loaded once; k and v with 8 consecutive
// elements a lane, which are one 32-bit K word (or two 16-bit halves of V words), the rotation's
// partners by a second load that hits L1, extrema by shuffles over a group's 4-16 lanes. The
// passes' loads are all issued before the token's position is waited for.
// Measured, 16381 tokens of 32 / 8 heads of 128, graph replays: fp16 append 95.6 us, read 29.3 (their bytes alone 53.2 and 12.5); fp32
// 121 and 35.5 (103 and 22.4). The first form, one pass shape for q, k and v, took 177 us for both in fp16.
// Bound, fp16 append: neither bytes (3.4 TB/s) nor issue alone: 67.8 M warp instructions (4140 a token) fill 58% of the issue slots,
// and 16 warps an SM (128 registers) leave the rest to fixed latencies and loads. The fp32 append is bound by its bytes.
// Read: one block for four tokens; slot, code and store one after the other, without a second round to hide behind.
#include <type_traits>

#include "kv4.cuh"
#include "mnb_device.cuh"
#include "mnb_internal.h"

namespace mnb {
namespace {

struct V8 {
  float x[8];
};

template <bool F32>
__device__ __forceinline__ V8 load8(const void* base, int64_t i) {
  V8 r;
  if constexpr (F32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
    const float4 a = p[0], b = p[1];
    r.x[0] = a.x, r.x[1] = a.y, r.x[2] = a.z, r.x[3] = a.w;
    r.x[4] = b.x, r.x[5] = b.y, r.x[6] = b.z, r.x[7] = b.w;
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const __half*>(base) + i);
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[j]));
      r.x[2 * j] = f.x, r.x[2 * j + 1] = f.y;
    }
  }
  return r;
}

template <bool F32>
__device__ __forceinline__ void store8(void* base, int64_t i, const V8& v) {
  if constexpr (F32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + i);
    p[0] = make_float4(v.x[0], v.x[1], v.x[2], v.x[3]);
    p[1] = make_float4(v.x[4], v.x[5], v.x[6], v.x[7]);
  } else {
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __half2 h = __floats2half2_rn(v.x[2 * j], v.x[2 * j + 1]);
      u[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(static_cast<__half*>(base) + i) = make_uint4(u[0], u[1], u[2], u[3]);
  }
}

// 8 elements as they lie: 16 bytes of fp16 or 32 of fp32.
template <bool F32>
struct Raw8 {
  uint4 v[F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* base, int64_t i) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base) + i * (F32 ? 4 : 2));
    v[0] = p[0];
    if constexpr (F32) v[1] = p[1];
  }
  __device__ __forceinline__ V8 get() const {
    V8 r;
#pragma unroll
    for (int j = 0; j < (F32 ? 2 : 1); ++j) {
      const uint32_t u[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (F32) {
          r.x[4 * j + k] = __uint_as_float(u[k]);
        } else {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[k]));
          r.x[2 * k] = f.x, r.x[2 * k + 1] = f.y;
        }
      }
    }
    return r;
  }
};

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

// Page and place of a slot within the cache's capacity: 32 bits where they do.
__device__ __forceinline__ void split_slot(int64_t slot, int page_size, int64_t& page, int& in_page) {
  if (slot >> 32 == 0) {
    const uint32_t p = (uint32_t)slot / (uint32_t)page_size;
    page = p;
    in_page = (int)((uint32_t)slot - p * (uint32_t)page_size);
  } else {
    page = slot / page_size;
    in_page = (int)(slot - page * page_size);
  }
}

constexpr int kAppendThreads = 128;

// Passes of a block of kAppendThreads over one token's heads: q first, then k, then v.
template <int D>
struct Passes {
  static constexpr int kQLanes = D / 16, kLanes = D / 8;
  static constexpr int kQHeads = kAppendThreads / kQLanes, kHeads = kAppendThreads / kLanes;  // heads a pass
  int q, kv;
  __host__ __device__ Passes(int q_heads, int kv_heads)
      : q((q_heads + kQHeads - 1) / kQHeads), kv((kv_heads + kHeads - 1) / kHeads) {}
  __host__ __device__ int count() const { return q + 2 * kv; }
};

// q_out may be q itself: a lane loads both of its chunks before it stores either, and no other lane
// reads them.
template <int D, bool F32, int kU>
__global__ void __launch_bounds__(kAppendThreads) kv4_append_kernel(const Kv4Cache c, const Kv4Append a, uint32_t* status) {
  pdl_wait();
  using P = Passes<D>;
  constexpr int kLanes = P::kLanes;
  const P passes(a.q_heads, c.kv_heads);
  const int tid = threadIdx.x;
  const int gl = c.group / 8;  // lanes of a group: 4, 8 or 16
  // q: the lane's two chunks of 8 elements. Rotated elements come first, half-split pairs as one chunk of each side.
  const int qj = tid % P::kQLanes, half = a.rot / 2;
  const bool q_turns = 16 * qj < a.rot;
  const int q0 = q_turns && !a.interleaved ? 8 * qj : 16 * qj, q1 = q_turns && !a.interleaved ? q0 + half : q0 + 8;
  // k, v: one chunk, and for k its partners (half-split)
  const int sub = tid % kLanes, d = 8 * sub;
  const bool k_turns = d < a.rot;
  const int partner = d < half ? d + half : d - half;
  const int64_t capacity = (int64_t)c.num_pages * c.page_size;
  int64_t slot = a.slots[blockIdx.x];
  int pos = a.rot ? a.positions[blockIdx.x] : 0;
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
  const int64_t slot_now = slot;
  const int pos_now = pos;
  if (t + gridDim.x < a.T) {  // the next token's numbers are on their way while this one is worked on
    slot = a.slots[t + gridDim.x];
    if (a.rot) pos = a.positions[t + gridDim.x];
  }
  bool known = false, store = false, pos_ok = true;
  int r = 0;
  uint8_t* blk0 = nullptr;  // the token's block of key head 0
  V8 qc = {}, qs = {}, kc = {}, ks = {};
  for (int p0 = blockIdx.y; p0 < passes.count(); p0 += kU * gridDim.y) {
    Raw8<F32> x[kU][2];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int p = p0 + u * gridDim.y;
      if (p < passes.q) {
        const int h = p * P::kQHeads + tid / P::kQLanes;
        if (h < a.q_heads) {
          const int64_t at = t * a.q_stride + (int64_t)h * D;
          x[u][0].load(a.q, at + q0);
          x[u][1].load(a.q, at + q1);
        }
      } else if (p < passes.count()) {
        const bool is_k = p < passes.q + passes.kv;
        const int h = (p - passes.q - (is_k ? 0 : passes.kv)) * P::kHeads + tid / kLanes;
        if (h < c.kv_heads) {
          const int64_t at = t * (is_k ? a.k_stride : a.v_stride) + (int64_t)h * D;
          x[u][0].load(is_k ? a.k : a.v, at + d);
          if (is_k && k_turns && !a.interleaved) x[u][1].load(a.k, at + partner);
        }
      }
    }
    if (!known) {  // the token's own numbers
      known = true;
      pos_ok = a.rot == 0 || (pos_now >= 0 && pos_now < a.rows);
      store = slot_now >= 0 && slot_now < capacity && pos_ok;
      if (tid == 0 && blockIdx.y == 0 && (slot_now >= capacity || !pos_ok)) report_status(status, kStatusBadIndex);
      if (a.rot && pos_ok) {
        const float *cos = a.cos + (int64_t)pos_now * half, *sin = a.sin + (int64_t)pos_now * half;
        if (q_turns) qc = load8<true>(cos, 8 * qj), qs = load8<true>(sin, 8 * qj);
        if (k_turns) {
          // interleaved: pairs d / 2 .. d / 2 + 3, the first four values
          const int i = a.interleaved ? d / 2 : d < half ? d : d - half;
          if (a.interleaved) {
            const float4 cv = *reinterpret_cast<const float4*>(cos + i), sv = *reinterpret_cast<const float4*>(sin + i);
            kc.x[0] = cv.x, kc.x[1] = cv.y, kc.x[2] = cv.z, kc.x[3] = cv.w;
            ks.x[0] = sv.x, ks.x[1] = sv.y, ks.x[2] = sv.z, ks.x[3] = sv.w;
          } else {
            kc = load8<true>(cos, i), ks = load8<true>(sin, i);
          }
        }
      }
      if (store) {
        int64_t page;
        int in_page;
        split_slot(slot_now, c.page_size, page, in_page);
        r = in_page % 16;
        blk0 = c.pages + page * c.kv_heads * c.head_bytes() + (in_page / 16) * c.block_bytes();
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int p = p0 + u * gridDim.y;
      if (p >= passes.count()) break;
      if (p < passes.q) {
        const int h = p * P::kQHeads + tid / P::kQLanes;
        if (h >= a.q_heads) continue;
        V8 y0 = x[u][0].get(), y1 = x[u][1].get();
        if (q_turns) {
          if (a.interleaved) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float a0 = y0.x[2 * i], b0 = y0.x[2 * i + 1], a1 = y1.x[2 * i], b1 = y1.x[2 * i + 1];
              y0.x[2 * i] = __fsub_rn(__fmul_rn(a0, qc.x[i]), __fmul_rn(b0, qs.x[i]));
              y0.x[2 * i + 1] = __fadd_rn(__fmul_rn(b0, qc.x[i]), __fmul_rn(a0, qs.x[i]));
              y1.x[2 * i] = __fsub_rn(__fmul_rn(a1, qc.x[4 + i]), __fmul_rn(b1, qs.x[4 + i]));
              y1.x[2 * i + 1] = __fadd_rn(__fmul_rn(b1, qc.x[4 + i]), __fmul_rn(a1, qs.x[4 + i]));
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float av = y0.x[i], bv = y1.x[i];
              y0.x[i] = __fsub_rn(__fmul_rn(av, qc.x[i]), __fmul_rn(bv, qs.x[i]));
              y1.x[i] = __fadd_rn(__fmul_rn(bv, qc.x[i]), __fmul_rn(av, qs.x[i]));
            }
          }
        }
        if (!pos_ok) y0 = y1 = V8{};
        const int64_t at = ((int64_t)t * a.q_heads + h) * D;
        store8<F32>(a.q_out, at + q0, y0);
        store8<F32>(a.q_out, at + q1, y1);
        continue;
      }
      const bool is_k = p < passes.q + passes.kv;
      const int h = (p - passes.q - (is_k ? 0 : passes.kv)) * P::kHeads + tid / kLanes;
      V8 y = h < c.kv_heads ? x[u][0].get() : V8{};
      if (is_k && k_turns) {
        if (a.interleaved) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float av = y.x[2 * i], bv = y.x[2 * i + 1];
            y.x[2 * i] = __fsub_rn(__fmul_rn(av, kc.x[i]), __fmul_rn(bv, ks.x[i]));
            y.x[2 * i + 1] = __fadd_rn(__fmul_rn(bv, kc.x[i]), __fmul_rn(av, ks.x[i]));
          }
        } else if (h < c.kv_heads) {
          const V8 z = x[u][1].get();
          const float sign = d < half ? -1.0f : 1.0f;  // exact: a c - b s or b c + a s
#pragma unroll
          for (int i = 0; i < 8; ++i) y.x[i] = __fadd_rn(__fmul_rn(y.x[i], kc.x[i]), sign * __fmul_rn(z.x[i], ks.x[i]));
        }
      }
      float lo = y.x[0], hi = y.x[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) lo = min_nan(lo, y.x[i]), hi = max_nan(hi, y.x[i]);
      for (int o = 1; o < gl; o <<= 1) {
        lo = min_nan(lo, __shfl_xor_sync(kFull, lo, o));
        hi = max_nan(hi, __shfl_xor_sync(kFull, hi, o));
      }
      if (h >= c.kv_heads || !store) continue;
      const bool finite = fabsf(lo) < INFINITY && fabsf(hi) < INFINITY;
      const __half offset = finite ? __float2half_rn(fminf(fmaxf(lo, -65504.0f), 65504.0f)) : __ushort_as_half(0x7fff);
      const __half scale = finite ? __float2half_rn(fminf(__fmul_rn(__fsub_rn(hi, lo), 1.0f / 15.0f), 65504.0f))
                                  : __ushort_as_half(0x7fff);
      const float sf = __half2float(scale);
      const float of = finite ? __half2float(offset) : 0.0f;
      const float inv = sf > 0.0f ? __frcp_rn(sf) : 0.0f;
      // 1.5 2^23 + x has the integer nearest to x, ties to even, in its low bits; what lies above a code's
      // 4 bits is the same for every element and goes with one subtraction. fmaxf turns a NaN into 0.
      uint32_t word = 0;
#pragma unroll
      for (int i = 7; i >= 0; --i) {
        const float f = fminf(fmaxf(__fmul_rn(__fsub_rn(y.x[i], of), inv), 0.0f), 15.0f);
        word = (word << 4) + __float_as_uint(__fadd_rn(f, 12582912.0f));
      }
      word -= 0x4B400000u * 0x11111111u;
      uint8_t* blk = blk0 + h * c.head_bytes();
      if (is_k) {
        *reinterpret_cast<uint32_t*>(blk + kv4::k_word_byte<D>(r, sub % 4, sub / 4)) = word;
      } else {
        uint8_t* vb = blk + 8 * D;
        const int g = sub % 4 * 2, hw = (sub >> 2 & 1) * 2;
        *reinterpret_cast<uint16_t*>(vb + kv4::v_word_byte<D>(g, r, sub / 8) + hw) = (uint16_t)word;
        *reinterpret_cast<uint16_t*>(vb + kv4::v_word_byte<D>(g + 1, r, sub / 8) + hw) = (uint16_t)(word >> 16);
      }
      if (sub % gl == 0)
        *reinterpret_cast<__half2*>(blk + 16 * D + ((is_k ? 0 : c.ng() * 16) + sub / gl * 16 + r) * 4) =
            __halves2half2(scale, offset);
    }
  }
  }
}

constexpr int kReadThreads = 256;

// kU tokens a lane in flight: slot, then code and parameters, then the store.
template <int D, bool F32, int kU>
__global__ void __launch_bounds__(kReadThreads) kv4_read_kernel(const Kv4Cache c, const int64_t* slots, int T, void* k_out,
                                                       void* v_out, uint32_t* status) {
  pdl_wait();
  constexpr int kLanes = D / 8;
  const int t0 = blockIdx.x * kU;
  const int sub = threadIdx.x % kLanes;
  const int64_t capacity = (int64_t)c.num_pages * c.page_size;
  const int per = blockDim.x / kLanes, ng = c.ng(), gl = c.group / 8;
  int64_t at0[kU];  // of the token's block of key head 0, -1: zeros
  int r[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int64_t slot = t0 + u < T ? slots[t0 + u] : -1;
    if (threadIdx.x == 0 && blockIdx.y == 0 && slot >= capacity) report_status(status, kStatusBadIndex);
    at0[u] = -1;
    r[u] = 0;
    if (slot >= 0 && slot < capacity) {
      int64_t page;
      int in_page;
      split_slot(slot, c.page_size, page, in_page);
      r[u] = in_page % 16;
      at0[u] = page * c.kv_heads * c.head_bytes() + (in_page / 16) * c.block_bytes();
    }
  }
  for (int h = blockIdx.y * per + threadIdx.x / kLanes; h < 2 * c.kv_heads; h += gridDim.y * per) {
    const bool is_k = h < c.kv_heads;
    const int kvh = is_k ? h : h - c.kv_heads;
    const int64_t head = kvh * c.head_bytes();
    uint32_t word[kU], par[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      word[u] = par[u] = 0;
      if (at0[u] < 0) continue;
      const uint8_t* blk = c.pages + at0[u] + head;
      if (is_k) {
        word[u] = *reinterpret_cast<const uint32_t*>(blk + kv4::k_word_byte<D>(r[u], sub % 4, sub / 4));
      } else {
        const uint8_t* vb = blk + 8 * D;
        const int g = sub % 4 * 2, hw = (sub >> 2 & 1) * 2;
        word[u] = *reinterpret_cast<const uint16_t*>(vb + kv4::v_word_byte<D>(g, r[u], sub / 8) + hw) |
                  (uint32_t)*reinterpret_cast<const uint16_t*>(vb + kv4::v_word_byte<D>(g + 1, r[u], sub / 8) + hw) << 16;
      }
      par[u] = *reinterpret_cast<const uint32_t*>(blk + 16 * D + ((is_k ? 0 : ng * 16) + sub / gl * 16 + r[u]) * 4);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (t0 + u >= T) continue;
      const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&par[u]));
      V8 y;
#pragma unroll
      for (int i = 0; i < 8; ++i)  // 2^23 + c has the code in its low bits
        y.x[i] = fmaf(__uint_as_float((word[u] >> (4 * i) & 15u) | 0x4B000000u) - 8388608.0f, p.x, p.y);
      store8<F32>(is_k ? k_out : v_out, ((int64_t)(t0 + u) * c.kv_heads + kvh) * D + sub * 8, y);
    }
  }
}

}  // namespace

// Few tokens: their passes are spread over the SMs. Many: a block takes a token's passes, four (fp32: two) in flight
// (append), or four tokens (read).
constexpr int kFewTokens = 304, kManyBlocks = 4;  // blocks an SM holds: by registers

cudaError_t launch_kv4_append(LaunchCtx& ctx, const Kv4Cache& c, const Kv4Append& a) {
  ctx.variant = "kv4_append";
  const bool few = a.T <= kFewTokens;
  auto pick = [&](auto d) {
    constexpr int D = decltype(d)::value;
    const int blocks = kManyBlocks * ctx.num_sms;
    const dim3 grid(few || a.T < blocks ? a.T : blocks, few ? Passes<D>(a.q_heads, c.kv_heads).count() : 1);
    auto go = [&](auto kern) { return launch_kernel(ctx, kern, grid, dim3(kAppendThreads), 0, c, a, ctx.status); };
    if (a.f32) return few ? go(kv4_append_kernel<D, true, 1>) : go(kv4_append_kernel<D, true, 2>);
    return few ? go(kv4_append_kernel<D, false, 1>) : go(kv4_append_kernel<D, false, 4>);
  };
  if (c.head_dim == 64) return pick(std::integral_constant<int, 64>{});
  if (c.head_dim == 128) return pick(std::integral_constant<int, 128>{});
  return pick(std::integral_constant<int, 256>{});
}

cudaError_t launch_kv4_read(LaunchCtx& ctx, const Kv4Cache& c, const int64_t* slots, int T, int f32, void* k_out,
                            void* v_out) {
  ctx.variant = "kv4_read";
  const int per = kReadThreads / (c.head_dim / 8), turns = (2 * c.kv_heads + per - 1) / per;
  const bool few = T <= kFewTokens;
  auto go = [&](auto kern, int u) {
    return launch_kernel(ctx, kern, dim3((T + u - 1) / u, turns), dim3(kReadThreads), 0, c, slots, T, k_out, v_out,
                         ctx.status);
  };
  auto pick = [&](auto d) {
    constexpr int D = decltype(d)::value;
    if (f32) return few ? go(kv4_read_kernel<D, true, 1>, 1) : go(kv4_read_kernel<D, true, 4>, 4);
    return few ? go(kv4_read_kernel<D, false, 1>, 1) : go(kv4_read_kernel<D, false, 4>, 4);
  };
  if (c.head_dim == 64) return pick(std::integral_constant<int, 64>{});
  if (c.head_dim == 128) return pick(std::integral_constant<int, 128>{});
  return pick(std::integral_constant<int, 256>{});
}

}  // namespace mnb
