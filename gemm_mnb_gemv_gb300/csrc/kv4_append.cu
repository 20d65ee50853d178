// Append to, and read back from, the paged 4-bit key/value cache.
//
// Append: y = R(pos) x for q and k (pairs (a, b) -> (a c - b s, b c + a s)), then per group of
// K and V: offset = fp16(min), scale = fp16((max - min) / 15), code = rint((x - offset) / scale).
// D / 8 lanes hold one head of one token, 8 consecutive elements each: a 16-byte load (fp16),
// the rotation partner's 8 elements by a second load that hits L1 (half-split pairs sit in
// another lane; a load costs fewer instructions than 4-8 shuffles), the group's extrema by
// shuffles over 4-16 lanes, and exactly one 32-bit K word or two 16-bit halves of V words to
// store. Bound: HBM bytes of q, k, v, q_out.
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

// Rotates the 8 elements at d of a head whose elements start at `head` (element offset into base).
template <bool F32>
__device__ __forceinline__ V8 rotate8(const V8& x, const void* base, int64_t head, int d, const float* cos,
                                      const float* sin, int rot, int interleaved) {
  if (d >= rot) return x;
  V8 y;
  const int half = rot / 2;
  if (interleaved) {
    const float4 c = *reinterpret_cast<const float4*>(cos + d / 2);
    const float4 s = *reinterpret_cast<const float4*>(sin + d / 2);
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = x.x[2 * i], b = x.x[2 * i + 1];
      y.x[2 * i] = __fsub_rn(__fmul_rn(a, cc[i]), __fmul_rn(b, ss[i]));
      y.x[2 * i + 1] = __fadd_rn(__fmul_rn(b, cc[i]), __fmul_rn(a, ss[i]));
    }
  } else {
    const bool first = d < half;
    const int i0 = first ? d : d - half;
    const V8 p = load8<F32>(base, head + (first ? d + half : d - half));
    const V8 c = load8<true>(cos, i0), s = load8<true>(sin, i0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float xc = __fmul_rn(x.x[i], c.x[i]), ps = __fmul_rn(p.x[i], s.x[i]);
      y.x[i] = first ? __fsub_rn(xc, ps) : __fadd_rn(xc, ps);
    }
  }
  return y;
}

// q_out may be q itself: each lane reads its partner's elements before any lane stores, which
// a sub-warp of lanes in step does (the __syncwarp between the two).
template <int D, bool F32>
__global__ void kv4_append_kernel(const Kv4Cache c, const Kv4Append a, uint32_t* status) {
  pdl_wait();
  constexpr int kLanes = D / 8;
  const int t = blockIdx.x;
  const int nheads = a.q_heads + 2 * c.kv_heads;
  const int sub = threadIdx.x % kLanes, d = sub * 8;
  const int64_t slot = a.slots[t];
  const int64_t capacity = (int64_t)c.num_pages * c.page_size;
  const int pos = a.rot ? a.positions[t] : 0;
  const bool pos_ok = a.rot == 0 || (pos >= 0 && pos < a.rows);
  const bool store = slot >= 0 && slot < capacity && pos_ok;
  if (threadIdx.x == 0 && blockIdx.y == 0 && (slot >= capacity || !pos_ok)) report_status(status, kStatusBadIndex);
  const float* cos = a.rot && pos_ok ? a.cos + (int64_t)pos * (a.rot / 2) : nullptr;
  const float* sin = a.rot && pos_ok ? a.sin + (int64_t)pos * (a.rot / 2) : nullptr;
  const int rot = pos_ok ? a.rot : 0;
  const int per = blockDim.x / kLanes;
  const int block_bytes = c.block_bytes(), ng = c.ng();
  // every lane of a warp runs the same number of turns (the shuffles need them all)
  for (int h0 = blockIdx.y * per; h0 < nheads; h0 += gridDim.y * per) {
    const int h = h0 + threadIdx.x / kLanes;
    const bool live = h < nheads;
    const bool is_q = h < a.q_heads, is_k = !is_q && h < a.q_heads + c.kv_heads;
    const int kvh = is_q ? 0 : is_k ? h - a.q_heads : h - a.q_heads - c.kv_heads;
    const void* base = is_q ? a.q : is_k ? a.k : a.v;
    const int64_t head = is_q ? t * a.q_stride + (int64_t)h * D : t * (is_k ? a.k_stride : a.v_stride) + (int64_t)kvh * D;
    V8 x = {};
    if (live) {
      x = load8<F32>(base, head + d);
      if (is_q || is_k) x = rotate8<F32>(x, base, head, d, cos, sin, rot, a.interleaved);
    }
    __syncwarp();
    if (live && is_q) {
      if (!pos_ok) x = V8{};
      store8<F32>(a.q_out, ((int64_t)t * a.q_heads + h) * D + d, x);
    }
    float lo = x.x[0], hi = x.x[0];
    bool finite = true;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo = fminf(lo, x.x[i]);
      hi = fmaxf(hi, x.x[i]);
      finite &= fabsf(x.x[i]) < INFINITY;
    }
    const int gl = c.group / 8;  // lanes of a group: 4, 8 or 16
    for (int o = 1; o < gl; o <<= 1) {
      lo = fminf(lo, __shfl_xor_sync(kFull, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(kFull, hi, o));
      finite = __shfl_xor_sync(kFull, (int)finite, o) && finite;
    }
    if (!live || is_q || !store) continue;
    const __half offset = finite ? __float2half_rn(fminf(fmaxf(lo, -65504.0f), 65504.0f)) : __ushort_as_half(0x7fff);
    const __half scale = finite ? __float2half_rn(fminf(__fmul_rn(__fsub_rn(hi, lo), 1.0f / 15.0f), 65504.0f))
                                : __ushort_as_half(0x7fff);
    const float of = __half2float(offset), sf = __half2float(scale);
    const float inv = sf == 0.0f || !finite ? 0.0f : __fdiv_rn(1.0f, sf);
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float f = rintf(__fmul_rn(__fsub_rn(x.x[i], of), inv));
      const uint32_t code = finite ? (uint32_t)fminf(fmaxf(f, 0.0f), 15.0f) : 0u;
      word |= code << (4 * i);
    }
    const int64_t page = slot / c.page_size;
    const int in_page = (int)(slot - page * c.page_size), r = in_page % 16;
    uint8_t* blk = c.pages + ((page * c.kv_heads + kvh) * (c.page_size / 16) + in_page / 16) * block_bytes;
    if (is_k) {
      *reinterpret_cast<uint32_t*>(blk + kv4::k_word_byte<D>(r, sub % 4, sub / 4)) = word;
    } else {
      uint8_t* vb = blk + 8 * D;
      const int g = sub % 4 * 2, hw = (sub >> 2 & 1) * 2;
      *reinterpret_cast<uint16_t*>(vb + kv4::v_word_byte<D>(g, r, sub / 8) + hw) = (uint16_t)word;
      *reinterpret_cast<uint16_t*>(vb + kv4::v_word_byte<D>(g + 1, r, sub / 8) + hw) = (uint16_t)(word >> 16);
    }
    if (sub % gl == 0)
      *reinterpret_cast<__half2*>(blk + 16 * D + ((is_k ? 0 : ng * 16) + sub / gl * 16 + r) * 4) =
          __halves2half2(scale, offset);
  }
}

template <int D, bool F32>
__global__ void kv4_read_kernel(const Kv4Cache c, const int64_t* slots, void* k_out, void* v_out, uint32_t* status) {
  pdl_wait();
  constexpr int kLanes = D / 8;
  const int t = blockIdx.x;
  const int sub = threadIdx.x % kLanes;
  const int64_t slot = slots[t];
  const int64_t capacity = (int64_t)c.num_pages * c.page_size;
  if (threadIdx.x == 0 && blockIdx.y == 0 && slot >= capacity) report_status(status, kStatusBadIndex);
  const bool ok = slot >= 0 && slot < capacity;
  const int per = blockDim.x / kLanes, ng = c.ng(), gl = c.group / 8;
  for (int h = blockIdx.y * per + threadIdx.x / kLanes; h < 2 * c.kv_heads; h += gridDim.y * per) {
    const bool is_k = h < c.kv_heads;
    const int kvh = is_k ? h : h - c.kv_heads;
    V8 y = {};
    if (ok) {
      const int64_t page = slot / c.page_size;
      const int in_page = (int)(slot - page * c.page_size), r = in_page % 16;
      const uint8_t* blk = c.pages + ((page * c.kv_heads + kvh) * (c.page_size / 16) + in_page / 16) * c.block_bytes();
      uint32_t word;
      if (is_k) {
        word = *reinterpret_cast<const uint32_t*>(blk + kv4::k_word_byte<D>(r, sub % 4, sub / 4));
      } else {
        const uint8_t* vb = blk + 8 * D;
        const int g = sub % 4 * 2, hw = (sub >> 2 & 1) * 2;
        word = *reinterpret_cast<const uint16_t*>(vb + kv4::v_word_byte<D>(g, r, sub / 8) + hw) |
               (uint32_t)*reinterpret_cast<const uint16_t*>(vb + kv4::v_word_byte<D>(g + 1, r, sub / 8) + hw) << 16;
      }
      const float2 p = __half22float2(
          *reinterpret_cast<const __half2*>(blk + 16 * D + ((is_k ? 0 : ng * 16) + sub / gl * 16 + r) * 4));
#pragma unroll
      for (int i = 0; i < 8; ++i) y.x[i] = fmaf((float)(word >> (4 * i) & 15u), p.x, p.y);
    }
    store8<F32>(is_k ? k_out : v_out, ((int64_t)t * c.kv_heads + kvh) * D + sub * 8, y);
  }
}

// One block per token, up to 1024 threads over its heads; few tokens are spread over the second
// grid dimension so that a decode step's heads run on several SMs.
dim3 token_grid(int T, int units, int lanes, int threads) {
  const int per = threads / lanes;
  const int turns = (units + per - 1) / per;
  return dim3(T, T < 64 ? turns : 1);
}

}  // namespace

cudaError_t launch_kv4_append(LaunchCtx& ctx, const Kv4Cache& c, const Kv4Append& a) {
  ctx.variant = "kv4_append";
  const int heads = a.q_heads + 2 * c.kv_heads, threads = 256;
  const dim3 grid = token_grid(a.T, heads, c.head_dim / 8, threads);
  auto go = [&](auto kern) { return launch_kernel(ctx, kern, grid, dim3(threads), 0, c, a, ctx.status); };
  if (c.head_dim == 64) return a.f32 ? go(kv4_append_kernel<64, true>) : go(kv4_append_kernel<64, false>);
  if (c.head_dim == 128) return a.f32 ? go(kv4_append_kernel<128, true>) : go(kv4_append_kernel<128, false>);
  return a.f32 ? go(kv4_append_kernel<256, true>) : go(kv4_append_kernel<256, false>);
}

cudaError_t launch_kv4_read(LaunchCtx& ctx, const Kv4Cache& c, const int64_t* slots, int T, int f32, void* k_out,
                            void* v_out) {
  ctx.variant = "kv4_read";
  const int threads = 256;
  const dim3 grid = token_grid(T, 2 * c.kv_heads, c.head_dim / 8, threads);
  auto go = [&](auto kern) {
    return launch_kernel(ctx, kern, grid, dim3(threads), 0, c, slots, k_out, v_out, ctx.status);
  };
  if (c.head_dim == 64) return f32 ? go(kv4_read_kernel<64, true>) : go(kv4_read_kernel<64, false>);
  if (c.head_dim == 128) return f32 ? go(kv4_read_kernel<128, true>) : go(kv4_read_kernel<128, false>);
  return f32 ? go(kv4_read_kernel<256, true>) : go(kv4_read_kernel<256, false>);
}

}  // namespace mnb
