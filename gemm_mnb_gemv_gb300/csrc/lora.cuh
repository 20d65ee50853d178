// What the adapter kernels share: copies, and the list of a call's items.
#pragma once

#include "mnb_device.cuh"
#include "mnb_internal.h"

namespace mnb {
namespace lora {

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Two fp32 as fp16 pairs: hi + lo is within 2^-22 of them.
struct Split {
  uint32_t hi, lo;
};
__device__ __forceinline__ Split split(float x, float y) {
  const uint32_t h = half2_bits(x, y);
  const float2 f = half2_floats(h);
  return {h, half2_bits(x - f.x, y - f.y)};
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// 16 bytes global -> shared, asynchronously.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void store_zeros(uint32_t dst) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(dst), "r"(0u) : "memory");
}
__device__ __forceinline__ void store16(uint32_t dst, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(dst), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// The first `bytes` (2..14, even) of 16 and zeros, by this thread itself: what the ends of rows and ranks need.
static __device__ __noinline__ void copy_some(uint32_t dst, const void* src, int bytes) {
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (2 * i < bytes) w[i / 2] |= (uint32_t)__ldcg(static_cast<const unsigned short*>(src) + i) << (16 * (i & 1));
  store16(dst, w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Elements at .. at + width - 1 of a base of `end` elements whose rows lie anywhere (at < 0: zeros): their 16-byte chunks, brought into
// place. kWords * 4 bytes are worked on; what lies behind `width` is anything. (Element by element, and stored so too, 900 rows of
// 4095 took 34 us instead of 18; now 16, at a stride of 4096 13.)
template <typename T, int kWords>
__device__ __forceinline__ void loose_row(const T* base, int64_t at, int64_t end, int width, uint32_t (&y)[kWords]) {
  constexpr int kVec = 16 / sizeof(T), kChunks = kWords / 4 + 1;
  uint32_t w[4 * kChunks];
#pragma unroll
  for (int i = 0; i < 4 * kChunks; ++i) w[i] = 0;
  int skew = 0;
  if (at >= 0) {
    skew = (int)(at % kVec);
    const T* p = base + at - skew;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      if (kVec * c < skew + width) {
        if (at - skew + kVec * (c + 1) <= end) {
          const uint4 v = __ldcg(reinterpret_cast<const uint4*>(p) + c);
          w[4 * c] = v.x, w[4 * c + 1] = v.y, w[4 * c + 2] = v.z, w[4 * c + 3] = v.w;
        } else {  // behind the last row there may be nothing
#pragma unroll
          for (int i = 0; i < kVec; ++i)
            if (at - skew + kVec * c + i < end) {
              if constexpr (sizeof(T) == 4) w[4 * c + i] = __ldcg(reinterpret_cast<const uint32_t*>(p) + kVec * c + i);
              else w[4 * c + i / 2] |= (uint32_t)__ldcg(reinterpret_cast<const unsigned short*>(p) + kVec * c + i) << (16 * (i & 1));
            }
        }
      }
    }
  }
  const int words = skew * (int)sizeof(T) / 4;
#pragma unroll
  for (int i = 0; i < kWords + 2; ++i) w[i] = words & 2 ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < kWords + 1; ++i) w[i] = words & 1 ? w[i + 1] : w[i];
#pragma unroll
  for (int i = 0; i < kWords; ++i) y[i] = sizeof(T) == 2 && (skew & 1) ? __byte_perm(w[i], w[i + 1], 0x5432) : w[i];
}

__device__ __forceinline__ int64_t base_end(const Lora& a) { return (int64_t)(a.M - 1) * a.base_stride + a.N; }

// The rows of one adapter (negative: none) in a tile.
struct Item {
  int m0, adapter;
  uint64_t rows[2];  // bit i: row m0 + i
};

// Power of two that brings a row whose largest magnitude is `top` to [2^13, 2^14): the row is held times 2^-power.
__device__ __forceinline__ int row_power(float top) {
  const int ex = (int)(__float_as_uint(top) >> 23) - 127;
  return top < INFINITY && top > 0.0f ? max(ex, -110) - 13 : 0;
}

// A call's items, with `rest` but the first of each tile: those with more than `few` rows from the front of `list`, the others from
// its back. One CTA, a warp a tile: 1 to 3 us, 8 where a tile of 128 rows has 63 adapters. The order within the two parts hangs on the warps' pace, and
// nothing hangs on the order.
template <int TM>
__global__ void __launch_bounds__(1024) list_kernel(const Lora a, int few, int rest, uint32_t* counts, Item* list, int capacity,
                                                    uint32_t* status) {
  constexpr int H = (TM + 31) / 32;
  __shared__ uint32_t count[2];
  pdl_wait();
  pdl_launch_dependents();  // behind the wait: the next launch reads its inputs without one
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x < 2) count[threadIdx.x] = 0;
  __syncthreads();
  auto fetch = [&](int m0, int (&v)[H]) {
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const int i = 32 * h + lane;
      v[h] = -2;  // no row
      if (i < TM && m0 + i < a.M) v[h] = max(a.adapter[m0 + i], -1);
    }
  };
  int next[H];
  fetch(warp * TM, next);
  for (int m0 = warp * TM; m0 < a.M; m0 += 32 * TM) {
    int v[H];
    uint32_t left[H], any = 0;
#pragma unroll
    for (int h = 0; h < H; ++h) {
      v[h] = next[h];
      if (v[h] >= a.count) {
        report_status(status, kStatusBadIndex);
        v[h] = -1;
      }
      left[h] = __ballot_sync(kFull, v[h] != -2);
      any |= left[h];
    }
    fetch(m0 + 32 * TM, next);
    auto put = [&](int value, const uint32_t (&same)[4], int n) {
      const int small = n <= few;
      const int at = (int)atomicAdd(&count[small], 1u);
      list[small ? capacity - 1 - at : at] = {m0, value, {(uint64_t)same[1] << 32 | same[0], (uint64_t)same[3] << 32 | same[2]}};
    };
    if constexpr (H == 1) {  // each adapter's first row, all at once
      const uint32_t same[4] = {__match_any_sync(kFull, v[0]), 0, 0, 0};
      if (v[0] != -2 && __ffs(same[0]) - 1 == lane && (lane > 0 || !rest)) put(v[0], same, __popc(same[0]));
      continue;
    }
    bool skip = rest != 0;
    while (any) {
      int value = -2;
#pragma unroll
      for (int h = H - 1; h >= 0; --h)
        if (left[h]) value = __shfl_sync(kFull, v[h], __ffs(left[h]) - 1);
      uint32_t same[4] = {0, 0, 0, 0};
      int n = 0;
      any = 0;
#pragma unroll
      for (int h = 0; h < H; ++h) {
        same[h] = __ballot_sync(kFull, v[h] == value);
        left[h] &= ~same[h];
        any |= left[h];
        n += __popc(same[h]);
      }
      if (lane == 0 && !skip) put(value, same, n);
      skip = false;
    }
  }
  __syncthreads();
  if (threadIdx.x < 2) counts[threadIdx.x] = count[threadIdx.x];
}

constexpr int kSmallItem = 16;  // rows of the items that the tcgen05 kernel leaves to the other one

// The list's places in a call's workspace.
struct List {
  uint32_t* counts;
  Item* items;
  explicit List(void* workspace) : counts(static_cast<uint32_t*>(workspace)), items(reinterpret_cast<Item*>(counts + 4)) {}
};

}  // namespace lora

// The small items of a list that is there already, beside the kernel before, whose end it waits for at its own.
cudaError_t launch_lora_small(LaunchCtx& ctx, const Lora& a);

}  // namespace mnb
