// Low-rank adapters of many requests beside a shared product:
//   out[m] = base[m] + scale[a] * up[a] (down[a] x[m]),  a = adapter[m].
//
// A cluster of CTAs takes the rows of one adapter among a tile of consecutive rows, in one launch for both products:
//   1. s = down x: the CTAs split K, the warps of a CTA split it further; partial sums meet in shared memory, then over
//      the cluster;
//   2. up s: the CTAs split N, each with all of s.
// Rows are the M side of the warp's matrix instructions and ranks (then output columns) the N side; a lane loads 8 consecutive
// elements of K (or of the rank), and both operands number the products' inner index alike, so neither passes
// through shared memory.
// fp16 activations: s is rounded to fp16 after its row was scaled by a power of two to [2^13, 2^14), as the result is
// rounded. fp32: x and s are split into two tf32 parts (2^-23 together), the weights are exact in tf32.
#include "cluster.cuh"
#include "mma_sync.cuh"
#include "mnb_device.cuh"
#include "mnb_internal.h"

namespace mnb {
namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 half2_floats(uint32_t u) {
  return __half22float2(*reinterpret_cast<const __half2*>(&u));
}
__device__ __forceinline__ uint32_t tf32(float x) {
  uint32_t r;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
  return r;
}
// c += A . B, m16n8k8: lane 4g + t holds A rows g, g + 8 and B column g at k = t, t + 4
__device__ __forceinline__ void mma1688(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// E halves from p, zeros from element `have` on.
template <int E>
__device__ __forceinline__ void load_weights(uint32_t (&w)[E / 2], const __half* p, int have) {
#pragma unroll
  for (int i = 0; i < E / 2; ++i) w[i] = 0;
  if (have > 0) {
    if constexpr (E == 8) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (E == 4) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
      w[0] = v.x, w[1] = v.y;
    } else {
      w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
    }
    if (have < E) {
#pragma unroll
      for (int i = 0; i < E / 2; ++i) w[i] &= have >= 2 * i + 2 ? 0xffffffffu : have == 2 * i + 1 ? 0xffffu : 0u;
    }
  }
}

// One tile's products with 4 inner elements a lane for each row (fp32 activations): a[part][row][element].
struct Split {
  uint32_t hi, lo;
};
__device__ __forceinline__ Split split(float x) {
  const uint32_t h = tf32(x);
  return {h, tf32(x - __uint_as_float(h))};
}

template <int RB, int MT, bool F32>
struct LoraSmem {
  static constexpr int RP = RB * 8;                              // ranks, padded
  static constexpr int kPart = kWarps * 16 * RP * 4;             // partial sums of s
  static constexpr int kS = F32 ? 16 * MT * (RP + 4) * 4 : 16 * MT * (RP + 8) * 2;  // s, rows apart by an odd number of 16 bytes
  static constexpr int kBytes = kPart + kS;
};

template <int RB, int MT, bool F32>
__global__ void __launch_bounds__(kThreads) lora_kernel(const Lora a, int tiles, int subs, int cluster, uint32_t* status) {
  using T = std::conditional_t<F32, float, __half>;
  using L = LoraSmem<RB, MT, F32>;
  constexpr int RP = L::RP, TM = 16 * MT;
  constexpr int E = RB >= 4 ? 8 : RB == 2 ? 4 : 2;  // elements of the rank that a lane has of a chunk
  constexpr int KC = RP / (4 * E);                  // chunks of the rank
  constexpr int kSRow = F32 ? RP + 4 : RP + 8;      // elements between the rows of s
  extern __shared__ __align__(128) uint8_t smem[];
  float* part = reinterpret_cast<float*>(smem);
  T* s_mem = reinterpret_cast<T*>(smem + L::kPart);
  __shared__ int index[TM], rows[TM];
  __shared__ float factors[TM];
  __shared__ uint32_t firsts[2];
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, g = lane / 4, t = lane % 4;
  const int rank_of_cta = cluster_ctarank(), id = blockIdx.x / cluster;
  const int tile = id % tiles, sub = id / tiles;
  const int m0 = tile * TM;
  pdl_launch_dependents();
  pdl_wait();

  // ---- the tile's distinct adapters ----
  if (tid < TM) {
    int v = -2;  // no row
    if (m0 + tid < a.M) {
      v = a.adapter[m0 + tid];
      if (v >= a.count) {
        if (rank_of_cta == 0 && sub == 0) report_status(status, kStatusBadIndex);
        v = -1;
      }
      v = max(v, -1);
    }
    index[tid] = v;
  }
  if (tid < 2) firsts[tid] = 0;
  __syncthreads();
  if (tid < TM) {
    const int v = index[tid];
    bool first = v != -2;
    for (int j = 0; j < tid; ++j) first = first && index[j] != v;
    if (first) atomicOr(&firsts[tid / 32], 1u << (tid % 32));
  }
  __syncthreads();
  uint64_t left = (uint64_t)firsts[1] << 32 | firsts[0];
  for (int i = 0; i < sub && left; ++i) left &= left - 1;

  while (left) {
    const int value = index[__ffsll(left) - 1];
    for (int i = 0; i < subs && left; ++i) left &= left - 1;
    // ---- this adapter's rows ----
    uint64_t mine = 0;
#pragma unroll
    for (int h = 0; h < (TM + 31) / 32; ++h) {
      const int i = 32 * h + lane;
      mine |= (uint64_t)__ballot_sync(kFull, i < TM && index[i < TM ? i : 0] == value) << (32 * h);
    }
    const int n_rows = __popcll(mine);
    if (tid < TM && (mine >> tid & 1)) rows[__popcll(mine & ((1ull << tid) - 1))] = m0 + tid;
    __syncthreads();
    const int rank = value < 0 ? 0 : a.ranks ? min(max(a.ranks[value], 0), a.max_rank) : a.max_rank;
    if (rank == 0 && a.base == a.out && a.base_stride == a.out_stride) {
      __syncthreads();
      continue;
    }
    const int mt_all = (n_rows + 15) / 16;
    if (rank > 0) {
      // ---- s = down x over this CTA's part of K ----
      const int groups = mt_all > 2 ? 4 : mt_all;      // warps side by side over the rows,
      const int splits = kWarps / groups;              // and over K
      const int mg = warp % groups, kg = warp / groups;
      const int granules = (a.K + 31) / 32;
      const int g0 = (int)((int64_t)granules * rank_of_cta / cluster), g1 = (int)((int64_t)granules * (rank_of_cta + 1) / cluster);
      float acc[RB][4];
#pragma unroll
      for (int j = 0; j < RB; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][i] = 0.0f;
      const T* xr[2];
      bool live[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = mg * 16 + g + 8 * h;
        live[h] = r < n_rows;
        xr[h] = static_cast<const T*>(a.x) + (int64_t)rows[live[h] ? r : 0] * a.x_stride;
      }
      const __half* down = static_cast<const __half*>(a.down) + ((int64_t)value * a.max_rank + g) * a.K;
      if (mg < mt_all) {
        for (int i = g0 + kg; i < g1; i += splits) {
          const int k = i * 32 + 8 * t;
          const bool in = k < a.K;
          uint4 w[RB];
#pragma unroll
          for (int j = 0; j < RB; ++j) {
            w[j] = make_uint4(0, 0, 0, 0);
            if (in && j * 8 + g < rank) w[j] = __ldg(reinterpret_cast<const uint4*>(down + (int64_t)j * 8 * a.K + k));
          }
          if constexpr (F32) {
            float x[2][8];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                float4 v = make_float4(0, 0, 0, 0);
                if (in && live[h]) v = *reinterpret_cast<const float4*>(xr[h] + k + 4 * q);
                x[h][4 * q] = v.x, x[h][4 * q + 1] = v.y, x[h][4 * q + 2] = v.z, x[h][4 * q + 3] = v.w;
              }
#pragma unroll
            for (int s = 0; s < 4; ++s) {
              const Split x0 = split(x[0][2 * s]), x1 = split(x[1][2 * s]), x2 = split(x[0][2 * s + 1]), x3 = split(x[1][2 * s + 1]);
              const uint32_t hi[4] = {x0.hi, x1.hi, x2.hi, x3.hi}, lo[4] = {x0.lo, x1.lo, x2.lo, x3.lo};
#pragma unroll
              for (int j = 0; j < RB; ++j) {
                if (j * 8 < rank) {
                  const uint32_t u[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
                  const float2 b = half2_floats(u[s]);
                  mma1688(acc[j], lo, __float_as_uint(b.x), __float_as_uint(b.y));
                  mma1688(acc[j], hi, __float_as_uint(b.x), __float_as_uint(b.y));
                }
              }
            }
          } else {
            uint4 x[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              x[h] = make_uint4(0, 0, 0, 0);
              if (in && live[h]) x[h] = *reinterpret_cast<const uint4*>(xr[h] + k);
            }
#pragma unroll
            for (int j = 0; j < RB; ++j) {
              if (j * 8 < rank) {
                mma16816(acc[j], x[0].x, x[1].x, x[0].y, x[1].y, w[j].x, w[j].y);
                mma16816(acc[j], x[0].z, x[1].z, x[0].w, x[1].w, w[j].z, w[j].w);
              }
            }
          }
        }
#pragma unroll
        for (int j = 0; j < RB; ++j) {
          float* p = part + ((kg * groups + mg) * 16 + g) * RP + j * 8 + 2 * t;
          *reinterpret_cast<float2*>(p) = make_float2(acc[j][0], acc[j][1]);
          *reinterpret_cast<float2*>(p + 8 * RP) = make_float2(acc[j][2], acc[j][3]);
        }
      }
      __syncthreads();
      // ---- over the warps, then over the cluster; every CTA gets all of s ----
      for (int e = tid * 4; e < mt_all * 16 * RP; e += kThreads * 4) {
        float4 v = *reinterpret_cast<float4*>(part + e);
        for (int i = 1; i < splits; ++i) {
          const float4 o = *reinterpret_cast<float4*>(part + i * groups * 16 * RP + e);
          v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
        }
        *reinterpret_cast<float4*>(part + e) = v;
      }
      cluster_arrive();
      cluster_wait();
      const float scale = a.scales ? a.scales[value] : 1.0f;
      for (int e = tid * 4; e < mt_all * 16 * RP; e += kThreads * 4) {  // RP / 4 neighbouring lanes have a row
        float4 v = make_float4(0, 0, 0, 0);
        for (int c = 0; c < cluster; ++c) {
          const float4 o = cluster_ld_f4(cluster_map(smem_u32(part + e), c));
          v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
        }
        const int r = e / RP, col = e % RP;
        if constexpr (F32) {
          *reinterpret_cast<float4*>(s_mem + r * kSRow + col) = v;
          if (col == 0) factors[r] = scale;
        } else {
          float top = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
#pragma unroll
          for (int o = 1; o < RP / 4; o <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
          const int ex = (int)(__float_as_uint(top) >> 23) - 127;
          const int p = top < INFINITY && top > 0.0f ? max(ex, -110) - 13 : 0;
          const float f = __uint_as_float((uint32_t)(127 - p) << 23);
          *reinterpret_cast<uint2*>(s_mem + r * kSRow + col) = make_uint2(half2_bits(v.x * f, v.y * f), half2_bits(v.z * f, v.w * f));
          if (col == 0) factors[r] = scalbnf(scale, p);
        }
      }
      __syncthreads();
      cluster_arrive();  // no more reads of the others' sums
    }

    // ---- out = base + up s over this CTA's part of N, 32 columns at a time ----
    // Column c of the product's 8-column tile j is output column 8 (c / 2) + 2 j + c % 2 of the 32: a lane then has
    // 8 consecutive ones, of four tiles.
    const int blocks = (a.N + 31) / 32;
    const int n0 = (int)((int64_t)blocks * rank_of_cta / cluster), n1 = (int)((int64_t)blocks * (rank_of_cta + 1) / cluster);
    constexpr int kVec = 16 / sizeof(T);
    const bool base_vec = a.base_stride % kVec == 0, out_vec = a.out_stride % kVec == 0;
    for (int nb = n0 + warp; nb < n1; nb += kWarps) {
      uint32_t w[4][KC][E / 2];
      if (rank > 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int n = nb * 32 + 8 * (g / 2) + 2 * j + g % 2;
          const __half* up = static_cast<const __half*>(a.up) + ((int64_t)value * a.N + n) * a.max_rank + E * t;
#pragma unroll
          for (int c = 0; c < KC; ++c) load_weights<E>(w[j][c], up + 4 * E * c, n < a.N ? rank - 4 * E * c - E * t : 0);
        }
      }
      const int n = nb * 32 + 8 * t, width = min(8, a.N - n);
      for (int mt = 0; mt < mt_all; ++mt) {
        float acc[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[j][i] = 0.0f;
        float b[2][8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = mt * 16 + g + 8 * h;
#pragma unroll
          for (int i = 0; i < 8; ++i) b[h][i] = 0.0f;
          if (a.base && r < n_rows && width > 0) {
            const T* p = static_cast<const T*>(a.base) + (int64_t)rows[r] * a.base_stride + n;
            if (base_vec && width == 8) {
              if constexpr (F32) {
                const float4 v0 = *reinterpret_cast<const float4*>(p), v1 = *reinterpret_cast<const float4*>(p + 4);
                b[h][0] = v0.x, b[h][1] = v0.y, b[h][2] = v0.z, b[h][3] = v0.w;
                b[h][4] = v1.x, b[h][5] = v1.y, b[h][6] = v1.z, b[h][7] = v1.w;
              } else {
                const uint4 v = *reinterpret_cast<const uint4*>(p);
                const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const float2 f = half2_floats(u[i]);
                  b[h][2 * i] = f.x, b[h][2 * i + 1] = f.y;
                }
              }
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (i < width) b[h][i] = (float)p[i];
            }
          }
        }
        if (rank > 0) {
#pragma unroll
          for (int c = 0; c < KC; ++c) {
            if (4 * E * c < rank) {
              const T* sr = s_mem + (mt * 16 + g) * kSRow + 4 * E * c + E * t;
              if constexpr (F32) {
#pragma unroll
                for (int s = 0; s < E / 2; ++s) {
                  const float2 v0 = *reinterpret_cast<const float2*>(sr + 2 * s);
                  const float2 v1 = *reinterpret_cast<const float2*>(sr + 8 * kSRow + 2 * s);
                  const Split x0 = split(v0.x), x1 = split(v1.x), x2 = split(v0.y), x3 = split(v1.y);
                  const uint32_t hi[4] = {x0.hi, x1.hi, x2.hi, x3.hi}, lo[4] = {x0.lo, x1.lo, x2.lo, x3.lo};
#pragma unroll
                  for (int j = 0; j < 4; ++j) {
                    const float2 f = half2_floats(w[j][c][s]);
                    mma1688(acc[j], lo, __float_as_uint(f.x), __float_as_uint(f.y));
                    mma1688(acc[j], hi, __float_as_uint(f.x), __float_as_uint(f.y));
                  }
                }
              } else {
                uint32_t x[2][E / 2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const T* p = sr + 8 * h * kSRow;
                  if constexpr (E == 8) {
                    const uint4 v = *reinterpret_cast<const uint4*>(p);
                    x[h][0] = v.x, x[h][1] = v.y, x[h][2] = v.z, x[h][3] = v.w;
                  } else if constexpr (E == 4) {
                    const uint2 v = *reinterpret_cast<const uint2*>(p);
                    x[h][0] = v.x, x[h][1] = v.y;
                  } else {
                    x[h][0] = *reinterpret_cast<const uint32_t*>(p);
                  }
                }
#pragma unroll
                for (int s = 0; s < (E + 3) / 4; ++s)
#pragma unroll
                  for (int j = 0; j < 4; ++j) {
                    if constexpr (E == 2) mma16816(acc[j], x[0][0], x[1][0], 0u, 0u, w[j][c][0], 0u);
                    else mma16816(acc[j], x[0][2 * s], x[1][2 * s], x[0][2 * s + 1], x[1][2 * s + 1], w[j][c][2 * s], w[j][c][2 * s + 1]);
                  }
              }
            }
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = mt * 16 + g + 8 * h;
          if (r < n_rows && width > 0) {
            const float f = rank > 0 ? factors[r] : 0.0f;
            T* p = static_cast<T*>(a.out) + (int64_t)rows[r] * a.out_stride + n;
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = rank > 0 ? fmaf(acc[i / 2][2 * h + i % 2], f, b[h][i]) : b[h][i];
            if (out_vec && width == 8) {
              if constexpr (F32) {
                *reinterpret_cast<float4*>(p) = make_float4(y[0], y[1], y[2], y[3]);
                *reinterpret_cast<float4*>(p + 4) = make_float4(y[4], y[5], y[6], y[7]);
              } else {
                *reinterpret_cast<uint4*>(p) = make_uint4(half2_bits(y[0], y[1]), half2_bits(y[2], y[3]), half2_bits(y[4], y[5]),
                                                          half2_bits(y[6], y[7]));
              }
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (i < width) p[i] = (T)y[i];
            }
          }
        }
      }
    }
    if (rank > 0) cluster_wait();
    __syncthreads();
  }
}

template <int RB, int MT, bool F32>
cudaError_t launch_lora_t(LaunchCtx& ctx, const Lora& a, int subs, int cluster) {
  using L = LoraSmem<RB, MT, F32>;
  auto kern = lora_kernel<RB, MT, F32>;
  static std::atomic<uint64_t> sized{0}, wide{0};
  cudaError_t e = allow_smem(kern, L::kBytes, ctx.device, sized);
  if (e == cudaSuccess && cluster > 8) e = allow_wide_clusters(kern, ctx.device, wide);
  if (e != cudaSuccess) return e;
  const int tiles = (a.M + 16 * MT - 1) / (16 * MT);
  return launch_clusters(ctx, kern, cluster, dim3((unsigned)tiles * subs * cluster), dim3(kThreads), L::kBytes, a, tiles, subs, cluster,
                         ctx.status);
}

template <int RB, int MT>
cudaError_t launch_lora_rb(LaunchCtx& ctx, const Lora& a, int subs, int cluster) {
  return a.f32 ? launch_lora_t<RB, MT, true>(ctx, a, subs, cluster) : launch_lora_t<RB, MT, false>(ctx, a, subs, cluster);
}

template <int RB>
cudaError_t launch_lora_mt(LaunchCtx& ctx, const Lora& a) {
  // Few rows: tiles of 16 and a cluster for each adapter that a tile can have; many: tiles of 64, whose adapters four
  // clusters take in turn.
  if (a.M <= 1024) return launch_lora_rb<RB, 1>(ctx, a, a.M < 16 ? a.M : 16, a.M <= 16 ? 16 : 8);
  return launch_lora_rb<RB, 4>(ctx, a, 4, 8);
}

}  // namespace

cudaError_t launch_lora(LaunchCtx& ctx, const Lora& a) {
  ctx.variant = a.f32 ? "lora_f32" : "lora_f16";
  if (a.max_rank <= 8) return launch_lora_mt<1>(ctx, a);
  if (a.max_rank <= 16) return launch_lora_mt<2>(ctx, a);
  if (a.max_rank <= 32) return launch_lora_mt<4>(ctx, a);
  if (a.max_rank <= 64) return launch_lora_mt<8>(ctx, a);
  return launch_lora_mt<16>(ctx, a);
}

}  // namespace mnb
