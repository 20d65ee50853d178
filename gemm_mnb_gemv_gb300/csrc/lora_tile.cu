// Low-rank adapters of many rows (prompts) on the tcgen05 tensor cores, fp16: the products of lora.cu for tiles of 128
// rows.
//
// A cluster of 1 to 8 CTAs (one an SM) takes an item, the rows of one adapter in a tile:
//   1. partial s = down x over the CTA's part of K, 128 a stage (M 128 rows, N the rank), in tensor memory;
//   2. the CTAs exchange: CTA c adds up the rows c 128 / C .. of all partial sums, scales them by the row's power of two
//      and writes them as two fp16 (22 bits) into every CTA's operands s;
//   3. out = base + s up over the CTA's part of N, 128 columns a stage, accumulated in two tensor memory buffers in turn.
// Roles in 512 threads:
//   warps 0-3    producers, into one ring that runs on from product to product and item to item: x and base by tensor copies where
//                the item's rows are neighbours (as a prompt's are), else row by row in 16-byte asynchronous copies; down and up by
//                those (ranks end anywhere; a whole stage takes the four warps 0.75 us, more than its share of the bandwidth);
//   warp 4       MMA issuer (one lane) and tensor memory; warp 5 lets the launch behind start;
//   warps 8-15   exchange and epilogue: a row and 64 columns of a stage a thread, stored as whole sectors.
// Items of up to 16 rows (other requests' single tokens) are left to the kernel of lora.cu, launched behind: it starts on the SMs
// that this one leaves free. (A row alone takes a cluster 15 us here: 1500 rows of a prompt with 63 such rows 88 us.)
// Every wait is bounded: a role whose wait gave up reports it and stops, the others run into their own limits, and the
// rows left get NaN.
// Bound: 8192 rows, K 4096, N 14336, rank 64: 112 us (80 at the copy rate), of which 15 go to the first product, 6 to the exchange and 84
// to the second product at 5.6 TB/s of reads and writes. 2048 rows, K = N = 4096, rank 32: 22.3 us (7.7): one item a cluster, so the chain of
// start, first product, exchange and stages of 1.2 us of epilogue. 16 epilogue warps instead of 8 took 12 us more; waits that sleep changed nothing.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "cluster.cuh"
#include "lora.cuh"
#include "tcgen05.cuh"

namespace mnb {
namespace {

using namespace lora;

constexpr int kRows = 128, kSpan = 128, kEpiWarps = 8, kThreads = 256 + 32 * kEpiWarps, kProducers = 128;
constexpr int kPieces = kEpiWarps / 4, kOwnCols = kSpan / kPieces;  // of an epilogue warp in a stage

template <int RP>
struct TileGeo {
  static constexpr int kAct = kRows * kSpan * 2;                 // x or base: two halves of 64 columns, 128-byte rows
  static constexpr int kWeight = kSpan * 128 * (RP > 64 ? 2 : 1);  // down: two halves of K; up: halves of the rank
  static constexpr int kSlot = kAct + kWeight;
  // s: rows of 128 bytes. Ranks up to 32: the low parts behind the high ones in a row; up to 64: a half of their own; up to 128: two halves of
  // high parts, and the low ones over the partial sums, which take as many bytes as both together.
  static constexpr int kS = kRows * 128 * (RP > 32 ? 2 : 1);
  static constexpr bool kOver = RP > 64;
  static constexpr int kPart = kRows * RP * 4;
  static constexpr int kLowAt = kOver ? kS : RP > 32 ? kRows * 128 : RP * 2;  // from the high parts
  static constexpr int kLowGroup = kOver ? 8 * RP * 4 : 1024;  // of eight rows: where the eight rows of partial sums are, their halves side by side
  static constexpr int kLowHalf = 1024;
  static constexpr int kFit = (227 * 1024 - 2048 - kS - kPart) / kSlot;
  static constexpr int kStages = kFit > 4 ? 4 : kFit;
  static constexpr int kBytes = kStages * kSlot + kS + kPart + 1024;
  static_assert(kStages >= 2, "two stages in flight");
};

// Byte of 16-byte chunk `chunk` of a row of 128 bytes, in the 128-byte swizzle of the tensor cores' operands.
__device__ __forceinline__ uint32_t swizzled(int row, int chunk) { return (uint32_t)(row * 128 + ((chunk ^ row) & 7) * 16); }

// Place of float4 `chunk` of a row of partial sums: eight neighbouring rows' chunks in distinct banks.
template <int RP>
__device__ __forceinline__ uint32_t part_place(int row, int chunk) {
  constexpr int kChunks = RP / 4;
  return (uint32_t)(row * RP * 4 + (chunk ^ (kChunks >= 8 ? row & 7 : row >> 1 & 3)) * 16);
}

__device__ __forceinline__ void sts128(uint32_t addr, float a, float b, float c, float d) {
  asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "f"(a), "f"(b), "f"(c), "f"(d) : "memory");
}
// A warp arrives once at the barrier of each CTA, lane i at CTA i's: one after the other each would wait for the writes before
// it again (0.7 us). What the warp wrote before, and saw, is visible to those that wait there.
__device__ __forceinline__ void cluster_mbar_arrive(uint64_t* bar, int cluster) {
  __syncwarp();
  const int lane = threadIdx.x & 31;
  if (lane < cluster)
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_map(smem_u32(bar), lane)) : "memory");
}
__device__ __forceinline__ bool cluster_mbar_try_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// Waits, for a whole warp; what goes beyond the first try is kept out of line: the roles' code has to stay in the instruction cache together.
__device__ __noinline__ bool wait_more(uint64_t* bar, uint32_t parity) { return __all_sync(kFull, mbar_wait_bounded(bar, parity)); }
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity) {
  return __all_sync(kFull, mbar_try_wait(bar, parity)) || wait_more(bar, parity);
}
__device__ __noinline__ bool cluster_mbar_wait(uint64_t* bar, uint32_t parity) {
  if (cluster_mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t i = 0; i < kSpinLimit; ++i) {
    if (cluster_mbar_try_wait(bar, parity)) return true;
    if ((i & 255u) == 255u && global_timer_ns() - t0 > kWaitLimitNs) return false;
  }
  return false;
}
// The barrier is arrived at once this thread's copies have landed (it counts the threads).
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// Place of the n-th set bit.
__device__ __noinline__ int nth_bit(uint64_t m0, uint64_t m1, int n) {
  int at = 0;
  uint64_t w = m0;
  const int c0 = __popcll(w);
  if (n >= c0) n -= c0, w = m1, at = 64;
#pragma unroll
  for (int s = 32; s; s >>= 1) {
    const int c = __popcll(w & ((1ull << s) - 1));
    if (n >= c) n -= c, w >>= s, at += s;
  }
  return at;
}

// 64 columns of a warp's 32 rows of a base whose rows lie anywhere (zeros without one): 16-byte chunks, 4 rows and 8 chunks of each at a
// time, go as they are to the rows' places in shared memory; a row's ninth stays with its lane, which brings them into place. (Each lane its own
// row, 5 chunks for 32 columns: 4096 x 4095 of rank 16 78 us.)
__device__ __noinline__ uint4 last_chunk(const unsigned short* p, int n) {  // behind the last row there may be nothing
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) w[i / 2] |= (uint32_t)__ldcg(p + i) << (16 * (i & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
struct LooseBase {
  uint4 ninth;
  int skew;
  __device__ __forceinline__ static uint4 chunk(const unsigned short* base, int64_t at, int64_t end, bool live) {
    if (!live || at >= end) return make_uint4(0, 0, 0, 0);
    return at + 8 <= end ? __ldcg(reinterpret_cast<const uint4*>(base + at)) : last_chunk(base + at, (int)(end - at));
  }
  // The warp's rows are `first` .. of the tile at `tile`, `row` this lane's; columns n .. (below n1).
  __device__ __forceinline__ void fetch(const Lora& a, uint32_t tile, int first, int row, int n, int n1) {
    const int lane = threadIdx.x & 31, c = lane % 8;
    const unsigned short* base = static_cast<const unsigned short*>(a.base);
    const int64_t end = base_end(a);
    uint4 v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int from = __shfl_sync(kFull, row, 4 * k + lane / 8);
      const int64_t at = from * a.base_stride + n;
      const int off = (int)(at & 7);
      v[k] = chunk(base, at - off + 8 * c, end, base && from >= 0 && 8 * c < off + n1 - n);
    }
    const int64_t at = row * a.base_stride + n;
    skew = base && row >= 0 ? (int)(at & 7) : 0;
    ninth = chunk(base, at - skew + 64, end, base && row >= 0 && 64 < skew + n1 - n);
#pragma unroll
    for (int k = 0; k < 8; ++k) store16(tile + swizzled(first + 4 * k + lane / 8, c), v[k].x, v[k].y, v[k].z, v[k].w);
    __syncwarp();
  }
  // 32 columns from chunk c0 (0 or 4) on of row r.
  __device__ __forceinline__ void take(uint32_t tile, int r, int c0, uint32_t (&y)[16]) const {
    uint32_t w[20];
#pragma unroll
    for (int c = 0; c < 5; ++c) {
      uint4 v = ninth;
      if (c < 4 || c0 == 0) v = lds128_a(tile + swizzled(r, c0 + c));
      w[4 * c] = v.x, w[4 * c + 1] = v.y, w[4 * c + 2] = v.z, w[4 * c + 3] = v.w;
    }
#pragma unroll
    for (int i = 0; i < 18; ++i) w[i] = skew & 4 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 17; ++i) w[i] = skew & 2 ? w[i + 1] : w[i];
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = skew & 1 ? __byte_perm(w[i], w[i + 1], 0x5432) : w[i];
  }
};

// A warp's 32 rows of up to 64 results, from their places in shared memory to where they lie: a row's whole 16-byte chunks, 8 of 4 rows at a
// time, then its ends by elements. (A row after the other, 32 lanes of 2 bytes: 4096 x 4095 67 us, 54 so; rows at 32 bytes 29.)
__device__ __noinline__ void store_loose(unsigned short* out, int64_t stride, uint32_t tile, int first, int row, int width) {
  __syncwarp();
  const int lane = threadIdx.x & 31, c = lane % 8;
  const int skew_of = (int)(reinterpret_cast<uintptr_t>(out) / 2 % 8);
#pragma unroll 2
  for (int k = 0; k < 8; ++k) {
    const int r = first + 4 * k + lane / 8, to = __shfl_sync(kFull, row, 4 * k + lane / 8);
    const int off = (int)((skew_of + to * stride) & 7), s = 8 * c - off;  // the row begins `off` elements behind a chunk's start; this chunk at s
    unsigned short* p = out + to * stride;
    if (to >= 0) {
      if (s >= 0 && s + 8 <= width) {
        uint32_t w[8];
        const uint4 u = lds128_a(tile + swizzled(r, off ? c - 1 : c)), v = lds128_a(tile + swizzled(r, c));
        w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w, w[4] = v.x, w[5] = v.y, w[6] = v.z, w[7] = v.w;
        const int shift = (8 - off) & 7;
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = shift & 4 ? w[i + 2] : w[i];
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = shift & 2 ? w[i + 1] : w[i];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = shift & 1 ? __byte_perm(w[i], w[i + 1], 0x5432) : w[i];
        *reinterpret_cast<uint4*>(p + s) = make_uint4(w[0], w[1], w[2], w[3]);
      }
      const int head = min((8 - off) & 7, width), tail = (width - head) & 7;  // elements before and behind the whole chunks
      for (int j = c; j < head + tail; j += 8) {
        const int e = j < head ? j : width - tail + (j - head);
        p[e] = (unsigned short)lds_u16_a(tile + swizzled(r, e / 8) + (e & 7) * 2);
      }
    }
  }
  __syncwarp();
}

// An item as every role sees it.
struct Work {
  Item item;
  int n_rows, rank, cols;          // cols: the rank, in whole steps of 16
  int down_stages, stages;
};

template <int RP>
__global__ void __launch_bounds__(kThreads, 1)
    lora_tile_kernel(const Lora a, const __grid_constant__ CUtensorMap x_map, const __grid_constant__ CUtensorMap base_map, int maps,
                     int cluster, const uint32_t* counts, const Item* list, uint32_t* status) {
  using L = TileGeo<RP>;
  constexpr int S = L::kStages;
  constexpr uint32_t kColD1 = 0, kColD2 = 128;  // tensor memory columns: partial s, two buffers of results
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[4], empty_mma[4], empty_epi[4], d1_full, d2_full[2], d2_empty[2], part_ready, s_ready, drained;
  __shared__ float factors[kRows];
  __shared__ uint32_t tmem_base;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t cta = cluster_ctarank();
  const int id = blockIdx.x / cluster;
  const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u, s_at = ring + S * L::kSlot, part_at = s_at + L::kS;

  if (tid == 0) {
    for (int i = 0; i < 4; ++i) mbar_init(&full[i], kProducers + 1), mbar_init(&empty_mma[i], 1), mbar_init(&empty_epi[i], kEpiWarps + 1);
    for (int i = 0; i < 2; ++i) mbar_init(&d2_full[i], 1), mbar_init(&d2_empty[i], kEpiWarps);
    mbar_init(&d1_full, 1);
    mbar_init(&drained, 1);
    mbar_init(&part_ready, kEpiWarps * cluster);
    mbar_init(&s_ready, kEpiWarps * cluster);
    fence_mbar_init();
  }
  if (warp == 4) {
    tc::tmem_alloc(&tmem_base, 512);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  cluster_arrive();  // the others' barriers are there before anything arrives at them
  cluster_wait();
  const uint32_t tmem = tmem_base;

  const int units = (a.K + 63) / 64, blocks = (a.N + 31) / 32;
  const int k0 = 64 * (int)((int64_t)units * cta / cluster), k1 = min(a.K, 64 * (int)((int64_t)units * (cta + 1) / cluster));
  const int n0 = 32 * (int)((int64_t)blocks * cta / cluster), n1 = min(a.N, 32 * (int)((int64_t)blocks * (cta + 1) / cluster));
  const bool base_vec = a.base && a.base_stride % 8 == 0, out_vec = a.out_stride % 16 == 0 && (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
  const bool in_place = a.base == a.out;
  // Items come in turn: the first of each tile (the rows of its first row's adapter), which a warp finds itself while the list is being
  // made, then the list's, on from the cluster where those end. The list's launch lets this one start when its own inputs are there.
  const int tiles = (a.M + kRows - 1) / kRows, clusters = gridDim.x / cluster;
  int items = 0x7fffffff;
  auto more = [&](int it) {  // whether there is item `it`
    if (it >= tiles && items == 0x7fffffff) {
      pdl_wait();
      items = tiles + (int)__ldcg(counts);
    }
    return it < items;
  };
  auto work_of = [&](int it) {
    Work w;
    if (it < tiles) {
      const int m0 = it * kRows;
      int v[4];
#pragma unroll
      for (int h = 0; h < 4; ++h) v[h] = m0 + 32 * h + lane < a.M ? __ldcg(a.adapter + m0 + 32 * h + lane) : -1;
#pragma unroll
      for (int h = 0; h < 4; ++h) v[h] = v[h] < 0 || v[h] >= a.count ? -1 : v[h];
      w.item = {m0, __shfl_sync(kFull, v[0], 0), {0, 0}};
#pragma unroll
      for (int h = 0; h < 4; ++h)
        w.item.rows[h / 2] |= (uint64_t)__ballot_sync(kFull, v[h] == w.item.adapter && m0 + 32 * h + lane < a.M) << (h % 2 * 32);
    } else {
      const uint64_t* p = reinterpret_cast<const uint64_t*>(list + (it - tiles));
      const uint64_t head = __ldcg(p);
      w.item = {(int)(uint32_t)head, (int)(head >> 32), {__ldcg(p + 1), __ldcg(p + 2)}};
    }
    w.n_rows = __popcll(w.item.rows[0]) + __popcll(w.item.rows[1]);
    const int v = w.item.adapter;
    w.rank = v < 0 ? 0 : a.ranks ? min(max(__ldcg(a.ranks + v), 0), a.max_rank) : a.max_rank;
    w.cols = (w.rank + 15) / 16 * 16;
    w.down_stages = w.rank > 0 ? (max(k1 - k0, 0) + kSpan - 1) / kSpan : 0;
    w.stages = w.rank == 0 && in_place ? 0 : w.down_stages + (max(n1 - n0, 0) + kSpan - 1) / kSpan;
    return w;
  };
  bool ok = true;
  auto give_up = [&](uint32_t what) {
    if (lane == 0) report_status(status, what);
    ok = false;
  };

  if (warp < 4) {
    // ------------------------------ producers ------------------------------------
    int slot = 0, used = 0;
    uint32_t by_epi = 0, mma_phase = 0, epi_phase = 0;  // a bit for each slot: who frees it, and the phases of both
    const int c8 = tid & 7, r8 = tid >> 3;               // chunk of 8, first row of this thread's (16 apart)
    for (int it = id; ok && more(it); it += clusters) {
      const Work w = work_of(it);
      // Neighbouring rows, and enough of them that a whole box is no waste.
      const uint64_t *m = w.item.rows;
      const int first = m[0] ? __ffsll(m[0]) - 1 : 63 + __ffsll(m[1]), last = m[1] ? 127 - __clzll(m[1]) : 63 - __clzll(m[0]);
      const bool run = last - first + 1 == w.n_rows && w.n_rows > 32;
      const bool x_box = run && (maps & 1), base_box = run && (maps & 2);
      // What a copy needs is worked out ahead: four warps issue all of them, and every operation is on their way. This thread has chunk
      // c8 of rows r8 + 16 i, which lie 2 KB apart in shared memory.
      const int mine = w.n_rows > r8 ? (w.n_rows - r8 + 15) / 16 : 0;
      const __half* at[8];  // this thread's rows of x, then of base
      auto find_rows = [&](const void* p, int64_t stride) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          at[i] = static_cast<const __half*>(p) + (i < mine ? w.item.m0 + nth_bit(w.item.rows[0], w.item.rows[1], r8 + 16 * i) : 0) * stride + 8 * c8;
      };
      if (!x_box && w.down_stages > 0) find_rows(a.x, a.x_stride);
      const uint32_t to = swizzled(r8, c8);
      const __half* down = static_cast<const __half*>(a.down) + ((int64_t)w.item.adapter * a.max_rank + r8) * a.K + 8 * c8;
      const __half* up = static_cast<const __half*>(a.up) + ((int64_t)w.item.adapter * a.N + r8) * a.max_rank + 8 * c8;
      const int64_t down_step = 16 * (int64_t)a.K;
      const int up_step = 16 * a.max_rank;
      for (int q = 0; q < w.stages; ++q) {
        if (used >= S) {
          const bool epi = by_epi >> slot & 1;
          uint64_t* bar = epi ? &empty_epi[slot] : &empty_mma[slot];
          uint32_t& phase = epi ? epi_phase : mma_phase;
          if (!wait_warp(bar, phase >> slot & 1)) {
            give_up(kStatusEmptyWait);
            break;
          }
          phase ^= 1u << slot;
        }
        const uint32_t act = ring + slot * L::kSlot, weight = act + L::kAct;
        bool stored = false;  // by this thread itself, not by an asynchronous copy
        if (tid == 0) {
          const bool down_q = q < w.down_stages;
          if (down_q ? x_box : base_box) {
            const int at = down_q ? k0 + q * kSpan : n0 + (q - w.down_stages) * kSpan, end = down_q ? k1 : n1;
            const int boxes = at + 64 < end ? 2 : 1;
            mbar_arrive_expect_tx(&full[slot], boxes * kRows * 128);
            for (int h = 0; h < boxes; ++h)
              tc::tma_load_2d(smem_raw + (act + h * (kRows * 128) - smem_u32(smem_raw)), down_q ? &x_map : &base_map, at + 64 * h,
                              w.item.m0 + first, &full[slot]);
          } else {
            mbar_arrive(&full[slot]);
          }
        }
        if (q < w.down_stages) {
          const int k = k0 + q * kSpan;
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            const int kk = k + 64 * h;
            if (kk + 8 * c8 < k1) {  // steps beyond k1 are not made, nor are columns of s beyond the rank used
              if (!x_box) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  if (i < mine) copy16(act + h * (kRows * 128) + to + i * 2048, at[i] + kk);
              }
#pragma unroll
              for (int i = 0; i < RP / 16; ++i)
                if (r8 + 16 * i < w.rank) copy16(weight + h * (RP * 128) + to + i * 2048, down + i * down_step + kk);
            }
          }
          by_epi &= ~(1u << slot);
        } else {
          const int n = n0 + (q - w.down_stages) * kSpan;
          if (base_vec && !base_box) {
            if (q == w.down_stages) find_rows(a.base, a.base_stride);
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
              const int nn = n + 64 * h + 8 * c8;
              if (nn + 8 <= n1) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  if (i < mine) copy16(act + h * (kRows * 128) + to + i * 2048, at[i] + n + 64 * h);
              } else if (nn < n1) {
                stored = true;
                for (int i = 0; i < mine; ++i) {
                  const int64_t m = w.item.m0 + nth_bit(w.item.rows[0], w.item.rows[1], r8 + 16 * i);
                  const __half* row = static_cast<const __half*>(a.base) + m * a.base_stride;
                  copy_some(act + h * (kRows * 128) + to + i * 2048, row + nn, 2 * (n1 - nn));
                }
              }
            }
          }
#pragma unroll 1
          for (int h = 0; h < (RP > 64 ? 2 : 1); ++h) {
            const int col = 64 * h + 8 * c8, have = w.rank - col;
            const __half* p = up + (int64_t)n * a.max_rank + 64 * h;
            if (have >= 8) {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (n + r8 + 16 * i < n1) copy16(weight + h * (kSpan * 128) + to + i * 2048, p + i * up_step);
            } else if (col < w.cols) {  // zeros behind the rank, up to whole steps
              stored = true;
              if (have <= 0) {
#pragma unroll
                for (int i = 0; i < 8; ++i) store_zeros(weight + h * (kSpan * 128) + to + i * 2048);
              } else {
                for (int i = 0; i < 8; ++i)
                  if (n + r8 + 16 * i < n1) copy_some(weight + h * (kSpan * 128) + to + i * 2048, p + i * up_step, 2 * have);
              }
            }
          }
          by_epi |= 1u << slot;
        }
        if (stored) {
          asm volatile("cp.async.wait_all;" ::: "memory");
          tc::fence_proxy_async_smem();
          mbar_arrive(&full[slot]);
        } else {
          copies_arrive(&full[slot]);
        }
        ++used;
        if (++slot == S) slot = 0;
      }
    }
    copy_commit();
    copy_wait<0>();  // every copy has landed before the CTA can retire
  } else if (warp == 4) {
    // ------------------------------ MMA issuer ----------------------------------
    const bool leader = tc::elect_one();
    int slot = 0, results = 0;
    uint32_t full_phase = 0, d2_phase = 0, s_phase = 0;
    auto wait_full = [&]() {
      if (!wait_warp(&full[slot], full_phase >> slot & 1)) give_up(kStatusMmaWait);
      full_phase ^= 1u << slot;
      tc::fence_proxy_async_smem();  // the copies are generic writes, the products read through the async proxy
      tc::fence_after_sync();
      return ok;
    };
    auto next_slot = [&]() {
      if (++slot == S) slot = 0;
    };
    for (int it = id; ok && more(it); it += clusters) {
      const Work w = work_of(it);
      int q = 0;
      for (; q < w.down_stages && ok; ++q) {
        if (!wait_full()) break;
        const uint32_t act = ring + slot * L::kSlot;
        const uint64_t da = tc::smem_desc_k_sw128(act), db = tc::smem_desc_k_sw128(act + L::kAct);
        const uint32_t idesc = tc::idesc_f16_f32(kRows, w.cols);
        const int steps = (min(kSpan, k1 - k0 - q * kSpan) + 15) / 16;
        if (leader) {
#pragma unroll 1
          for (int kk = 0; kk < steps; ++kk)
            tc::mma_f16(tmem + kColD1, da + (((kk / 4) * (kRows * 128) + (kk % 4) * 32) >> 4),
                        db + (((kk / 4) * (RP * 128) + (kk % 4) * 32) >> 4), idesc, q > 0 || kk > 0);
          tc::mma_commit(&empty_mma[slot]);
          if (q == w.down_stages - 1) tc::mma_commit(&d1_full);
        }
        __syncwarp();
        next_slot();
      }
      // A CTA without any part of K and N has nothing to wait for, and nothing would keep its exchange from going on to the next item before this
      // warp has looked: with a part, the exchange waits for this warp's products.
      if (ok && w.rank > 0 && w.stages > 0) {
        if (!__all_sync(kFull, cluster_mbar_wait(&s_ready, s_phase))) give_up(kStatusMmaWait);
        s_phase ^= 1u;
        asm volatile("fence.proxy.async;" ::: "memory");
        tc::fence_after_sync();
      }
      for (; q < w.stages && ok; ++q) {
        if (!wait_full()) break;
        if (w.rank > 0) {
          const int b = results & 1;
          static_assert(L::kLowAt % 32 == 0 && (!L::kOver || (L::kS % 1024 == 0 && L::kLowGroup == 4 * L::kLowHalf)), "places in the swizzle");
          if (results >= 2) {
            if (!wait_warp(&d2_empty[b], d2_phase >> b & 1)) {
              give_up(kStatusMmaWait);
              break;
            }
            d2_phase ^= 1u << b;
            tc::fence_after_sync();
          }
          const uint64_t db = tc::smem_desc_k_sw128(ring + slot * L::kSlot + L::kAct);
          const uint32_t idesc = tc::idesc_f16_f32(kRows, kSpan);
          if (leader) {
            const uint64_t low = tc::smem_desc_k_sw128(s_at + L::kLowAt, L::kLowGroup), high = tc::smem_desc_k_sw128(s_at);
#pragma unroll 1
            for (int kk = 0; kk < w.cols / 16; ++kk)  // the low parts first
              tc::mma_f16(tmem + kColD2 + 128 * b, low + (((kk / 4) * L::kLowHalf + (kk % 4) * 32) >> 4),
                          db + (((kk / 4) * (kSpan * 128) + (kk % 4) * 32) >> 4), idesc, kk > 0);
#pragma unroll 1
            for (int kk = 0; kk < w.cols / 16; ++kk)
              tc::mma_f16(tmem + kColD2 + 128 * b, high + (((kk / 4) * (kRows * 128) + (kk % 4) * 32) >> 4),
                          db + (((kk / 4) * (kSpan * 128) + (kk % 4) * 32) >> 4), idesc, 1);
            tc::mma_commit(&d2_full[b]);
          }
          ++results;
        }
        // A stage of the second product is also this warp's to free: without products (no adapter) the epilogue doesn't wait for it, and the slot
        // could come round again before it has seen this turn's arrival.
        if (leader) mbar_arrive(&empty_epi[slot]);
        __syncwarp();
        next_slot();
      }
    }
    // the tensor memory is given back only after the products in flight are done
    if (leader) tc::mma_commit(&drained);
    __syncwarp();
    (void)mbar_wait_bounded(&drained, 0);
  } else if (warp == 5) {
    pdl_wait();
    pdl_launch_dependents();  // behind the wait: the launch for the small items reads the list without one
  } else if (warp >= 8) {
    // ------------------------------ exchange and epilogue -------------------------------
    const int e = warp - 8, quarter = warp & 3, piece = e >> 2;  // rows 32 quarter .., columns kOwnCols piece ..
    const int r = quarter * 32 + lane;
    const uint32_t lane_at = tmem + ((uint32_t)(quarter * 32) << 16);
    int slot = 0, results = 0;
    uint32_t full_phase = 0, d1_phase = 0, d2_phase = 0, s_phase = 0;
    for (int it = id; more(it); it += clusters) {
      const Work w = work_of(it);
      const int row = r < w.n_rows ? w.item.m0 + nth_bit(w.item.rows[0], w.item.rows[1], r) : -1;
      if (w.rank > 0) {
        // ---- this CTA's partial sums to shared memory ----
        constexpr int kOwn = RP >= 16 * kPieces ? RP / kPieces : 16;  // columns of a warp; of the smaller ranks some warps have none
        const int col0 = piece * kOwn;
        if (w.down_stages > 0) {
          if (ok && !wait_warp(&d1_full, d1_phase)) give_up(kStatusMmaWait);
          d1_phase ^= 1u;
          tc::fence_after_sync();
          for (int i = 0; i < w.down_stages; ++i) {  // their slots are the MMA issuer's to free
            full_phase ^= 1u << slot;
            if (++slot == S) slot = 0;
          }
        }
        if (ok) {
          if (col0 < RP) {
#pragma unroll 1
            for (int c = 0; c < kOwn; c += 16) {
              float v[16];
              const bool some = w.down_stages > 0 && col0 + c < w.cols;
              if (some) {
                tmem_ld16(lane_at + kColD1 + col0 + c, v);
                tc::tmem_wait_ld();
              }
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (!some || col0 + c + i >= w.rank) v[i] = 0.0f;
#pragma unroll
              for (int i = 0; i < 16; i += 4) sts128(part_at + part_place<RP>(r, (col0 + c + i) / 4), v[i], v[i + 1], v[i + 2], v[i + 3]);
            }
          }
          tc::fence_before_sync();
          cluster_mbar_arrive(&part_ready, cluster);
          if (!__all_sync(kFull, cluster_mbar_wait(&part_ready, s_phase))) give_up(kStatusMmaWait);
        }
        // ---- rows of this CTA's share: over the cluster, to two fp16, into every CTA's operands ----
        // The low parts of eight rows may lie over the sums of the same eight, which only the CTA that has them reads: shares are then whole
        // eights, and its warps meet between reading and writing, whatever became of their waits.
        constexpr int kRowUnit = L::kOver ? 8 : 1, kHeld = L::kOver ? 4 : 1;
        const float scale = a.scales ? __ldcg(a.scales + w.item.adapter) : 1.0f;
        const int sr0 = kRowUnit * (kRows / kRowUnit * (int)cta / cluster), sr1 = kRowUnit * (kRows / kRowUnit * ((int)cta + 1) / cluster);
        const int chunks = (sr1 - sr0) * (RP / 4);
        for (int u0 = e * 32; u0 < chunks; u0 += kHeld * kEpiWarps * 32) {
          uint2 low[kHeld];
          auto place_of = [&](int i, int& sr, int& ch) {  // of this lane's chunk i, and whether there is one
            const int u = u0 + i * (kEpiWarps * 32) + lane;
            sr = sr0 + (u < chunks ? u : 0) / (RP / 4), ch = (u < chunks ? u : 0) % (RP / 4);
            return u < chunks;
          };
          auto put_low = [&](int i) {
            int sr, ch;
            if (!place_of(i, sr, ch)) return;
            const uint32_t to = s_at + L::kLowAt + sr / 8 * L::kLowGroup + (ch / 16) * L::kLowHalf +
                                (RP > 32 ? swizzled(sr % 8, ch / 2 % 8) : swizzled(sr % 8, ch / 2 + RP / 8) - RP * 2) + (ch & 1) * 8;
            for (int c = 0; c < cluster; ++c) cluster_st_u64(cluster_map(to, c), low[i].x, low[i].y);
          };
#pragma unroll
          for (int i = 0; i < kHeld; ++i) {
            if (!ok || u0 + i * (kEpiWarps * 32) >= chunks) continue;
            int sr, ch;
            const bool mine = place_of(i, sr, ch);
            const float4 v = cluster_sum_f4(part_at + part_place<RP>(sr, ch), cluster);
            float top = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
#pragma unroll
            for (int o = 1; o < RP / 4; o <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
            const int p = row_power(top);
            const float f = pow2(-p);
            const Split x = split(v.x * f, v.y * f), y = split(v.z * f, v.w * f);
            low[i] = make_uint2(x.lo, y.lo);
            const uint32_t to = s_at + (ch / 16) * (kRows * 128) + swizzled(sr, ch / 2 % 8) + (ch & 1) * 8;
            for (int c = 0; mine && c < cluster; ++c) {
              cluster_st_u64(cluster_map(to, c), x.hi, y.hi);
              if (ch == 0) cluster_st_f32(cluster_map(smem_u32(&factors[sr]), c), scalbnf(scale, p));
            }
            if (!L::kOver) put_low(i);
          }
          if constexpr (L::kOver) {
            __syncwarp();
            asm volatile("barrier.sync.aligned 1, %0;" ::"n"(kEpiWarps * 32) : "memory");
#pragma unroll
            for (int i = 0; i < kHeld; ++i)
              if (ok && u0 + i * (kEpiWarps * 32) < chunks) put_low(i);
          }
          __syncwarp();
        }
        if (ok) {
          asm volatile("fence.proxy.async;" ::: "memory");  // the products read s through the async proxy
          cluster_mbar_arrive(&s_ready, cluster);
          if (!__all_sync(kFull, cluster_mbar_wait(&s_ready, s_phase))) give_up(kStatusMmaWait);  // for the rows' factors
        }
        s_phase ^= 1u;
      }
      const float factor = ok && w.rank > 0 ? factors[r] : 0.0f;
      // ---- out = base + s up, 128 columns at a time ----
      for (int q = w.down_stages; q < w.stages; ++q) {
        const int b = results & 1;
        if (ok && w.rank > 0) {
          if (!wait_warp(&d2_full[b], d2_phase >> b & 1)) give_up(kStatusMmaWait);
          d2_phase ^= 1u << b;
          tc::fence_after_sync();
        }
        if (ok && !wait_warp(&full[slot], full_phase >> slot & 1)) give_up(kStatusFullWait);
        full_phase ^= 1u << slot;
        if (quarter * 32 < w.n_rows) {
          LooseBase loose;
          const int n_own = n0 + (q - w.down_stages) * kSpan + piece * kOwnCols;  // this warp's 64 columns
          const bool direct = out_vec && min(kOwnCols, n1 - n_own) % 32 == 0;
          const uint32_t tile = ring + slot * L::kSlot + piece * (kRows * 128);
          if (a.base && !base_vec && n_own < n1) loose.fetch(a, tile, quarter * 32, row, n_own, n1);
#pragma unroll 1
          for (int g = 0; g < kOwnCols; g += 32) {
            const int n = n_own + g;
            if (n >= n1) break;
            const int ch0 = g / 8;  // first 16-byte chunk of the 32 columns
            uint32_t y[16];
            if (base_vec) {
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const uint4 v = lds128_a(tile + swizzled(r, ch0 + c));
                y[4 * c] = v.x, y[4 * c + 1] = v.y, y[4 * c + 2] = v.z, y[4 * c + 3] = v.w;
              }
            } else if (a.base) {
              loose.take(tile, r, ch0, y);
            } else {
#pragma unroll
              for (int i = 0; i < 16; ++i) y[i] = 0;
            }
            if (w.rank > 0) {
              float d[32];
              tc::tmem_ld32(lane_at + kColD2 + 128 * b + piece * kOwnCols + g, d);
              tc::tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float2 x = half2_floats(y[i]);
                y[i] = half2_bits(fmaf(d[2 * i], factor, x.x), fmaf(d[2 * i + 1], factor, x.y));
              }
            }
            if (!ok) {
#pragma unroll
              for (int i = 0; i < 16; ++i) y[i] = 0x7fff7fffu;
            }
            if (direct) {  // whole sectors
              if (row >= 0) {
                __half* p = static_cast<__half*>(a.out) + (int64_t)row * a.out_stride + n;
#pragma unroll
                for (int c = 0; c < 16; c += 8)
                  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p + 2 * c), "r"(y[c]), "r"(y[c + 1]),
                               "r"(y[c + 2]), "r"(y[c + 3]), "r"(y[c + 4]), "r"(y[c + 5]), "r"(y[c + 6]), "r"(y[c + 7])
                               : "memory");
              }
              __syncwarp();  // the next columns' loads from tensor memory want a whole warp
            } else {  // through the base's place
#pragma unroll
              for (int c = 0; c < 4; ++c) store16(tile + swizzled(r, ch0 + c), y[4 * c], y[4 * c + 1], y[4 * c + 2], y[4 * c + 3]);
            }
          }
          if (!direct && n_own < n1)
            store_loose(static_cast<unsigned short*>(a.out) + n_own, a.out_stride, tile, quarter * 32, row, min(kOwnCols, n1 - n_own));
          // where bases or results went through these bytes, a tensor copy may write them next
          if ((a.base && !base_vec) || !direct) tc::fence_proxy_async_smem();
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0 && ok) {
          if (w.rank > 0) mbar_arrive(&d2_empty[b]);
          mbar_arrive(&empty_epi[slot]);
        }
        if (w.rank > 0) ++results;
        if (++slot == S) slot = 0;
      }
    }
  }
  __syncwarp();  // lanes leave a bounded wait each at its own time
  pdl_wait();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  cluster_arrive();  // nobody reads or writes this CTA's memory any more
  cluster_wait();
  if (warp == 4) tc::tmem_dealloc(tmem, 512);
}

// CTAs of a cluster: the number with the shortest longest queue, an item's time being its part of a tile and a fixed sixteenth
// of one (start, exchange). room: how many clusters of each size the GPU holds.
constexpr int kMostCtas = 8;
int tile_cluster(int items, const int (&room)[kMostCtas]) {
  int best = 0;
  double least = 1e30;
  for (int i = 0; i < kMostCtas; ++i) {
    if (room[i] < 1) continue;
    const int rounds = (items + room[i] - 1) / room[i];
    const double time = rounds * (1.0 / (i + 1) + 1.0 / 16);
    if (time < least) least = time, best = i;
  }
  return best;
}

// Boxes of 128 rows and 64 columns of a [M, cols] matrix; false where it can't be one (rows then come one by one).
bool make_map(CUtensorMap* map, const void* p, int M, int cols, int64_t stride) {
  auto encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encode_fn());
  if (!encode || !p || stride % 8 != 0 || stride >= (int64_t)1 << 38) return false;
  const cuuint64_t dim[2] = {(cuuint64_t)cols, (cuuint64_t)M}, pitch[1] = {(cuuint64_t)stride * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)kRows}, step[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(p), dim, pitch, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int RP>
cudaError_t launch_tile(LaunchCtx& ctx, const Lora& a) {
  using L = TileGeo<RP>;
  auto kern = lora_tile_kernel<RP>;
  static std::atomic<uint64_t> sized{0};
  cudaError_t e = allow_smem(kern, L::kBytes, ctx.device, sized);
  if (e != cudaSuccess) return e;
  CUtensorMap x_map = {}, base_map = {};
  const int maps = (make_map(&x_map, a.x, a.M, a.K, a.x_stride) ? 1 : 0) | (make_map(&base_map, a.base, a.M, a.N, a.base_stride) ? 2 : 0);
  const List list(a.workspace);
  e = launch_kernel(ctx, list_kernel<kRows>, dim3(1), dim3(1024), 0, a, kSmallItem, 1, list.counts, list.items, a.M, ctx.status);
  if (e != cudaSuccess) return e;
  static std::atomic<int> known[kMostCtas][64];
  int room[kMostCtas];
  for (int i = 0; i < kMostCtas; ++i) room[i] = clusters_held(ctx, kern, i + 1, kThreads, L::kBytes, known[i]);
  // A tile in which one prompt ends and the next begins is two items. (Where they are more than thought, a few clusters get two: 1784 rows of four
  // prompts 28.4 us instead of 22.3 with clusters of 6, which take 22.3 for two prompts, too, instead of 19.5.)
  const int tiles = (a.M + kRows - 1) / kRows;
  const int pick = tile_cluster(tiles + tiles / 8, room), cluster = pick + 1, clusters = room[pick] > 0 ? room[pick] : 1;
  const bool pdl = ctx.pdl;
  ctx.pdl = true;  // it waits for the list on the device
  e = launch_clusters(ctx, kern, cluster, dim3((unsigned)(clusters * cluster)), dim3(kThreads), L::kBytes, a, x_map, base_map, maps,
                      cluster, (const uint32_t*)list.counts, (const Item*)list.items, ctx.status);
  if (e == cudaSuccess) e = launch_lora_small(ctx, a);
  ctx.pdl = pdl;
  return e;
}

}  // namespace

cudaError_t launch_lora_tile(LaunchCtx& ctx, const Lora& a) {
  if (a.max_rank <= 16) return launch_tile<16>(ctx, a);
  if (a.max_rank <= 32) return launch_tile<32>(ctx, a);
  if (a.max_rank <= 64) return launch_tile<64>(ctx, a);
  return launch_tile<128>(ctx, a);
}

}  // namespace mnb
