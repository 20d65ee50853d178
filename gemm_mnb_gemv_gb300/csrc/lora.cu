// Low-rank adapters of many requests beside a shared product:
//   out[m] = base[m] + scale[a] * up[a] (down[a] x[m]),  a = adapter[m].
//
// A cluster of CTAs takes an item, the rows of one adapter in a tile, in one launch for both products:
//   1. s = down x: the CTAs split K; partial sums meet in shared memory, over the warps and then over the cluster;
//   2. out = base + up s: the CTAs split N, each with all of s.
// Tiles have 16 rows (decode and verify steps, and the items of up to 16 rows that the tcgen05 kernel leaves) or, for many rows in
// fp32, 64. One ring of asynchronous copies feeds both products: a stage is 32 WN of K (x and down) or 32 WN columns of N (base
// and up), and the first stages of the second product are on their way while the first one's sums are joined.
// Rows are the M side of the warp's matrix instructions, ranks (then output columns) the N side; a lane takes 8 consecutive
// elements of the inner index, which both operands number alike.
// s is held as two fp16 after its row was scaled by a power of two to [2^13, 2^14), and up takes both: 22 bits of s. fp32: x, too, as two
// fp16, of the scale of the 32 elements that a granule of K has of a row; each is multiplied on its own and the granule's scale put
// back in fp32 (2^-22; two tf32 parts took twice the instructions at half their rate).
// Bound: what a warp has to issue, one after the other. 64 rows of 48 adapters of up to 64 ranks, K = N = 4096, take 15.5 us, 2.7 of them
// bytes at the copy rate. By the clock: 2 to find the adapter, 4 for the first product, 2 for its sums, 4 for the second product, the last CTAs 2.5
// later, 1 from launch to launch; in the 10 us of its products a warp issues about 2860 instructions, 7 cycles each (12 warps an SM,
// registers allow 16). With one part of s instead of two: 14.7. Weights straight from memory to the products' registers, without the
// ring: 22 us against 14.7 (half of each line at a time, and spills); a ring for each warp, without barriers: the same.  One row of rank 16: 6.1
// us, a chain: adapter 1.2, first product 1.4, its sums 1.4, second product 1.3, launch to launch 0.8.
#include <type_traits>

#include "cluster.cuh"
#include "lora.cuh"
#include "mma_sync.cuh"

namespace mnb {
namespace {

using namespace lora;

// Of two rows; out of line: inlined, rows at 16 bytes paid 1 to 2 % for the code.
template <int kWords>
struct LooseRows {
  uint32_t y[2][kWords];
};
template <typename T, int kWords>
__device__ __noinline__ LooseRows<kWords> loose_rows(const T* base, int64_t at0, int64_t at1, int64_t end, int width) {
  LooseRows<kWords> r;
  loose_row(base, at0, end, width, r.y[0]);
  loose_row(base, at1, end, width, r.y[1]);
  return r;
}

// Rows up to which each cluster finds its tile's adapters itself, in one launch. Beyond, a launch makes a list of all items but each tile's first.
// On the GPU, without a list / with one: 64 rows of 64 adapters, 4096 x 4096, rank 16 9.7 / 11.0, 132 rows of them 22.9 / 17.3; fp32, four rows a
// request, 896 x 1152, rank 8: 64 rows 6.5 / 7.5, 132 8.2 / 7.6, 256 10.0 / 8.0; 803 rows of three prompts and 8 more, 1680 x 192: 14.1 / 7.9. A
// call without one has one launch and no workspace, 3 us less of host time, which eager calls of this size are bound by (18 us for 8 on the GPU); replayed
// ones of more than 130 rows would be faster with a list.
constexpr int kFewRows = 256;
// Rows up to which tiles have 16 rows. More come in tiles of 64 (fp32) or 128 (fp16, the tcgen05 kernel), which read the weights that
// much less often but fill the GPU later; a GPU holds 74 clusters, the tiles of 1184 rows. Four prompts, us in tiles of 16 / in the large ones:
//   fp16, K = N = 4096: rank 16 12.4 / 18.3 at 1152 rows, 18.7 / 18.3 at 1536; rank 32 15.4 / 18.7 and 23.0 / 18.9; rank 64 18.4 / 20.2 at 768, 21.1 / 20.2 at
//   1024; rank 128 32 / 25 at 272, 61 / 25 at 768. 4096 x 14336: rank 32 26.8 / 31.9 at 1152, 42 / 34 at 1536; rank 64 31.5 / 34.1 at 768, 37.1 / 33.9 at 1024.
//   1024 x 1024, where a launch counts for more: rank 64 13.7 / 14.3 at 1024, 19.4 / 14.9 at 1536.
//   fp32, K = N = 4096: rank 32 25.5 / 26.7 at 1152, 28.0 / 26.9 at 1536; rank 64 17.5 / 24.8 at 512, 28.6 / 24.9 at 768; rank 128 35.8 / 32.2 at 272. 4096 x
//   14336: rank 64 50.5 / 51.8 at 768, 81 / 75 at 1536; rank 128 62 / 65 at 272, 91 / 66 at 512. 1024 x 1024: rank 32 13.3 / 11.4 at 1024, rank 64 10.5 / 11.3
//   at 512 and 15.9 / 11.5 at 768: fp32's border is too far out for small layers.
constexpr int tile_rows(int max_rank) { return max_rank > 64 ? 256 : max_rank > 32 ? 768 : 1152; }
// Whether calls of this kind of tile take a list: those of 16 rows and ranks above 64 have no more rows than need none, and in fp16 only the
// launch for small items.
constexpr bool takes_list(int RB, int WM) { return WM > 1 || tile_rows(8 * RB) > kFewRows; }

// RB: ranks in eights; WM: row tiles of 16.
template <int RB, int WM, bool F32>
struct Geo {
  static constexpr int kWarps = WM == 1 ? 4 : 8, kThreads = kWarps * 32;
  static constexpr int RP = RB * 8, TM = 16 * WM, WN = kWarps / WM;
  static constexpr int kSpan = 32 * WN;                       // of K or N in a stage
  static constexpr int kElem = F32 ? 4 : 2;
  static constexpr int kRow = kSpan * kElem;                  // bytes of a row of x or base in a stage
  static constexpr int kDownRow = kSpan * 2, kUpRow = RP * 2;  // of down, up
  static constexpr int kAct = TM * kRow, kWeight = RP * kSpan * 2;
  static constexpr int kStage = kAct + kWeight;
  static constexpr int kPart = (WN - 1) * TM * RP * 4;        // partial sums of the warps; the CTA's own in the first
  static constexpr int kSRow = RP >= 64 ? RP * 2 + 64 : RP * 2;  // bytes of a row of s
  // The low parts lie behind the high ones or, with tiles of 16 rows in fp16, over the partial sums of the other warps, which are joined by
  // then (and which the other CTAs do not read): room for one more stage or CTA hangs on it.
  static constexpr int kSHalf = (TM * kSRow + 127) / 128 * 128, kS = kSHalf * (F32 ? 2 : 1);
  static constexpr int kLow = F32 ? kSHalf : TM * RP * 4 - kPart;  // from the high parts
  static_assert(F32 || (WN > 2 && kSHalf <= (WN - 2) * TM * RP * 4), "the low parts fit over the other warps' sums");
  // Stages that fit when an SM holds n CTAs. As many CTAs as can have three, or else two (16 warps an SM are what registers allow).
  static constexpr int fit(int n) {
    const int stages = (228 * 1024 / n - 1024 - 768 - kPart - kS) / kStage;
    return stages > 4 ? 4 : stages;
  }
  static constexpr int most(int stages) {
    int n = 16 / kWarps;
    while (n > 1 && fit(n) < stages) --n;
    return n;
  }
  static constexpr int kCtas = fit(most(3)) >= 3 && most(3) + 1 >= most(2) ? most(3) : most(2);
  static constexpr int kStages = fit(kCtas);
  static constexpr int kBytes = kStages * kStage + kPart + kS;
  static_assert(kStages >= 2, "one stage is read while the next one lands");
  // With few stages a slot is filled again behind a second barrier, as soon as it is free; with more, behind the next stage's.
  static constexpr bool kFew = kStages <= 3;
  static constexpr int kAhead = kFew ? kStages : kStages - 1;
};

// Where 16-byte chunk `chunk` of a row lies in it: the chunks that a quarter warp reads of two neighbouring rows come from
// distinct banks. fp16: chunks 4 i + t of each; fp32: 2 (4 i + t) and its neighbour.
template <bool F32>
__device__ __forceinline__ int place(int row, int chunk) {
  return (chunk ^ ((row & 1) * (F32 ? 1 : 4))) * 16;
}
template <int RP>
__device__ __forceinline__ int up_place(int row, int chunk) {  // rows of 64 bytes and less are neighbours without conflicts
  return (chunk ^ (RP >= 64 ? (row & 1) * 4 : 0)) * 16;
}

template <int RB, int WM, bool F32>
__global__ void __launch_bounds__(Geo<RB, WM, F32>::kThreads, Geo<RB, WM, F32>::kCtas)
    lora_kernel(const Lora a, int cluster, int subs, const uint32_t* counts, const Item* list, int capacity, int small_only, uint32_t* status) {
  using T = std::conditional_t<F32, float, __half>;
  using L = Geo<RB, WM, F32>;
  if constexpr (F32 && !takes_list(RB, WM)) list = nullptr;
  constexpr int RP = L::RP, TM = L::TM, WN = L::WN, S = L::kStages, kThreads = L::kThreads;
  constexpr int E = RB >= 4 ? 8 : RB == 2 ? 4 : 2;  // elements of the rank that a lane has of a chunk of 4 E
  constexpr int KC = RP / (4 * E);
  extern __shared__ __align__(128) uint8_t smem[];
  float* part = reinterpret_cast<float*>(smem + S * L::kStage);
  uint8_t* s_mem = smem + S * L::kStage + L::kPart;
  __shared__ int rows[TM];
  __shared__ float factors[TM];
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, g = lane / 4, t = lane % 4;
  const int wm = warp % WM, wn = warp / WM;
  const int cta = cluster_ctarank(), id = blockIdx.x / cluster;
  const uint32_t ring = smem_u32(smem);
  pdl_launch_dependents();
  if (!list) pdl_wait();  // the list's launch lets this one start when its own inputs are there

  const int granules = (a.K + 31) / 32, blocks = (a.N + 31) / 32;
  const int g0 = (int)((int64_t)granules * cta / cluster), g1 = (int)((int64_t)granules * (cta + 1) / cluster);
  const int b0 = (int)((int64_t)blocks * cta / cluster), b1 = (int)((int64_t)blocks * (cta + 1) / cluster);
  constexpr int kVec = 16 / sizeof(T);
  const bool base_vec = a.base && a.base_stride % kVec == 0, out_vec = a.out_stride % kVec == 0;
  const bool in_place = a.base == a.out;

  // With a list: the first item of each tile (the rows of its first row's adapter), which the clusters find themselves while the list is
  // being made, then its items; or its small ones alone. Without one each cluster finds its tile's adapters itself: cluster `id` takes
  // tile id / subs and every subs-th of its adapters, in the order of their first rows.
  const int tiles = list && !small_only ? (a.M + TM - 1) / TM : 0;
  constexpr int kUnknown = 0x7fffffff;
  int big = 0, items, first, step, of_row = -2;
  uint32_t same = 0, firsts = 0;
  const int m0 = id / subs * TM;
  if (list) {
    items = small_only ? (int)__ldcg(counts + 1) : kUnknown, first = id, step = gridDim.x / cluster;
  } else {
    first = id % subs, step = subs;
    if (lane < TM && m0 + lane < a.M) {
      of_row = max(a.adapter[m0 + lane], -1);
      if (of_row >= a.count) {
        if (first == 0 && cta == 0 && warp == 0) report_status(status, kStatusBadIndex);
        of_row = -1;
      }
    }
    same = __match_any_sync(kFull, of_row);
    firsts = __ballot_sync(kFull, of_row != -2 && __ffs(same) - 1 == lane);
    items = __popc(firsts);
    for (int k = 0; k < first; ++k) firsts &= firsts - 1;
  }
  for (int it = first;; it += step) {
    if (it >= tiles && items == kUnknown) {
      pdl_wait();
      big = (int)__ldcg(counts), items = tiles + big + (int)__ldcg(counts + 1);
    }
    if (it >= items) break;
    Item item;
    if (it < tiles) {
      constexpr int H = (TM + 31) / 32;
      int v[H];
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const int i = 32 * h + lane;
        const bool in = i < TM && it * TM + i < a.M;
        v[h] = in ? __ldcg(a.adapter + it * TM + i) : 0;
        v[h] = !in ? -2 : v[h] < 0 || v[h] >= a.count ? -1 : v[h];
      }
      item = {it * TM, __shfl_sync(kFull, v[0], 0), {0, 0}};
#pragma unroll
      for (int h = 0; h < H; ++h) item.rows[h / 2] |= (uint64_t)__ballot_sync(kFull, v[h] == item.adapter) << (h % 2 * 32);
    } else if (list) {
      const int at = it - tiles;
      const uint64_t* p = reinterpret_cast<const uint64_t*>(list + (at < big ? at : capacity - 1 - (at - big)));
      const uint64_t head = __ldcg(p);
      item = {(int)(uint32_t)head, (int)(head >> 32), {__ldcg(p + 1), __ldcg(p + 2)}};
    } else {
      const int from = __ffs(firsts) - 1;
      item = {m0, __shfl_sync(kFull, of_row, from), {__shfl_sync(kFull, same, from), 0}};
      for (int k = 0; k < step; ++k) firsts &= firsts - 1;
    }
    const int n_rows = __popcll(item.rows[0]) + __popcll(item.rows[1]), value = item.adapter;
    const int rank = value < 0 ? 0 : a.ranks ? min(max(__ldcg(a.ranks + value), 0), a.max_rank) : a.max_rank;
    if (rank == 0 && in_place) continue;
    __syncthreads();  // the item before is done with rows, s and the ring
    if (tid < 128 && (item.rows[tid / 64] >> (tid % 64) & 1))
      rows[(tid < 64 ? 0 : __popcll(item.rows[0])) + __popcll(item.rows[tid / 64] & ((1ull << (tid % 64)) - 1))] = item.m0 + tid;
    __syncthreads();

    const int down_stages = rank > 0 ? (g1 - g0 + WN - 1) / WN : 0;
    const int stages = down_stages + (b1 - b0 + WN - 1) / WN;
    // What a copy needs is worked out ahead, as every operation is on the way of the copies behind it: a thread has one chunk of
    // rows that lie whole passes apart, of x and base, of down and of up.
    constexpr int kChunks = L::kRow / 16, kPass = kThreads / kChunks, kPasses = TM / kPass;
    constexpr int kDownChunks = L::kDownRow / 16, kDownPass = kThreads / kDownChunks, kDownPasses = (RP + kDownPass - 1) / kDownPass;
    constexpr int kUpChunks = L::kUpRow / 16, kUpPass = kThreads / kUpChunks, kUpPasses = (L::kSpan + kUpPass - 1) / kUpPass;
    static_assert(kPass % 2 == 0 && kDownPass % 2 == 0 && kUpPass % 2 == 0, "a chunk's place depends on its row's parity");
    const int xr = tid / kChunks, xc = tid % kChunks, dr = tid / kDownChunks, dc = tid % kDownChunks, ur = tid / kUpChunks, uc = tid % kUpChunks;
    const uint32_t x_to = xr * L::kRow + place<F32>(xr, xc), d_to = L::kAct + dr * L::kDownRow + place<false>(dr, dc);
    const uint32_t u_to = L::kAct + ur * L::kUpRow + up_place<RP>(ur, uc);
    const T *x_at[kPasses], *base_at[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int64_t row = xr + i * kPass < n_rows ? rows[xr + i * kPass] : 0;
      x_at[i] = static_cast<const T*>(a.x) + row * a.x_stride + xc * kVec;
      base_at[i] = static_cast<const T*>(a.base) + row * a.base_stride + xc * kVec;
    }
    const __half* down = static_cast<const __half*>(a.down) + ((int64_t)value * a.max_rank + dr) * a.K + dc * 8;
    const __half* up = static_cast<const __half*>(a.up) + ((int64_t)value * a.N + ur) * a.max_rank + uc * 8;
    const int64_t down_step = (int64_t)kDownPass * a.K, up_step = (int64_t)kUpPass * a.max_rank;
    const int up_have = min(rank - 8 * uc, 8);  // of this thread's chunk of the rank
    auto issue = [&](int q) {
      if (q < stages) {
        const uint32_t at = ring + q % S * L::kStage;
        if (q < down_stages) {
          const int k0 = (g0 + q * WN) * 32, k1 = min(a.K, g1 * 32);
          const bool x_in = k0 + xc * kVec < k1, d_in = k0 + dc * 8 < k1;
#pragma unroll
          for (int i = 0; i < kPasses; ++i)
            if (xr + i * kPass < n_rows) {
              if (x_in) copy16(at + x_to + i * (kPass * L::kRow), x_at[i] + k0);
              else store_zeros(at + x_to + i * (kPass * L::kRow));
            }
#pragma unroll
          for (int i = 0; i < kDownPasses; ++i)
            if (dr + i * kDownPass < rank) {  // columns of s beyond the rank are not used
              if (d_in) copy16(at + d_to + i * (kDownPass * L::kDownRow), down + i * down_step + k0);
              else store_zeros(at + d_to + i * (kDownPass * L::kDownRow));
            }
        } else {
          const int n0 = (b0 + (q - down_stages) * WN) * 32, n1 = min(a.N, b1 * 32);
          if (base_vec) {
            const int bytes = (n1 - n0 - xc * kVec) * (int)sizeof(T);
#pragma unroll
            for (int i = 0; i < kPasses; ++i)
              if (xr + i * kPass < n_rows && bytes > 0) {
                if (bytes >= 16) copy16(at + x_to + i * (kPass * L::kRow), base_at[i] + n0);
                else copy_some(at + x_to + i * (kPass * L::kRow), base_at[i] + n0, bytes);
              }
          }
          const __half* p = up + (int64_t)n0 * a.max_rank;
          if (up_have == 8) {
#pragma unroll
            for (int i = 0; i < kUpPasses; ++i)
              if (ur + i * kUpPass < min(L::kSpan, n1 - n0)) copy16(at + u_to + i * (kUpPass * L::kUpRow), p + i * up_step);
          } else if (up_have > 0) {
            for (int i = 0; i < kUpPasses; ++i)
              if (ur + i * kUpPass < min(L::kSpan, n1 - n0)) copy_some(at + u_to + i * (kUpPass * L::kUpRow), p + i * up_step, 2 * up_have);
          } else if (8 * uc < (rank + 4 * E - 1) / (4 * E) * (4 * E)) {  // zeros behind the rank, as far as the products read
#pragma unroll
            for (int i = 0; i < kUpPasses; ++i)
              if (ur + i * kUpPass < L::kSpan) store_zeros(at + u_to + i * (kUpPass * L::kUpRow));
          }
        }
      }
      copy_commit();
    };
    for (int q = 0; q < L::kAhead; ++q) issue(q);

    const bool live = wm * 16 < n_rows;
    float acc[RB][4];
#pragma unroll
    for (int j = 0; j < RB; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] = 0.0f;
    int q = 0;
    // ---- s = down x over this CTA's part of K ----
    for (; q < down_stages; ++q) {
      copy_wait<L::kAhead - 1>();
      __syncthreads();
      if (!L::kFew) issue(q + L::kAhead);
      if (live) {
        const uint32_t act = ring + q % S * L::kStage, weight = act + L::kAct;
        const int r0 = wm * 16 + g;
        // Rows beyond the last and ranks beyond the item's hold what was there: they do not reach the others' sums. Four eights of the rank
        // at a time: their loads and products do not wait for each other.
        constexpr int kGroup = RB < 4 ? RB : 4;
        if constexpr (F32) {
          float x[2][8];
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int r = r0 + 8 * h;
              const uint4 v = lds128_a(act + r * L::kRow + place<true>(r, 2 * (4 * wn + t) + i));
              x[h][4 * i] = __uint_as_float(v.x), x[h][4 * i + 1] = __uint_as_float(v.y);
              x[h][4 * i + 2] = __uint_as_float(v.z), x[h][4 * i + 3] = __uint_as_float(v.w);
            }
          Split v[2][4];
          float back[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[h][i]));
            top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));  // four lanes have the granule's 32 elements of a row
            top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
            const int p = row_power(top);
            const float f = pow2(-p);
            back[h] = pow2(p);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[h][i] = split(x[h][2 * i] * f, x[h][2 * i + 1] * f);
          }
#pragma unroll
          for (int j0 = 0; j0 < RB; j0 += kGroup) {
            if (j0 * 8 < rank) {
              uint4 w[kGroup];
#pragma unroll
              for (int j = 0; j < kGroup; ++j) w[j] = lds128_a(weight + ((j0 + j) * 8 + g) * L::kDownRow + place<false>(g, 4 * wn + t));
              float d[kGroup][4];
#pragma unroll
              for (int j = 0; j < kGroup; ++j) mma16816_zero(d[j], v[0][0].lo, v[1][0].lo, v[0][1].lo, v[1][1].lo, w[j].x, w[j].y);
#pragma unroll
              for (int j = 0; j < kGroup; ++j) mma16816(d[j], v[0][2].lo, v[1][2].lo, v[0][3].lo, v[1][3].lo, w[j].z, w[j].w);
#pragma unroll
              for (int j = 0; j < kGroup; ++j) mma16816(d[j], v[0][0].hi, v[1][0].hi, v[0][1].hi, v[1][1].hi, w[j].x, w[j].y);
#pragma unroll
              for (int j = 0; j < kGroup; ++j) mma16816(d[j], v[0][2].hi, v[1][2].hi, v[0][3].hi, v[1][3].hi, w[j].z, w[j].w);
#pragma unroll
              for (int j = 0; j < kGroup; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[j0 + j][i] = fmaf(d[j][i], back[i / 2], acc[j0 + j][i]);
            }
          }
        } else {
          uint4 x[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) x[h] = lds128_a(act + (r0 + 8 * h) * L::kRow + place<false>(g, 4 * wn + t));
#pragma unroll
          for (int j0 = 0; j0 < RB; j0 += kGroup) {
            if (j0 * 8 < rank) {
              uint4 w[kGroup];
#pragma unroll
              for (int j = 0; j < kGroup; ++j) w[j] = lds128_a(weight + ((j0 + j) * 8 + g) * L::kDownRow + place<false>(g, 4 * wn + t));
#pragma unroll
              for (int j = 0; j < kGroup; ++j) mma16816(acc[j0 + j], x[0].x, x[1].x, x[0].y, x[1].y, w[j].x, w[j].y);
#pragma unroll
              for (int j = 0; j < kGroup; ++j) mma16816(acc[j0 + j], x[0].z, x[1].z, x[0].w, x[1].w, w[j].z, w[j].w);
            }
          }
        }
      }
      if (L::kFew) {
        __syncthreads();
        issue(q + L::kAhead);
      }
    }
    if (rank > 0) {
      // ---- over the warps ----
      auto at = [&](int w, int r, int col) { return part + ((w * TM + r) * RP + col); };
      const int r0 = wm * 16 + g;
      if (live && wn > 0) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (wm * 16 + 8 * h < n_rows) {
#pragma unroll
            for (int j = 0; j < RB; ++j)
              *reinterpret_cast<float2*>(at(wn - 1, r0 + 8 * h, j * 8 + 2 * t)) = make_float2(acc[j][2 * h], acc[j][2 * h + 1]);
          }
      }
      __syncthreads();
      if (live && wn == 0) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (wm * 16 + 8 * h < n_rows) {
#pragma unroll
            for (int j = 0; j < RB; ++j) {
              float2 v = make_float2(acc[j][2 * h], acc[j][2 * h + 1]);
#pragma unroll
              for (int w = 0; w < WN - 1; ++w) {
                const float2 o = *reinterpret_cast<float2*>(at(w, r0 + 8 * h, j * 8 + 2 * t));
                v.x += o.x, v.y += o.y;
              }
              *reinterpret_cast<float2*>(at(0, r0 + 8 * h, j * 8 + 2 * t)) = v;
            }
          }
      }
      // ---- over the cluster; every CTA gets all of s. RP / 4 neighbouring lanes have a row. Few rows: each CTA reads all of them; many: it
      // reads its share and hands the result to the others (an eighth of the reads, one barrier more) ----
      constexpr bool kShare = WM > 1;
      cluster_arrive();
      cluster_wait();
      const float scale = a.scales ? __ldcg(a.scales + value) : 1.0f;
      const int e_first = kShare ? TM * cta / cluster * RP : 0, e_end = kShare ? min(TM * (cta + 1) / cluster, n_rows) * RP : n_rows * RP;
      for (int e0 = e_first + warp * 128; e0 < e_end; e0 += kThreads * 4) {
        // a warp may reach beyond the last row, in a tile or a share that is less than 128 elements
        const bool mine = e0 + lane * 4 < e_end;
        const int e = mine ? e0 + lane * 4 : e_first, r = e / RP, col = e % RP;
        float4 v = cluster_sum_f4(smem_u32(part + e), cluster);
        if (col + 4 > rank) {
          if (col >= rank) v.x = 0.0f;
          if (col + 1 >= rank) v.y = 0.0f;
          if (col + 2 >= rank) v.z = 0.0f;
          v.w = 0.0f;
        }
        uint8_t* row = s_mem + r * L::kSRow;
        float top = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
#pragma unroll
        for (int o = 1; o < RP / 4; o <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
        const int p = row_power(top);
        const float f = pow2(-p);
        const Split x = split(v.x * f, v.y * f), y = split(v.z * f, v.w * f);
        if constexpr (kShare) {
          const uint32_t to = smem_u32(row + col * 2);
          for (int c = 0; mine && c < cluster; ++c) {
            cluster_st_u64(cluster_map(to, c), x.hi, y.hi);
            cluster_st_u64(cluster_map(to + L::kLow, c), x.lo, y.lo);
            if (col == 0) cluster_st_f32(cluster_map(smem_u32(&factors[r]), c), scalbnf(scale, p));
          }
        } else if (mine) {
          *reinterpret_cast<uint2*>(row + col * 2) = make_uint2(x.hi, y.hi);
          *reinterpret_cast<uint2*>(row + L::kLow + col * 2) = make_uint2(x.lo, y.lo);
          if (col == 0) factors[r] = scalbnf(scale, p);
        }
      }
      __syncwarp();      // the cluster's barriers want whole warps
      cluster_arrive();  // no more reads of the others' sums
      if (kShare) cluster_wait();
    }

    // ---- out = base + up s over this CTA's part of N ----
    // Column c of the product's 8-column tile j is output column 8 (c / 2) + 2 j + c % 2 of the warp's 32: a lane then has
    // 8 consecutive ones, of four tiles.
    for (; q < stages; ++q) {
      constexpr int kWords = F32 ? 8 : 4;
      const int r0 = wm * 16 + g;
      const int n_warp = (b0 + (q - down_stages) * WN + wn) * 32, n = n_warp + 8 * t, width = min(8, min(a.N, b1 * 32) - n);
      LooseRows<kWords> base;  // as they lie
      auto& y = base.y;
      copy_wait<L::kAhead - 1>();
      __syncthreads();
      if (!L::kFew) issue(q + L::kAhead);
      if (live) {
        const uint32_t act = ring + q % S * L::kStage, weight = act + L::kAct;
        if (!base_vec) {
          auto at = [&](int r) { return a.base && r < n_rows ? rows[r] * a.base_stride + n : -1; };
          base = loose_rows<T, kWords>(static_cast<const T*>(a.base), at(r0), at(r0 + 8), base_end(a), width);
        }
        float d[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) d[j][i] = 0.0f;
        if (rank > 0) {
#pragma unroll
          for (int c = 0; c < KC; ++c) {
            if (4 * E * c < rank) {
              uint32_t w[4][E / 2];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const int r = 32 * wn + 8 * (g / 2) + 2 * j + g % 2;
                const uint32_t p = weight + r * L::kUpRow;
                if constexpr (E == 8) {
                  const uint4 v = lds128_a(p + up_place<RP>(r, 4 * c + t));
                  w[j][0] = v.x, w[j][1] = v.y, w[j][2] = v.z, w[j][3] = v.w;
                } else if constexpr (E == 4) {
                  const uint2 v = lds_u64_a(p + 8 * t);
                  w[j][0] = v.x, w[j][1] = v.y;
                } else {
                  w[j][0] = lds_u32_a(p + 4 * t);
                }
              }
#pragma unroll
              for (int part = 1; part >= 0; --part) {  // the low parts first
                uint32_t x[2][E / 2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const uint32_t p = smem_u32(s_mem + part * L::kLow + (r0 + 8 * h) * L::kSRow) + (4 * E * c + E * t) * 2;
                  if constexpr (E == 8) {
                    const uint4 v = lds128_a(p);
                    x[h][0] = v.x, x[h][1] = v.y, x[h][2] = v.z, x[h][3] = v.w;
                  } else if constexpr (E == 4) {
                    const uint2 v = lds_u64_a(p);
                    x[h][0] = v.x, x[h][1] = v.y;
                  } else {
                    x[h][0] = lds_u32_a(p);
                  }
                }
#pragma unroll
                for (int s = 0; s < (E + 3) / 4; ++s)
#pragma unroll
                  for (int j = 0; j < 4; ++j) {
                    if constexpr (E == 2) mma16816(d[j], x[0][0], x[1][0], 0u, 0u, w[j][0], 0u);
                    else mma16816(d[j], x[0][2 * s], x[1][2 * s], x[0][2 * s + 1], x[1][2 * s + 1], w[j][2 * s], w[j][2 * s + 1]);
                  }
              }
            }
          }
        }
        // places of this lane's 8 columns of row r in the stage, and of the warp's column `col`
        auto own = [&](int r, int i) { return act + r * L::kRow + place<F32>(r, F32 ? 2 * (4 * wn + t) + i : 4 * wn + t); };
        auto col_at = [&](int r, int col) {
          return act + r * L::kRow + place<F32>(r, F32 ? 8 * wn + col / 4 : 4 * wn + col / 8) + (F32 ? col % 4 * 4 : col % 8 * 2);
        };
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = r0 + 8 * h;
          if (r < n_rows && width > 0) {
            if (base_vec) {
#pragma unroll
              for (int i = 0; i < kWords / 4; ++i) {
                const uint4 v = lds128_a(own(r, i));
                y[h][4 * i] = v.x, y[h][4 * i + 1] = v.y, y[h][4 * i + 2] = v.z, y[h][4 * i + 3] = v.w;
              }
            }
            if (rank > 0) {
              const float f = factors[r];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float d0 = d[i][2 * h], d1 = d[i][2 * h + 1];
                if constexpr (F32) {
                  y[h][2 * i] = __float_as_uint(fmaf(d0, f, __uint_as_float(y[h][2 * i])));
                  y[h][2 * i + 1] = __float_as_uint(fmaf(d1, f, __uint_as_float(y[h][2 * i + 1])));
                } else {
                  const float2 v = half2_floats(y[h][i]);
                  y[h][i] = half2_bits(fmaf(d0, f, v.x), fmaf(d1, f, v.y));
                }
              }
            }
            if (out_vec && width == 8) {
              uint4* p = reinterpret_cast<uint4*>(static_cast<T*>(a.out) + (int64_t)rows[r] * a.out_stride + n);
#pragma unroll
              for (int i = 0; i < kWords / 4; ++i) p[i] = make_uint4(y[h][4 * i], y[h][4 * i + 1], y[h][4 * i + 2], y[h][4 * i + 3]);
            } else {
#pragma unroll
              for (int i = 0; i < kWords / 4; ++i) store16(own(r, i), y[h][4 * i], y[h][4 * i + 1], y[h][4 * i + 2], y[h][4 * i + 3]);
            }
          }
        }
        // what a lane can't store as it has it goes out a row after the other
        const int whole = out_vec ? min(a.N, b1 * 32) / 8 * 8 : 0, col = n_warp + lane;
        if (n_warp + 32 > whole) {
          __syncwarp();
          if (col >= whole && col < min(a.N, b1 * 32)) {
#pragma unroll 4
            for (int i = wm * 16; i < min(wm * 16 + 16, n_rows); ++i) {
              T* p = static_cast<T*>(a.out) + (int64_t)rows[i] * a.out_stride + col;
              if constexpr (F32) *p = __uint_as_float(lds_u32_a(col_at(i, lane)));
              else *reinterpret_cast<unsigned short*>(p) = (unsigned short)lds_u16_a(col_at(i, lane));
            }
          }
        }
      }
      if (L::kFew) {
        __syncthreads();
        issue(q + L::kAhead);
      }
    }
    if (WM == 1 && rank > 0) {
      __syncwarp();
      cluster_wait();
    }
  }
  if (list) pdl_wait();  // who waits for this kernel waits for the one before it too
}

template <int RB, int WM, bool F32>
cudaError_t launch_lora_t(LaunchCtx& ctx, const Lora& a) {
  using L = Geo<RB, WM, F32>;
  auto kern = lora_kernel<RB, WM, F32>;
  static std::atomic<uint64_t> sized{0}, wide{0};
  const int tiles = (a.M + L::TM - 1) / L::TM;
  const int cluster = a.M <= 16 ? 16 : 8;
  cudaError_t e = allow_smem(kern, L::kBytes, ctx.device, sized);
  if (e == cudaSuccess && cluster > 8) e = allow_wide_clusters(kern, ctx.device, wide);
  if (e != cudaSuccess) return e;
  if (!takes_list(RB, WM) || (WM == 1 && a.M <= kFewRows)) {
    // A cluster for each adapter that a tile can have, as long as the GPU holds about that many: clusters without one cost their
    // start, adapters that share one come after each other.
    const int most = a.M < 16 ? a.M : 16, some = 8 * 16 / tiles;
    const int subs = some > most ? most : some < 2 ? 2 : some;
    return launch_clusters(ctx, kern, cluster, dim3((unsigned)(tiles * subs * cluster)), dim3(L::kThreads), L::kBytes, a, cluster, subs,
                           (const uint32_t*)nullptr, (const Item*)nullptr, 0, 0, ctx.status);
  }
  if constexpr (takes_list(RB, WM)) {
    const List list(a.workspace);
    e = launch_kernel(ctx, list_kernel<L::TM>, dim3(1), dim3(1024), 0, a, L::TM / 2, 1, list.counts, list.items, a.M, ctx.status);
    if (e != cudaSuccess) return e;
    const bool pdl = ctx.pdl;
    ctx.pdl = true;  // it waits for the list on the device
    static std::atomic<int> known[64];
    const int room = clusters_held(ctx, kern, cluster, L::kThreads, L::kBytes, known);
    e = launch_clusters(ctx, kern, cluster, dim3((unsigned)((room > 0 ? room : 1) * cluster)), dim3(L::kThreads), L::kBytes, a, cluster, 1,
                        (const uint32_t*)list.counts, (const Item*)list.items, a.M, 0, ctx.status);
    ctx.pdl = pdl;
  }
  return e;
}

template <int RB>
cudaError_t launch_lora_r(LaunchCtx& ctx, const Lora& a) {
  if (!a.f32) return launch_lora_t<RB, 1, false>(ctx, a);
  return a.M <= tile_rows(a.max_rank) ? launch_lora_t<RB, 1, true>(ctx, a) : launch_lora_t<RB, 4, true>(ctx, a);
}

template <int RB>
cudaError_t launch_small_r(LaunchCtx& ctx, const Lora& a) {
  using L = Geo<RB, 1, false>;
  auto kern = lora_kernel<RB, 1, false>;
  static std::atomic<uint64_t> sized{0};
  static std::atomic<int> known[64];
  const cudaError_t e = allow_smem(kern, L::kBytes, ctx.device, sized);
  if (e != cudaSuccess) return e;
  constexpr int cluster = 8;
  const int room = clusters_held(ctx, kern, cluster, L::kThreads, L::kBytes, known);
  const List list(a.workspace);
  const bool pdl = ctx.pdl;
  ctx.pdl = true;
  const cudaError_t r = launch_clusters(ctx, kern, cluster, dim3((unsigned)((room > 0 ? room : 1) * cluster)), dim3(L::kThreads), L::kBytes, a,
                                        cluster, 1, (const uint32_t*)list.counts, (const Item*)list.items, a.M, 1, ctx.status);
  ctx.pdl = pdl;
  return r;
}

}  // namespace

cudaError_t launch_lora_small(LaunchCtx& ctx, const Lora& a) {
  if (a.max_rank <= 8) return launch_small_r<1>(ctx, a);
  if (a.max_rank <= 16) return launch_small_r<2>(ctx, a);
  if (a.max_rank <= 32) return launch_small_r<4>(ctx, a);
  if (a.max_rank <= 64) return launch_small_r<8>(ctx, a);
  return launch_small_r<16>(ctx, a);
}

cudaError_t launch_lora_tile(LaunchCtx& ctx, const Lora& a);

size_t lora_workspace_bytes(int M) { return M > kFewRows ? 16 + (size_t)M * sizeof(Item) : 0; }

cudaError_t launch_lora(LaunchCtx& ctx, const Lora& a) {
  if (!a.f32 && a.M > tile_rows(a.max_rank)) {
    ctx.variant = "lora_tile_tcgen05";
    return launch_lora_tile(ctx, a);
  }
  ctx.variant = a.f32 ? "lora_f32" : "lora_f16";
  if (a.max_rank <= 8) return launch_lora_r<1>(ctx, a);
  if (a.max_rank <= 16) return launch_lora_r<2>(ctx, a);
  if (a.max_rank <= 32) return launch_lora_r<4>(ctx, a);
  if (a.max_rank <= 64) return launch_lora_r<8>(ctx, a);
  return launch_lora_r<16>(ctx, a);
}

}  // namespace mnb
