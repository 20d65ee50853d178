// Streaming attention over the paged 4-bit key/value cache (decode, verify, fp32 activations).
//
// Rows are (query token, head of the key head's group) pairs, 8 NT of them in a row tile, and are the N side
// of mma.sync m16n8k16; 16 keys (one block of the cache) are the M side of S = K Q^T and the
// K side of O^T = V^T P^T.  The cache's codes go into the products as small integers:
//   * K: the nibbles as they lie are fp16 subnormals (code * 2^-24, or * 2^-20 for the upper one of
//     a byte, undone in q), so one AND makes two operand elements and q . code is exact; a group's
//     scale multiplies its 32..128-element dot after it is formed, and offset_g * sum_{d in g} q_d is
//     added in fp32.
//   * V: codes become c - 8 (exact), probabilities become fp16(p * scale_g * 2^x) per group, and
//     sum_j p_j (offset + 8 scale) is kept in fp32.  Centring keeps the rounding of p * scale from being
//     multiplied by |offset| / |v| (fp32 activations centre K too: fp32 sums of uncentred products would lose
//     two bits).  With fp16 activations the power 2^x follows the largest scale among the keys that some row of the
//     tile sees, which then is 1 to 2; a scale 2^-y of it leaves its products a step of 2^(y - 33) of a row's largest
//     (2^-13 at y = 20).  With fp32 each group of each 16 keys has its own power, as their sums are added outside the
//     tensor cores anyway.
// A row's reference m moves only when a score passes it by 14 (in powers of two; one vote a
// block instead of shuffles) and is then set 8 below the largest: p = 2^(s - m) <= 2^14, so
// fp16 keeps probabilities down to 2^-22 of the largest normal.
// fp32 activations: q and p are split into two fp16 (2^-22 together), products run once for each.
//
// Work: tiles of 64 or 128 keys of every (sequence, row tile, key head) in one list, cut into equal ranges, one
// per resident CTA, on the device from the lengths (ragged batches balance, graphs
// follow new lengths).  Each of a CTA's four warps takes one or two 16-key blocks of a tile through its own
// ring of bulk copies (16 D + 128 ng bytes a block) that runs ahead across the ends of sequences; the
// warps meet only at a sequence's end.  Pieces of a sequence cut by a range's end go to the workspace
// as (m, l, o) and a second, dependent launch joins them in order.
// Bound: issue with four warps a scheduler (0.56 instructions a cycle, about 320 a block of 16 keys, ALU pipe 49%); at 128 registers
// 132 to 400 bytes a thread are spilled, 0.6% of the instructions. Measured at 32 / 8 heads of 128, graph replays: 64 ragged contexts of
// up to 8192 keys 74 us (3.9 TB/s; the bytes alone 43 us), one of 131071 keys 44 us, one of 1000 keys 11 us (launch,
// lengths, page, block and join one after the other); with heads of 256 64 contexts 119 us (86), fp32 101 us (heads of 128) and 186 (256).
// Every 16 rows read and convert the visible cache again: prompts of heads of 256 and of fp32, which no other kernel takes, are slow here
// (two prompts of up to 2048: 530 and 423 us; their products alone 34 and 17).
#pragma once

#include <type_traits>

#include "kv4_work.cuh"
#include "mma_sync.cuh"

namespace mnb {
namespace kv4 {

constexpr int kWarps = 4;      // warps of a CTA
constexpr int kPieceCost = 3;  // 64 ragged contexts: 1: 83.5 us, 2: 78.6, 3: 77.3, 4: 78.0, 6: 80.7, 8: 84.0

// 8 x 8 transpose of 16-bit elements across the warp.
__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// Codes to fp16 c - 8, exact, two at a time: the lower and the upper nibbles of two byte positions.
__device__ __forceinline__ uint32_t c_lower(uint32_t x) {
  uint32_t r = lop3_and_or(x, 0x000f000fu, 0x64006400u);  // 1024 + c
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(r), "r"(0xE408E408u));
  return r;
}
__device__ __forceinline__ uint32_t c_upper(uint32_t x) {
  uint32_t r = lop3_and_or(x, 0x00f000f0u, 0x64006400u);  // 1024 + 16 c
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(r), "r"(0x2C002C00u), "r"(0xD480D480u));
  return r;
}

// Power of two of an fp16 magnitude's bits: 2^e <= size < 2^(e + 1) for normal ones, smaller ones count as 2^-14.
__device__ __forceinline__ int half_exponent(uint32_t bits) { return max((int)(bits >> 10), 1) - 15; }
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// Shared memory of a CTA.
template <int D, int NG, int NT, int PB, bool F32>
struct Layout {
  static constexpr int kBlock = 16 * D + 128 * NG;                   // bytes of a cache block
  static constexpr int kQ = (D / 16) * NT * 32 * 8 * (F32 ? 2 : NT > 1 ? 1 : 0);  // q fragments
  static constexpr int kQs = NG * NT * 8 * 4;                        // row sums of q per group
  static constexpr int kCol = NT * 8 * 4;                            // score factors
  static constexpr int kEx = kWarps * 8 * 64 * 4;                    // exchange of 64 columns of o
  static constexpr int kMl = kWarps * NT * 8 * 8;                    // m, l of each warp
  static constexpr int kFixed = kQ + kQs + kCol + kEx + kMl + 1024;  // + barriers, flags, scan
  static constexpr int stages(int budget) {
    const int s = (budget - kFixed) / (kWarps * PB * kBlock);
    return s < 2 ? 2 : s > 16 ? 16 : s;
  }
};

// CTAs an SM holds: by registers (128, 168 or 255 a thread), and with heads of 256 by two stages of shared memory.
template <int D, int NT, bool F32>
constexpr int stream_ctas() {
  constexpr int o_regs = D / 4 * NT;
  return o_regs <= 32 ? (F32 ? 3 : 4) : o_regs <= 64 && D < 256 ? 3 : 2;
}

// Cache blocks (of 16 keys) that a warp takes at a time: two where registers hold their scores, for
// more independent chains and half the loop's own instructions.
template <int D, int NT>
constexpr int step_blocks() {
  return D / 4 * NT <= 64 ? 2 : 1;
}

template <int D, int NG, int NT, bool F32>
__global__ void __launch_bounds__(kWarps * 32, stream_ctas<D, NT, F32>())
    kv4_stream_kernel(const Kv4Cache c, const Kv4Attention a, uint64_t page_magic, uint32_t* status) {
  constexpr int RT = 8 * NT;
  constexpr int KW = D / 32;    // 32-element granules
  constexpr int VW = D / 64;    // V words of a lane's chunk
  constexpr int GR = KW / NG;   // granules of a group
  constexpr int PB = step_blocks<D, NT>();
  constexpr int kTile = 16 * PB * kWarps;  // keys of a work unit
  using L = Layout<D, NG, NT, PB, F32>;
  constexpr int block_bytes = L::kBlock, stage_bytes = PB * block_bytes;
  constexpr int stages = L::stages(227 * 1024 / stream_ctas<D, NT, F32>() - 1024);
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, g = lane / 4, t = lane % 4;
  uint8_t* ring = smem + warp * stages * stage_bytes;
  uint8_t* fixed = smem + kWarps * stages * stage_bytes;
  uint2* qf = reinterpret_cast<uint2*>(fixed);
  float* qsf = reinterpret_cast<float*>(fixed + L::kQ);
  float* colf = reinterpret_cast<float*>(fixed + L::kQ + L::kQs);
  float* exch = reinterpret_cast<float*>(fixed + L::kQ + L::kQs + L::kCol);
  float2* ml = reinterpret_cast<float2*>(fixed + L::kQ + L::kQs + L::kCol + L::kEx);
  uint8_t* misc = fixed + L::kQ + L::kQs + L::kCol + L::kEx + L::kMl;
  uint64_t* full = reinterpret_cast<uint64_t*>(misc) + warp * 16;  // [stage]
  int* flags = reinterpret_cast<int*>(misc + 512) + warp * 16;     // [stage] bit i: block i was read
  int64_t* scan = reinterpret_cast<int64_t*>(misc + 768);          // [10]

  if (lane < stages) mbar_init(&full[lane], 1);
  fence_mbar_init();
  pdl_launch_dependents();
  pdl_wait();

  // ---- the range of this CTA ----
  const Walk<RT, kTile, kPieceCost> walk(a, c);
  const int G = walk.G;
  Piece* pieces = reinterpret_cast<Piece*>(a.workspace);
  constexpr int kSlot = RT * (D + 2);  // floats of one partial result
  float* slots = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + kMaxCtas * sizeof(Piece));
  Range range;
  Cursor cur;
  if (!find_range(walk, status, scan, range, cur)) {
    if (tid == 0) pieces[blockIdx.x].first = -1;
    return;
  }
  const int64_t u0 = range.u0, u1 = range.u1;
  const int skipped = range.skipped;
  const Cut& cut = range.cut;

  // ---- the producer side of each warp: runs ahead of its consumer side by up to `stages` steps ----
  // Block numbers come in batches, lane i holding the i-th next; the page indices of the batch
  // after are on their way meanwhile.
  constexpr uint32_t kNone = 0xfffffffeu;  // nothing to read: past the end, or not in the cache
  const int ppb = c.page_blocks;
  Cursor pro = cur;
  int64_t pro_left = u1 - u0 + skipped;  // units, those of pro's piece cost included
  int pro_stage = 0, issued = 0;         // issued: steps of the batch that are used up
  int batch_n = 0, next_n = 0;           // steps of the batches
  uint32_t batch_at = 0, next_in = 0;    // this lane's block number, and block within its page
  int next_page = 0, next_kvh = 0;
  bool pro_new = true;                   // the piece cost of pro's part is still to be taken off
  auto fetch = [&]() {  // starts the next batch: tiles of one sequence and key head
    next_n = 0;
    while (next_n == 0) {
      if (pro_new) pro_left -= kPieceCost, pro_new = false;
      if (pro_left <= 0) return;
      const int tiles = (int)min((int64_t)min(32 / PB, pro.t1 - pro.tile), pro_left);
      const int first = pro.tile * kTile + warp * (16 * PB);  // this warp's first key
      next_n = min(tiles, max(0, (pro.n - first + kTile - 1) / kTile));
      const int key = first + lane / PB * kTile + lane % PB * 16;
      next_page = -2;
      if (lane < next_n * PB && key < pro.n) {
        const uint32_t blk = (uint32_t)key / 16;
        const uint32_t at = (uint32_t)((uint64_t)blk * page_magic >> 36);  // blk / ppb
        next_in = blk - at * ppb;
        next_page = max(a.page_table[(int64_t)pro.b * a.table_stride + at], -1);
      }
      next_kvh = pro.kvh;
      pro_left -= tiles;
      pro.tile += tiles;
      if (pro.tile == pro.t1 && pro_left > 0) walk.next_part(pro), pro_new = true;
    }
  };
  auto produce = [&]() {
    if (issued == batch_n) {
      if (next_n == 0) return;
      batch_n = next_n;
      issued = 0;
      const bool ok = next_page >= 0 && next_page < c.num_pages;
      if (next_page != -2 && !ok) report_status(status, kStatusBadIndex);
      batch_at = ok ? ((uint32_t)next_page * c.kv_heads + next_kvh) * ppb + next_in : kNone;
      fetch();
    }
    uint32_t at[PB];
#pragma unroll
    for (int i = 0; i < PB; ++i) at[i] = __shfl_sync(kFull, batch_at, issued * PB + i);
    ++issued;
    if (lane == 0) {
      uint64_t* bar = &full[pro_stage];
      uint8_t* dst = ring + pro_stage * stage_bytes;
      int have = 0;
#pragma unroll
      for (int i = 0; i < PB; ++i) have |= (at[i] != kNone) << i;
      flags[pro_stage] = have;
      if (have == 0) {
        mbar_arrive(bar);
      } else {
        mbar_arrive_expect_tx(bar, (have == 3 ? 2 : 1) * block_bytes);
        if (PB == 2 && have == 3 && at[PB - 1] == at[0] + 1) {
          bulk_g2s(dst, c.pages + (uint64_t)at[0] * block_bytes, 2 * block_bytes, bar);
        } else {
#pragma unroll
          for (int i = 0; i < PB; ++i)
            if (at[i] != kNone)
              bulk_g2s(dst + i * block_bytes, c.pages + (uint64_t)at[i] * block_bytes, block_bytes, bar);
        }
      }
    }
    if (++pro_stage == stages) pro_stage = 0;
  };
  // q rows of one column group as they lie: all warps the same one (NT = 1), or warp w group w
  constexpr int kRaw = KW * (F32 ? 2 : 1);
  const int my_nt = NT == 1 ? 0 : warp;
  uint4 raw[kRaw];
  auto load_q = [&](const Cursor& s) {
    const int r = s.rt * RT + my_nt * 8 + g;
    const bool live = my_nt < NT && r < s.qlen * G;
    const int tok = live ? r / G : 0, head = live ? r - tok * G : 0;
    const int64_t at = (int64_t)(s.q0 + tok) * a.q_stride + ((int64_t)s.kvh * G + head) * D + 8 * t;
#pragma unroll
    for (int i = 0; i < kRaw; ++i) {
      raw[i] = make_uint4(0, 0, 0, 0);
      if (live) {
        if constexpr (F32)
          raw[i] = *reinterpret_cast<const uint4*>(static_cast<const float*>(a.q) + at + 32 * (i / 2) + 4 * (i % 2));
        else
          raw[i] = *reinterpret_cast<const uint4*>(static_cast<const __half*>(a.q) + at + 32 * i);
      }
    }
  };
  load_q(cur);
  __syncwarp();
  fetch();
  for (int i = 0; i < stages; ++i) produce();

  // ---- the consumer side ----
  int stage = 0;
  uint32_t parity = 0;
  bool gave_up = false;
  int64_t left = u1 - u0 + skipped;
  if (tid == 0) pieces[blockIdx.x].first = -1;
  left -= kPieceCost;
  while (left > 0) {
    const bool from_start = cur.tile == cur.t0;
    const int row0 = cur.rt * RT, rows = cur.qlen * G;
    constexpr bool kQreg = NT == 1;  // one column group: its fragments stay in registers, no CTA barrier
    uint2 qreg[kQreg ? D / 16 : 1];
    float cf[NT][2];
    constexpr bool kQsReg = NG * NT <= 2 || NT == 1;
    float2 qsreg[kQsReg ? NG * NT : 1];
    if (my_nt < NT) {
      float q[KW][8], top = 0.0f;
#pragma unroll
      for (int i = 0; i < KW; ++i) {
        if constexpr (F32) {
          const uint4 v0 = raw[2 * i], v1 = raw[2 * i + 1];
          const uint32_t u[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
          for (int j = 0; j < 8; ++j) q[i][j] = __uint_as_float(u[j]);
        } else {
          const uint32_t u[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f = unpack_half2(u[j]);
            q[i][2 * j] = f.x, q[i][2 * j + 1] = f.y;
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(q[i][j]));
      }
      top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
      top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
      // rows are scaled by a power of two to [2^13, 2^14): the parts of q and its division by 16
      // then stay inside fp16
      const int ex = (int)(__float_as_uint(top) >> 23) - 127;  // subnormal rows count as 2^-127
      const int e = top < INFINITY && top > 0.0f ? max(ex, -110) - 13 : 0;
      const float down = __uint_as_float((uint32_t)(127 - e) << 23);
      float acc = 0.0f;
#pragma unroll
      for (int i = 0; i < KW; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          q[i][j] *= down;
          acc += q[i][j];
        }
        if ((i + 1) % GR == 0) {
          acc += __shfl_xor_sync(kFull, acc, 1);
          acc += __shfl_xor_sync(kFull, acc, 2);
          if (!F32) acc *= 5.9604644775390625e-8f;  // 2^-24, as the codes
          if constexpr (NT == 1)
            qsreg[i / GR] = make_float2(__shfl_sync(kFull, acc, 8 * t), __shfl_sync(kFull, acc, 8 * t + 4));
          else if (t == 0)
            qsf[(i / GR * NT + my_nt) * 8 + g] = acc;
          acc = 0.0f;
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const float x0 = q[i][2 * s], x1 = q[i][2 * s + 4];
          const float y0 = q[i][2 * s + 1] * (F32 ? 1.0f : 0.0625f), y1 = q[i][2 * s + 5] * (F32 ? 1.0f : 0.0625f);
          const uint2 hi = make_uint2(pack_half2(x0, x1), pack_half2(y0, y1));
          if constexpr (kQreg) qreg[2 * i + s] = hi;
          else qf[((2 * i + s) * NT + my_nt) * 32 + lane] = hi;
          if constexpr (F32) {  // NT = 1: every warp writes, and reads, the same values
            const float2 hx = unpack_half2(hi.x), hy = unpack_half2(hi.y);
            qf[((D / 16 + 2 * i + s) * NT + my_nt) * 32 + lane] =
                make_uint2(pack_half2(x0 - hx.x, x1 - hx.y), pack_half2(y0 - hy.x, y1 - hy.y));
          }
        }
      }
      const float fac = scalbnf(a.scale * kLog2e, F32 ? e : e + 24);
      if constexpr (NT == 1)
        cf[0][0] = __shfl_sync(kFull, fac, 8 * t), cf[0][1] = __shfl_sync(kFull, fac, 8 * t + 4);
      else if (t == 0)
        colf[my_nt * 8 + g] = fac;
    }
    if constexpr (NT == 1) {
      __syncwarp();
    } else {
      __syncthreads();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) cf[nt][j] = colf[nt * 8 + 2 * t + j];
      if constexpr (kQsReg) {
#pragma unroll
        for (int i = 0; i < NG * NT; ++i) qsreg[i] = *reinterpret_cast<const float2*>(&qsf[i * 8 + 2 * t]);
      }
    }

    // keys in [all_lo, all_hi) are seen by every row of the tile
    const int pos_a = cur.n - cur.qlen + row0 / G, pos_z = cur.n - cur.qlen + (row0 + RT - 1) / G;
    const int all_hi = a.causal ? min(cur.n, pos_a + 1) : cur.n;
    const int all_lo = a.window > 0 ? pos_z - a.window + 1 : 0;
    auto sees = [&](int key, int col) {
      const int pos = cur.n - cur.qlen + (row0 + col) / G;
      return key < cur.n && (!a.causal || key <= pos) && (a.window <= 0 || key > pos - a.window);
    };
    float m[NT][2], l[NT][2], o[D / 16][NT][4], oo[NG][NT][2];
    // fp16: V scales are held times vmul, o times vmul too
    float vmul = 1.0f, vinv = 1.0f;
    uint32_t vlim = F32 ? 0x7bff7bffu : 0x7bff0000u;  // fp16 pair: V scales stay up to this (offsets, and all of fp32's: any finite)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        m[nt][j] = -FLT_MAX, l[nt][j] = gave_up ? NAN : 0.0f;
#pragma unroll
        for (int gi = 0; gi < NG; ++gi) oo[gi][nt][j] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][nt][j] = 0.0f;
    }

    const int here = (int)min(left, (int64_t)(cur.t1 - cur.tile));
    const int tile_end = cur.tile + here;
    for (int base = cur.tile * kTile + warp * (16 * PB); base < min(tile_end * kTile, cur.n); base += kTile) {
      if (!__all_sync(kFull, gave_up || mbar_wait_bounded(&full[stage], parity))) {
        // give up: no more copies, a last bounded wait for those in flight, NaN results
        if (lane == 0) report_status(status, kStatusFullWait);
        gave_up = true;
        pro_left = 0, next_n = 0, issued = batch_n;
        int st = stage;
        uint32_t ph = parity;
        do {
          if (!__all_sync(kFull, mbar_wait_bounded(&full[st], ph))) break;
          if (++st == stages) st = 0, ph ^= 1u;
        } while (st != pro_stage);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) l[nt][0] = l[nt][1] = NAN;
      }
      const int have = flags[stage];
      if (have && !gave_up) {
        const uint32_t at = smem_u32(ring + stage * stage_bytes);
        // ---- scores, in units of 1 / cf ----
        float s[PB][NT][4];
        uint32_t kw[PB][2][KW];
#pragma unroll
        for (int p = 0; p < PB; ++p)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int r = g + 8 * h;
            if constexpr (D == 64) {
              const uint2 v = lds_u64_a(at + p * block_bytes + r * 32 + t * 8);
              kw[p][h][0] = v.x, kw[p][h][1] = v.y;
            } else {
#pragma unroll
              for (int k = 0; k < KW / 4; ++k) {
                const uint4 v = lds128_a(at + p * block_bytes + k_word_byte<D>(r, t, 4 * k));
                kw[p][h][4 * k] = v.x, kw[p][h][4 * k + 1] = v.y, kw[p][h][4 * k + 2] = v.z, kw[p][h][4 * k + 3] = v.w;
              }
            }
          }
        {
          // fp32: a scale after every 32 elements and the low parts first, as the tensor cores cut sums off at
          // fp32 and every further step would add an error of one last place of the running sum
          constexpr int SG = F32 ? 1 : GR;
#pragma unroll
          for (int gi = 0; gi < KW / SG; ++gi) {
            float acc[PB][NT][4];
#pragma unroll
            for (int i = gi * SG; i < (gi + 1) * SG; ++i) {
#pragma unroll
              for (int part = F32 ? 1 : 0; part >= 0; --part)
#pragma unroll
                for (int st = 0; st < 2; ++st)
#pragma unroll
                  for (int p = 0; p < PB; ++p) {
                    const uint32_t x = kw[p][0][i] >> (8 * st), y = kw[p][1][i] >> (8 * st);
                    const uint32_t a0 = F32 ? c_lower(x) : x & 0x000f000fu, a2 = F32 ? c_upper(x) : x & 0x00f000f0u;
                    const uint32_t a1 = F32 ? c_lower(y) : y & 0x000f000fu, a3 = F32 ? c_upper(y) : y & 0x00f000f0u;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                      uint2 b;
                      if (kQreg && part == 0) b = qreg[kQreg ? 2 * i + st : 0];
                      else b = qf[((part * (D / 16) + 2 * i + st) * NT + nt) * 32 + lane];
                      if (i == gi * SG && st == 0 && part == (F32 ? 1 : 0))
                        mma16816_zero(acc[p][nt], a0, a1, a2, a3, b.x, b.y);
                      else
                        mma16816(acc[p][nt], a0, a1, a2, a3, b.x, b.y);
                    }
                  }
            }
            const int grp = gi * SG / GR;
#pragma unroll
            for (int p = 0; p < PB; ++p) {
              const uint32_t kpar = at + p * block_bytes + 16 * D + g * 4 + grp * 64;  // rows g; g + 8 is 32 bytes on
              const float2 p0 = unpack_half2(lds_u32_a(kpar)), p1 = unpack_half2(lds_u32_a(kpar + 32));
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float* sp = s[p][nt];
                if (gi * SG % GR == 0) {
                  const float z0 = F32 ? fmaf(8.0f, p0.x, p0.y) : p0.y, z1 = F32 ? fmaf(8.0f, p1.x, p1.y) : p1.y;
                  float2 qs;
                  if constexpr (kQsReg) qs = qsreg[grp * NT + nt];
                  else qs = *reinterpret_cast<const float2*>(&qsf[(grp * NT + nt) * 8 + 2 * t]);
                  if (gi == 0) {
                    sp[0] = z0 * qs.x, sp[1] = z0 * qs.y;
                    sp[2] = z1 * qs.x, sp[3] = z1 * qs.y;
                  } else {
                    sp[0] = fmaf(z0, qs.x, sp[0]), sp[1] = fmaf(z0, qs.y, sp[1]);
                    sp[2] = fmaf(z1, qs.x, sp[2]), sp[3] = fmaf(z1, qs.y, sp[3]);
                  }
                }
                sp[0] = fmaf(acc[p][nt][0], p0.x, sp[0]), sp[1] = fmaf(acc[p][nt][1], p0.x, sp[1]);
                sp[2] = fmaf(acc[p][nt][2], p1.x, sp[2]), sp[3] = fmaf(acc[p][nt][3], p1.x, sp[3]);
              }
            }
          }
        }
        const bool masked = base < all_lo || base + 16 * PB > all_hi || have != (1 << PB) - 1;
        uint32_t vp[PB][NG][2];  // V parameters of rows g, g + 8
#pragma unroll
        for (int p = 0; p < PB; ++p) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[p][nt][j] *= cf[nt][j & 1];
#pragma unroll
          for (int gi = 0; gi < NG; ++gi)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              vp[p][gi][h] = lds_u32_a(at + p * block_bytes + 16 * D + NG * 64 + gi * 64 + h * 32 + g * 4);
        }
        if (masked) {
#pragma unroll
          for (int p = 0; p < PB; ++p) {
            const int key = base + 16 * p + g;
            const bool read = (have >> p & 1) != 0;
            bool own[2] = {false, false};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                if (read && sees(key + (j >> 1) * 8, nt * 8 + 2 * t + (j & 1))) own[j >> 1] = true;
                else s[p][nt][j] = -INFINITY;
              }
            // keys past the end hold anything, and those that no row sees have no part in the powers; four lanes have a key's rows
#pragma unroll
            for (int h = 0; h < 2; ++h)
              if (!(__ballot_sync(kFull, own[h]) >> (lane & ~3) & 15u))
#pragma unroll
                for (int gi = 0; gi < NG; ++gi) vp[p][gi][h] = 0u;
          }
        }
        // ---- references: rise when a score passes its row's, or a V scale its limit ----
        uint32_t vtop = 0;  // fp16 pair of largest magnitudes, NaN if there is one
#pragma unroll
        for (int p = 0; p < PB; ++p)
#pragma unroll
          for (int gi = 0; gi < NG; ++gi)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t v = vp[p][gi][h] & 0x7fff7fffu;
              if (p == 0 && gi == 0 && h == 0) vtop = v;
              else asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(vtop) : "r"(vtop), "r"(v));
            }
        bool rise = !__hble2(*reinterpret_cast<const __half2*>(&vtop), *reinterpret_cast<const __half2*>(&vlim));
        float tops[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            tops[nt][j] = fmaxf(s[0][nt][j], s[0][nt][j + 2]);
            if constexpr (PB == 2) tops[nt][j] = fmaxf(tops[nt][j], fmaxf(s[PB - 1][nt][j], s[PB - 1][nt][j + 2]));
            rise |= tops[nt][j] > m[nt][j] + kRise;
          }
        if (__any_sync(kFull, rise)) {
          // inf or NaN among the V parameters: rows that see such a key get NaN in its group, the others
          // go on without the key's value (0 * NaN would reach them in the products)
          const bool odd = (vtop & 0x7c00u) == 0x7c00u || (vtop & 0x7c000000u) == 0x7c000000u;
          if (__any_sync(kFull, odd)) {
            vtop = 0;
#pragma unroll
            for (int p = 0; p < PB; ++p)
#pragma unroll
              for (int gi = 0; gi < NG; ++gi)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const uint32_t v = vp[p][gi][h];
                  if ((v & 0x7c00u) == 0x7c00u || (v & 0x7c000000u) == 0x7c000000u) {
                    vp[p][gi][h] = 0u;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                      for (int j = 0; j < 2; ++j)
                        if (sees(base + 16 * p + g + 8 * h, nt * 8 + 2 * t + j)) oo[gi][nt][j] = NAN;
                  } else {
                    vtop = __vmaxu2(vtop, v & 0x7fff7fffu);
                  }
                }
          }
          float grow = 1.0f;
          if constexpr (!F32) {
            const uint32_t need = __reduce_max_sync(kFull, vtop & 0xffffu);
            if (need > (vlim & 0xffffu)) {
              const int ex = half_exponent(need);
              const float mul = pow2f(-ex);  // scales up to vlim = 2^(ex + 1) become at most 2
              grow = vinv * mul;
              vmul = mul;
              vinv = pow2f(ex);
              const __half lim = __float2half_rn(fminf(pow2f(ex + 1), 65504.0f));
              vlim = (uint32_t)__half_as_ushort(lim) | 0x7bff0000u;
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float top = tops[nt][j];
#pragma unroll
              for (int sh = 4; sh < 32; sh <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, sh));
              top = top > m[nt][j] + kRise ? top - kLift : m[nt][j];  // a row's arithmetic hangs on its own scores alone
              const float al = ex2(m[nt][j] - top);
              m[nt][j] = top;
              l[nt][j] *= al;
#pragma unroll
              for (int gi = 0; gi < NG; ++gi) oo[gi][nt][j] *= al;
              const float ag = al * grow;
#pragma unroll
              for (int i = 0; i < D / 16; ++i) o[i][nt][j] *= ag, o[i][nt][j + 2] *= ag;
            }
        }
        // ---- probabilities ----
#pragma unroll
        for (int p = 0; p < PB; ++p)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              s[p][nt][j] = ex2(s[p][nt][j] - m[nt][j & 1]);
              l[nt][j & 1] += s[p][nt][j];
            }
        // ---- sum_j p_j scale_j (c_j - 8), and sum_j p_j (offset + 8 scale) per lane ----
#pragma unroll
        for (int p = 0; p < PB; ++p) {
          uint32_t vw[4][VW];  // words of keys 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int r = 2 * t + 8 * h;
            const uint32_t vat = at + p * block_bytes + 8 * D;
            if constexpr (D == 64) {
              const uint2 v = lds_u64_a(vat + v_word_byte<D>(g, r, 0));
              vw[2 * h][0] = v.x, vw[2 * h + 1][0] = v.y;
            } else if constexpr (D == 128) {
              const uint4 v = lds128_a(vat + v_word_byte<D>(g, r, 0));
              vw[2 * h][0] = v.x, vw[2 * h][1] = v.y, vw[2 * h + 1][0] = v.z, vw[2 * h + 1][1] = v.w;
            } else {
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const uint4 v = lds128_a(vat + v_word_byte<D>(g, r + k, 0));
                vw[2 * h + k][0] = v.x, vw[2 * h + k][1] = v.y, vw[2 * h + k][2] = v.z, vw[2 * h + k][3] = v.w;
              }
            }
          }
          uint32_t bh[NT][2], bl[F32 ? NT : 1][2];
          float back = 1.0f;  // fp32: undoes the group's power
#pragma unroll
          for (int i = 0; i < KW; ++i) {  // granule of 32 elements: word i / 2, half i % 2
            if (i % GR == 0) {
              const int gi = i / GR;
              const float2 p0 = unpack_half2(vp[p][gi][0]), p1 = unpack_half2(vp[p][gi][1]);
              const float x0 = fmaf(p0.x, 8.0f, p0.y), x1 = fmaf(p1.x, 8.0f, p1.y);
              float mul = vmul;
              if constexpr (F32) {
                const uint32_t need = __reduce_max_sync(kFull, max(vp[p][gi][0] & 0x7fffu, vp[p][gi][1] & 0x7fffu));
                const int ex = half_exponent(need);
                mul = pow2f(-ex), back = pow2f(ex);
              }
              const float f0 = p0.x * mul, f1 = p1.x * mul;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                const float* sp = s[p][nt];
                oo[gi][nt][0] = fmaf(sp[0], x0, fmaf(sp[2], x1, oo[gi][nt][0]));
                oo[gi][nt][1] = fmaf(sp[1], x0, fmaf(sp[3], x1, oo[gi][nt][1]));
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const float f = h ? f1 : f0;
                  const float x = sp[2 * h] * f, y = sp[2 * h + 1] * f;
                  const uint32_t u = pack_half2(x, y);
                  bh[nt][h] = movmatrix(u);
                  if constexpr (F32) {
                    const float2 w = unpack_half2(u);
                    bl[nt][h] = movmatrix(pack_half2(x - w.x, y - w.y));
                  }
                }
              }
            }
            const uint32_t sel = i % 2 ? 0x7632u : 0x5410u;
            uint32_t x = __byte_perm(vw[0][i / 2], vw[1][i / 2], sel), y = __byte_perm(vw[2][i / 2], vw[3][i / 2], sel);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t a0 = c_lower(x), a1 = c_upper(x), a2 = c_lower(y), a3 = c_upper(y);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                if constexpr (F32) {  // added outside the tensor cores, with rounding
                  float acc[4];
                  mma16816_zero(acc, a0, a1, a2, a3, bl[nt][0], bl[nt][1]);
                  mma16816(acc, a0, a1, a2, a3, bh[nt][0], bh[nt][1]);
#pragma unroll
                  for (int k = 0; k < 4; ++k) o[2 * i + j][nt][k] = fmaf(acc[k], back, o[2 * i + j][nt][k]);
                } else {
                  mma16816(o[2 * i + j][nt], a0, a1, a2, a3, bh[nt][0], bh[nt][1]);
                }
              }
              x >>= 8, y >>= 8;
            }
          }
        }
      }
      __syncwarp();
      if (++stage == stages) stage = 0, parity ^= 1u;
      produce();
    }

    left -= here;
    // ---- the end of this piece: join the four warps ----
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) {
          l[nt][j] += __shfl_xor_sync(kFull, l[nt][j], sh);
#pragma unroll
          for (int gi = 0; gi < NG; ++gi) oo[gi][nt][j] += __shfl_xor_sync(kFull, oo[gi][nt][j], sh);
        }
        if (g == 0) ml[warp * RT + nt * 8 + 2 * t + j] = make_float2(m[nt][j], l[nt][j]);
      }
    __syncthreads();
    const bool ends = tile_end == cur.t1;
    const bool whole = from_start && ends;
    float* slot = slots + ((int64_t)blockIdx.x * 2 + (from_start ? 1 : 0)) * kSlot;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float fac[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float top = -FLT_MAX;
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[w * RT + nt * 8 + 2 * t + j].x);
        fac[j] = ex2(m[nt][j] - top);
      }
#pragma unroll
      for (int w64 = 0; w64 < VW; ++w64) {
#pragma unroll
        for (int i = 4 * w64; i < 4 * w64 + 4; ++i) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float base_sum = oo[i / 2 / GR][nt][j];
            const int d = (i % 4 / 2) * 32 + 4 * g + (i % 2) * 2;  // within the 64 elements
            const int col = 2 * t + j;
            float2 v;
            v.x = fmaf(o[i][nt][j], vinv, base_sum) * fac[j];
            v.y = fmaf(o[i][nt][j + 2], vinv, base_sum) * fac[j];
            *reinterpret_cast<float2*>(&exch[(warp * 8 + col) * 64 + d]) = v;
          }
        }
        __syncthreads();
        // 128 threads: column tid / 16, four elements each
        const int col = tid / 16, d4 = tid % 16 * 4;
        float4 sum = make_float4(0, 0, 0, 0);
        float top = -FLT_MAX, den = 0.0f;
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[w * RT + nt * 8 + col].x);
        for (int w = 0; w < kWarps; ++w) {
          const float2 x = ml[w * RT + nt * 8 + col];
          den = fmaf(x.y, ex2(x.x - top), den);
          const float4 v = *reinterpret_cast<const float4*>(&exch[(w * 8 + col) * 64 + d4]);
          sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
        }
        const int r = row0 + nt * 8 + col;
        if (r < rows) {
          if (whole) {
            const bool none = den == 0.0f;
            const float inv = none ? 0.0f : 1.0f / den;
            const int64_t row = (int64_t)(cur.q0 + r / G) * a.q_heads + (int64_t)cur.kvh * G + r % G;
            const int64_t at = row * D + 64 * w64 + d4;
            sum.x *= inv, sum.y *= inv, sum.z *= inv, sum.w *= inv;
            if (none) sum = make_float4(0, 0, 0, 0);
            if constexpr (F32)
              *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = sum;
            else
              *reinterpret_cast<uint2*>(static_cast<__half*>(a.out) + at) =
                  make_uint2(pack_half2(sum.x, sum.y), pack_half2(sum.z, sum.w));
            if (a.lse && w64 == 0 && tid % 16 == 0)
              a.lse[row] = none ? -INFINITY : (top + log2f(den)) * 0.6931471805599453f;
          } else {
            *reinterpret_cast<float4*>(slot + (nt * 8 + col) * D + 64 * w64 + d4) = sum;
            if (w64 == 0 && tid % 16 == 0)
              *reinterpret_cast<float2*>(slot + RT * D + (nt * 8 + col) * 2) = make_float2(top, den);
          }
        }
        __syncthreads();
      }
    }
    if (!from_start && ends && tid == 0) {
      // the CTA that holds the sequence's first unit
      const int64_t s0 = u1 - left - here - (cur.tile - cur.t0);
      pieces[blockIdx.x] = {(int)cut.part_of(s0), cur.q0, row0, rows, cur.kvh};
    }
    if (left <= kPieceCost) break;
    left -= kPieceCost;
    walk.next_part(cur);
    load_q(cur);
  }
}

template <int D, int NG, int NT, bool F32>
cudaError_t launch_stream(LaunchCtx& ctx, const Kv4Cache& c, const Kv4Attention& a) {
  constexpr int per_sm = stream_ctas<D, NT, F32>();
  constexpr int PB = step_blocks<D, NT>();
  using L = Layout<D, NG, NT, PB, F32>;
  constexpr int smem = L::kFixed + kWarps * L::stages(227 * 1024 / per_sm - 1024) * PB * L::kBlock;
  static_assert((smem + 1024) * per_sm <= 228 * 1024, "the SM holds so many CTAs (each with 1 KB of the system's)");
  auto kern = kv4_stream_kernel<D, NG, NT, F32>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(kern, smem, ctx.device, done);
  if (e != cudaSuccess) return e;
  const int grid = per_sm * (ctx.num_sms < 160 ? ctx.num_sms : 160);
  // n / ppb = n * magic >> 36 for n < 2^26 (2^30 tokens), ppb <= 256: n * ppb < 2^36
  const uint64_t ppb = (uint64_t)(c.page_size / 16), magic = ((1ull << 36) + ppb - 1) / ppb;
  e = launch_kernel(ctx, kern, dim3(grid), dim3(kWarps * 32), smem, c, a, magic, ctx.status);
  if (e != cudaSuccess) return e;
  const bool pdl = ctx.pdl;
  ctx.pdl = true;  // the joining kernel waits for the streaming kernel on the device
  e = launch_kernel(ctx, kv4_join_kernel<D, NT, F32>, dim3(ctx.num_sms), dim3(kJoinWarps * 32), 0, c, a, grid);
  ctx.pdl = pdl;
  return e;
}

template <int D, bool F32>
cudaError_t launch_stream_d(LaunchCtx& ctx, const Kv4Cache& c, const Kv4Attention& a, int nt) {
  auto go = [&](auto ng) -> cudaError_t {
    constexpr int NG = decltype(ng)::value;
    return nt == 1 ? launch_stream<D, NG, 1, F32>(ctx, c, a) : launch_stream<D, NG, 2, F32>(ctx, c, a);
  };
  if (c.group == 32) return go(std::integral_constant<int, D / 32>{});
  if (c.group == 64) return go(std::integral_constant<int, D / 64>{});
  if constexpr (D >= 128) return go(std::integral_constant<int, D / 128>{});
  return cudaErrorInvalidValue;
}

}  // namespace kv4

// One translation unit for each head size and activation type.
#define MNB_KV4_STREAM(name) cudaError_t launch_kv4_stream_##name(LaunchCtx& ctx, const Kv4Cache& c, const Kv4Attention& a, int nt)
MNB_KV4_STREAM(d64_f16);
MNB_KV4_STREAM(d64_f32);
MNB_KV4_STREAM(d128_f16);
MNB_KV4_STREAM(d128_f32);
MNB_KV4_STREAM(d256_f16);
MNB_KV4_STREAM(d256_f32);

}  // namespace mnb
