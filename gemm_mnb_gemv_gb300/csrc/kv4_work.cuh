// Work lists of the key/value cache's attention kernels: cutting sequences into equal ranges of key
// tiles, one for each CTA, and joining the pieces.
#pragma once

#include <float.h>

#include "kv4.cuh"
#include "mnb_device.cuh"
#include "mnb_internal.h"

namespace mnb {
namespace kv4 {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLift = 8.0f;   // a row's reference is set this far below its largest score (log2)
constexpr float kRise = 14.0f;  // and moves when a score passes it by this much

// Largest number of CTAs a launch may have: the workspace's sizing.
constexpr int kMaxCtas = 160 * 4;

struct Piece {  // what the joining kernel needs of a cut sequence, written by the CTA of its last piece
  int first;    // CTA of the first piece, -1: this CTA ends no cut sequence
  int q0, row0, rows, kvh;
};

// a / b for a, b >= 0: 32 bits where they are enough (a 64-bit division is a subroutine).
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// `total` units over `parts` CTAs: each gets `each` or, the first `extra` of them, one more.
struct Cut {
  int64_t each, extra;
  Cut() = default;
  __device__ __forceinline__ Cut(int64_t total, int64_t parts) {
    each = quotient(total, parts);
    extra = total - each * parts;
  }
  __device__ __forceinline__ int64_t start(int64_t part) const { return part * each + min(part, extra); }
  __device__ __forceinline__ int64_t part_of(int64_t unit) const {
    const int64_t head = extra * (each + 1);
    return unit < head ? quotient(unit, each + 1) : extra + quotient(unit - head, each);
  }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_half2(uint32_t u) {
  return __half22float2(*reinterpret_cast<const __half2*>(&u));
}

// One sequence's place in the work list.
struct Cursor {
  int b, rt, kvh, tile;
  int q0, qlen, n;    // query rows and keys of sequence b
  int R;              // row tiles of sequence b
  int lo, hi;         // keys that some row of row tile rt sees: 32 bits hold them (2^30 keys, 2^20 tokens, a window of 2^30)
  int t0, t1;         // their tiles
};

// kPieceCost: what starting and ending a piece of a sequence costs, in tiles; counted where the work is
// cut, so that a CTA with many short sequences gets fewer keys.
template <int RT, int kTile, int kPieceCost>
struct Walk {
  const Kv4Attention& a;
  const Kv4Cache& c;
  int G, capacity;

  __device__ __forceinline__ Walk(const Kv4Attention& a_, const Kv4Cache& c_)
      : a(a_), c(c_), G(a_.q_heads / c_.kv_heads), capacity(a_.table_stride * c_.page_size) {}
  __device__ __forceinline__ void load(Cursor& s) const {
    const int lo = min(max(a.q_start[s.b], 0), a.T), hi = min(max(a.q_start[s.b + 1], lo), a.T);
    s.q0 = lo;
    s.qlen = hi - lo;
    s.n = min(max(a.kv_len[s.b], 0), capacity);
    s.R = (int)(((int64_t)s.qlen * G + RT - 1) / RT);
  }
  // of row tile rt
  __device__ __forceinline__ void range(Cursor& s) const {
    const int first = s.rt * RT / G, last = min(s.qlen - 1, (s.rt * RT + RT - 1) / G);
    s.hi = a.causal ? max(0, min(s.n, s.n - s.qlen + last + 1)) : s.n;
    s.lo = a.window > 0 ? max(0, s.n - s.qlen + first - a.window + 1) : 0;
    s.t0 = s.lo / kTile;
    s.t1 = max(s.t0 + 1, (s.hi + kTile - 1) / kTile);  // a row tile without keys still has a unit: it writes zeros
  }
  __device__ __forceinline__ int64_t units(Cursor s) const {  // of sequence s.b, loaded
    int64_t u = 0;
    for (s.rt = 0; s.rt < s.R; ++s.rt) {
      range(s);
      u += s.t1 - s.t0 + kPieceCost;
    }
    return u * c.kv_heads;
  }
  __device__ __forceinline__ void next_part(Cursor& s) const {  // to the first tile of the next row tile or key head
    if (++s.kvh == c.kv_heads) {
      s.kvh = 0;
      if (++s.rt == s.R) {
        s.rt = 0;
        do {
          ++s.b;
          if (s.b >= a.batch) return;  // past the end: not used
          load(s);
        } while (s.R == 0);
      }
      range(s);
    }
    s.tile = s.t0;
  }
};

// A CTA's share of the work: units [u0, u1); `skipped` of the first piece's cost units are the CTA before's.
struct Range {
  int64_t u0, u1;
  int skipped;
  Cut cut;
};

// The whole CTA of at least 128 threads calls it; scan: 10 words of shared memory. False: no work. The first 128
// threads take the sequences in turn, 128 at a time.
template <int RT, int kTile, int kPieceCost>
__device__ __forceinline__ bool find_range(const Walk<RT, kTile, kPieceCost>& walk, uint32_t* status, int64_t* scan, Range& out,
                                           Cursor& cur) {
  constexpr int kScan = 128;
  const Kv4Attention& a = walk.a;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  cur = Cursor{};
  int64_t total = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kScan) {
    if (tid < kScan && b0 + tid < a.batch) {
      cur.b = b0 + tid;
      walk.load(cur);
      total += walk.units(cur);
      if (blockIdx.x == 0 && a.kv_len[cur.b] > walk.capacity) report_status(status, kStatusBadIndex);
    }
  }
  const int64_t mine = total;
  for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(kFull, total, o);
  if (lane == 0 && warp < 4) scan[warp] = total;
  __syncthreads();
  total = scan[0] + scan[1] + scan[2] + scan[3];
  __syncthreads();
  const int64_t ncta = min((int64_t)gridDim.x, total);
  if ((int64_t)blockIdx.x >= ncta) return false;
  out.cut = Cut(total, ncta);
  out.u0 = out.cut.start(blockIdx.x), out.u1 = out.cut.start(blockIdx.x + 1);
  // the sequence that holds unit u0, by prefix sums
  int64_t before = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kScan) {
    int64_t own = 0;
    if (a.batch <= kScan) {
      own = mine;
    } else if (tid < kScan && b0 + tid < a.batch) {
      cur.b = b0 + tid;
      walk.load(cur);
      own = walk.units(cur);
    }
    int64_t inc = own;
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(kFull, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31 && warp < 4) scan[warp] = inc;
    __syncthreads();
    int64_t base = before;
    for (int w = 0; w < min(warp, 4); ++w) base += scan[w];
    const int64_t hi = base + inc, lo = hi - own;
    if (tid < kScan && out.u0 >= lo && out.u0 < hi) {
      scan[4] = b0 + tid;
      scan[5] = out.u0 - lo;
      scan[6] = cur.q0, scan[7] = cur.qlen, scan[8] = cur.n, scan[9] = cur.R;
    }
    before += scan[0] + scan[1] + scan[2] + scan[3];
    __syncthreads();
    if (before > out.u0) break;
  }
  cur.b = (int)scan[4];
  int64_t off = scan[5];
  cur.q0 = (int)scan[6], cur.qlen = (int)scan[7], cur.n = (int)scan[8], cur.R = (int)scan[9];
  for (cur.rt = 0;; ++cur.rt) {
    walk.range(cur);
    const int64_t len = (int64_t)(cur.t1 - cur.t0 + kPieceCost) * walk.c.kv_heads;
    if (off < len) break;
    off -= len;
  }
  const int each = cur.t1 - cur.t0 + kPieceCost;
  cur.kvh = (int)quotient(off, each);
  const int rest = (int)(off - (int64_t)cur.kvh * each);
  cur.tile = cur.t0 + max(0, rest - kPieceCost);
  out.skipped = min(rest, kPieceCost);
  return true;
}

// Joins the pieces of cut sequences: o = sum_p e^(m_p - m) o_p / sum_p e^(m_p - m) l_p, in a fixed order. Each
// block lists the cut sequences from the CTAs' entries; teams of warps take their rows in turn, each warp its share of
// the pieces, several of them in flight. With few rows a team is four warps (many pieces each), with more rows than such
// teams it is one.
constexpr int kJoinWarps = 16, kRounds = (kMaxCtas + kJoinWarps * 32 - 1) / (kJoinWarps * 32);
template <int D, int NT, bool F32>
__global__ void __launch_bounds__(kJoinWarps * 32) kv4_join_kernel(const Kv4Cache c, const Kv4Attention a, int ctas) {
  constexpr int RT = 8 * NT, kSlot = RT * (D + 2), E = D / 32, kFlight = NT > 4 ? 4 : D > 128 ? 5 : 10;
  __shared__ float part[kJoinWarps][D + 4];  // o, then l and m
  __shared__ Piece list[kMaxCtas];
  __shared__ int list_last[kMaxCtas];  // the CTA that wrote the entry
  __shared__ int count[kRounds][kJoinWarps];
  pdl_wait();
  const Piece* pieces = reinterpret_cast<const Piece*>(a.workspace);
  const float* slots = reinterpret_cast<const float*>(static_cast<const uint8_t*>(a.workspace) + kMaxCtas * sizeof(Piece));
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  Piece own[kRounds];
#pragma unroll
  for (int k = 0; k < kRounds; ++k) {
    const int i = k * kJoinWarps * 32 + threadIdx.x;
    own[k].first = -1;
    if (i < ctas) own[k] = pieces[i];
  }
  uint32_t vote[kRounds];
#pragma unroll
  for (int k = 0; k < kRounds; ++k) {
    vote[k] = __ballot_sync(kFull, own[k].first >= 0);
    if (lane == 0) count[k][warp] = __popc(vote[k]);
  }
  __syncthreads();
  int n_list = 0;
#pragma unroll
  for (int k = 0; k < kRounds; ++k) {
    int at = n_list;
    for (int w = 0; w < kJoinWarps; ++w) {
      if (w < warp) at += count[k][w];
      n_list += count[k][w];
    }
    at += __popc(vote[k] & ((1u << lane) - 1));
    if (own[k].first >= 0) list[at] = own[k], list_last[at] = k * kJoinWarps * 32 + threadIdx.x;
  }
  __syncthreads();
  const int G = a.q_heads / c.kv_heads;
  const int items = n_list * RT;
  const int team = items > (int)gridDim.x * (kJoinWarps / 4) ? 1 : 4;
  const int teams = kJoinWarps / team, sub = warp % team;
  for (int item0 = blockIdx.x * teams; item0 < items; item0 += gridDim.x * teams) {
    const int item = item0 + warp / team;
    const int col = item % RT;
    int last = 0;
    Piece p = {};
    if (item < items) p = list[item / RT], last = list_last[item / RT];
    const bool live = item < items && p.row0 + col < p.rows;
    const int n = live ? last - p.first + 1 : 0;
    float m = -FLT_MAX, l = 0.0f, acc[E] = {};
    for (int i0 = sub; i0 < n; i0 += team * kFlight) {
      float2 ml[kFlight];
      float v[kFlight][E];
#pragma unroll
      for (int k = 0; k < kFlight; ++k) {
        const int i = i0 + k * team;
        ml[k] = make_float2(-FLT_MAX, 0.0f);
        if (i < n) {
          const float* s = slots + ((int64_t)(p.first + i) * 2 + (i == 0 ? 1 : 0)) * kSlot;
          ml[k] = *reinterpret_cast<const float2*>(s + RT * D + col * 2);
#pragma unroll
          for (int e = 0; e < E; e += 2)
            *reinterpret_cast<float2*>(&v[k][e]) = *reinterpret_cast<const float2*>(s + col * D + e * 32 + lane * 2);
        }
      }
      float top = m;
#pragma unroll
      for (int k = 0; k < kFlight; ++k) top = fmaxf(top, ml[k].x);
      const float al = ex2(m - top);
      m = top;
      l *= al;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] *= al;
#pragma unroll
      for (int k = 0; k < kFlight; ++k) {
        if (i0 + k * team < n) {
          const float f = ex2(ml[k].x - top);
          l = fmaf(ml[k].y, f, l);
#pragma unroll
          for (int e = 0; e < E; ++e) acc[e] = fmaf(v[k][e], f, acc[e]);
        }
      }
    }
#pragma unroll
    for (int e = 0; e < E; e += 2) *reinterpret_cast<float2*>(&part[warp][e * 32 + lane * 2]) = make_float2(acc[e], acc[e + 1]);
    if (lane == 0) part[warp][D] = l, part[warp][D + 1] = m;
    __syncthreads();
    if (live && sub == 0) {
      float top = part[warp][D + 1];
      for (int w = 1; w < team; ++w) top = fmaxf(top, part[warp + w][D + 1]);
      float den = 0.0f, f[4] = {};
#pragma unroll
      for (int w = 0; w < 4; ++w)
        if (w < team) {
          f[w] = ex2(part[warp + w][D + 1] - top);
          den = fmaf(part[warp + w][D], f[w], den);
        }
      const int r = p.row0 + col;
      const int64_t row = (int64_t)(p.q0 + r / G) * a.q_heads + (int64_t)p.kvh * G + r % G;
      const bool none = den == 0.0f;
      const float inv = none ? 0.0f : 1.0f / den;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const int d = e * 32 + lane * 2;
        float2 v = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < 4; ++w)
          if (w < team) v.x = fmaf(part[warp + w][d], f[w], v.x), v.y = fmaf(part[warp + w][d + 1], f[w], v.y);
        v.x *= inv, v.y *= inv;
        if (none) v = make_float2(0.0f, 0.0f);
        if constexpr (F32) *reinterpret_cast<float2*>(static_cast<float*>(a.out) + row * D + d) = v;
        else *reinterpret_cast<uint32_t*>(static_cast<__half*>(a.out) + row * D + d) = pack_half2(v.x, v.y);
      }
      if (a.lse && lane == 0) a.lse[row] = none ? -INFINITY : (top + log2f(den)) * 0.6931471805599453f;
    }
    __syncthreads();
  }
}

}  // namespace kv4
}  // namespace mnb
