// Attention of many query rows over the paged 4-bit key/value cache on the tcgen05 tensor cores
// (prefill, chunks of a prompt, long drafts): fp16 activations, heads of 64 and 128.
//
// A CTA (one per SM) takes row tiles of 2 x 128 rows (query token, head of the group) and key tiles of 128:
//   S = Q K^T (M 128, N 128 keys, Q and K in shared memory), P = 2^(c S - m) in fp16 back to tensor
//   memory over S, O += P V (P from tensor memory, V in shared memory).
// Roles in 512 threads:
//   warp 0       producer: per key tile eight 16-key blocks of the cache as they lie, by bulk copies;
//   warp 1       MMA issuer (one lane) and tensor memory (512 columns: S and O of both row tiles);
//   warps 4-7    dequantisers: codes -> fp16 offset + code * scale in the 128-byte-swizzled operand layouts,
//                one key a thread, K rows K-major and V rows N-major, into a ring of three buffers (K, V, K, ..);
//                both row tiles read a buffer, which halves the conversion per product;
//   warps 8-11, 12-15  softmax of row tile A, B: a row a thread, no shuffles.
// The issuer alternates S_A, P_B V, S_B, P_A V, so each softmax has the other tile's products to hide behind.
// Conversion: a code's byte is the 8-bit float (4 exponent bits) of c * 2^-9, two of which one instruction turns into fp16, exactly;
// with the scale times 2^9 one FMA gives offset + code * scale, rounded once. The scale has to stay below 2^7 then. K is
// held, a key tile at a time, at the power of two of its value that puts its largest just below 2^11: parts of 2^-24 of
// the largest still have all of fp16's bits, whether their rows see the largest or not. The power goes into the softmax's factor. V is
// held as it is (what mnb_kv4_read gives in fp16); a tile beyond 2^11 is held at the power that brings it there, which goes, as a
// difference to the largest tile so far, into P (2^-9 at the least, where P's last place is 2^-23 of its largest).
// Other ways: the nibbles as they lie, fp16 subnormals c * 2^-24, save two operations in eleven a word, but the scale times 2^24 stays
// inside fp16 only where a tile's largest is held below 2^-4, and parts of 2^-10 of it are subnormals then (chunk and prompts below
// 825 and 75.8 us in the same run in which this form took 845 and 76.3); codes as 1024 + c, less 1024: 852 and 78.0.
// A row's reference m moves as in the streaming kernel, and only then is O rescaled in tensor memory.
// A non-finite V value enters as 0 (0 * NaN would reach every row of the tile) and marks its piece: at the piece's
// end the rows look for such keys among those that they see, and get NaN in the groups.
// Element order: the nibbles of a word convert to elements n0, n2, n4, n6, n1, n3, n5, n7; q is permuted
// alike, and O's columns are put back when they are stored.
// Fewer bits: K, V and P are each rounded once to fp16, as the result is; the error (norm, against fp64) is 3.8e-4 to 4.5e-4,
// of which the result's own rounding is 2.1e-4. Keeping the codes exact would take a multiplication of each score and each
// probability by its key's scale, in the softmax, whose instructions the kernel has least to spare of.
// Measured, graph replays: 2048 tokens over 32768 keys, 32 / 8 heads of 128: 850 us, 1.25 PFLOP/s, 64% of the measured peak (an earlier
// conversion: 817; without it 704 us, without the softmax 685 us, without either 637 us). Two prompts of up to 2048: 77 us.
// Where the compiler places the roles' code alone moves the chunk by up to 10%.
// Work is cut and joined as in the streaming kernel (kv4_work.cuh), so a few rows over a long context
// use every SM too.
#include <type_traits>

#include "kv4_work.cuh"
#include "tcgen05.cuh"

namespace mnb {
namespace {

using namespace kv4;

constexpr int kRows = 256, kKeys = 128, kThreads = 512;
constexpr int kCost = 3;   // tiles that a piece's start and end cost: 2: 50 and 86 us (16 drafted tokens over 32768 keys; prompts), 3: 47 and 85 (now 43 and 77)
constexpr int kBufs = 3;   // K / V operand buffers
constexpr int kMeta = 4;   // tiles whose flags are kept
constexpr uint32_t kLate = 0xffffffffu;  // in a size's place: this warp's wait gave up

// The power of two e for a tile whose largest parameter has the fp16 bits `size` (of |offset|, 16 |scale|): size * 2^e is in
// [2^10, 2^11).
__device__ __forceinline__ int tile_power(uint32_t size) { return 25 - max((int)(size >> 10), 1); }

template <int D, int NG>
struct TileSmem {
  static constexpr int kBlock = 16 * D + 128 * NG;
  static constexpr int kRaw = 8 * kBlock;                // one key tile of the cache
  static constexpr int kOperand = kKeys * D * 2;         // K or V of a tile in fp16
  static constexpr int kQ = kRows * D * 2;
  static constexpr int kFree = 227 * 1024 - 2048 - kQ - kBufs * kOperand;
  static constexpr int kStages = kFree / kRaw < 4 ? kFree / kRaw : 4;
  static constexpr int kBytes = kQ + kBufs * kOperand + kStages * kRaw + 1024;
  static_assert(kStages >= 2, "two raw tiles in flight");
};

// max over 3 values
__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

// (x0, x1) = (x0, x1) * (c, c) + (d, d)
__device__ __forceinline__ void fma2(float& x0, float& x1, float c, float d) {
  asm("{\n\t.reg .b64 a, b, e;\n\t"
      "mov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %2};\n\tmov.b64 e, {%3, %3};\n\t"
      "fma.rn.f32x2 a, a, b, e;\n\t"
      "mov.b64 {%0, %1}, a;\n\t}"
      : "+f"(x0), "+f"(x1)
      : "f"(c), "f"(d));
}
__device__ __forceinline__ void add2(float& s0, float& s1, float x0, float x1) {
  asm("{\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\t"
      "add.rn.f32x2 a, a, b;\n\t"
      "mov.b64 {%0, %1}, a;\n\t}"
      : "+f"(s0), "+f"(s1)
      : "f"(x0), "f"(x1));
}

__device__ __forceinline__ uint32_t hfma2_bits(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// Scale and offset of a group, times 2^e, as pairs for convert().
struct Group {
  uint32_t scale, offset;
};
__device__ __forceinline__ Group group_of(uint32_t param, int e) {
  const float2 so = unpack_half2(param);
  const float f = pow2(e), s = so.x * f * 512.0f;
  return {pack_half2(s, s), pack_half2(so.y * f, so.y * f)};
}

// Bytes 0 and 1, and 2 and 3, of codes 0..15 to fp16 c * 2^-9.
__device__ __forceinline__ uint2 codes_to_half(uint32_t x) {
  uint2 r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(r.x), "=r"(r.y)
      : "r"(x));
  return r;
}

// A word's 8 codes to offset + code * scale, in the order n0, n2, n4, n6, n1, n3, n5, n7; n0..n3 are of group `a`, n4..n7 of `b`.
__device__ __forceinline__ uint4 convert(uint32_t w, const Group& a, const Group& b) {
  const uint2 even = codes_to_half(w & 0x0f0f0f0fu), odd = codes_to_half(w >> 4 & 0x0f0f0f0fu);
  return make_uint4(hfma2_bits(even.x, a.scale, a.offset), hfma2_bits(even.y, b.scale, b.offset),
                    hfma2_bits(odd.x, a.scale, a.offset), hfma2_bits(odd.y, b.scale, b.offset));
}
// Elements of q in the same order.
__device__ __forceinline__ uint4 in_code_order(uint4 v) {
  return make_uint4(__byte_perm(v.x, v.y, 0x5410), __byte_perm(v.z, v.w, 0x5410), __byte_perm(v.x, v.y, 0x7632),
                    __byte_perm(v.z, v.w, 0x7632));
}

__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

template <int D, int NG>
__global__ void __launch_bounds__(kThreads, 1)
    kv4_tile_kernel(const Kv4Cache c, const Kv4Attention a, uint64_t page_magic, uint32_t* status) {
  using L = TileSmem<D, NG>;
  constexpr int KW = D / 32, VW = D / 64;
  constexpr uint32_t kColS = 0, kColO = 256;  // tensor memory columns: S_A, S_B, O_A, O_B
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t raw_full[4], raw_empty[4], kv_full[kBufs], kv_empty[kBufs], q_full[2], s_full[2], p_full[2][2], o_full;
  __shared__ int64_t scan[10];
  __shared__ uint32_t tmem_base;
  __shared__ int raw_have[4];                 // blocks of a raw tile that were read
  __shared__ uint32_t tile_info[kMeta];       // for the softmax: bits 0-7 blocks read, 8-15 and 16-23 powers of K and V + 64
  __shared__ int odd_piece[kMeta];            // 1 + the last piece (modulo kMeta) with a V value that is not finite
  __shared__ uint2 sizes[2][4];               // fp16 bits of the largest K and V parameters, by dequantiser warp; kLate

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  const uint32_t q_at = smem_u32(smem), buf_at = q_at + L::kQ;
  uint8_t* raw_ring = smem + L::kQ + kBufs * L::kOperand;

  if (tid == 0) {
    for (int i = 0; i < kMeta; ++i) odd_piece[i] = 0;
    for (int i = 0; i < 4; ++i) mbar_init(&raw_full[i], 1), mbar_init(&raw_empty[i], 4);
    for (int i = 0; i < kBufs; ++i) mbar_init(&kv_full[i], 4), mbar_init(&kv_empty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&q_full[i], 4), mbar_init(&s_full[i], 1), mbar_init(&p_full[i][0], 4), mbar_init(&p_full[i][1], 4);
    mbar_init(&o_full, 1);
    fence_mbar_init();
  }
  pdl_launch_dependents();
  pdl_wait();

  const Walk<kRows, kKeys, kCost> walk(a, c);
  const int G = walk.G;
  Piece* pieces = reinterpret_cast<Piece*>(a.workspace);
  constexpr int kSlot = kRows * (D + 2);
  float* slots = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + kMaxCtas * sizeof(Piece));
  Range range;
  Cursor cur;
  if (!find_range(walk, status, scan, range, cur)) {
    if (tid == 0) pieces[blockIdx.x].first = -1;
    return;
  }
  if (warp == 1) {
    tc::tmem_alloc(&tmem_base, 512);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = tmem_base;
  // every role walks the same pieces
  int64_t left = range.u1 - range.u0 + range.skipped - kCost;
  auto next_piece = [&](int done) {  // false: that was the last
    left -= done;
    if (left <= kCost) return false;
    left -= kCost;
    walk.next_part(cur);
    return true;
  };
  // a role whose wait gave up says so and stops; the others run into their own limits, and rows get NaN
  auto give_up = [&](uint32_t what) { report_status(status, what); };

  const int wg = warp >> 2;
  if (wg == 0) {
    tc::setmaxnreg_dec<72>();
    if (warp == 0) {
      // ------------------------------ producer ------------------------------------
      const int ppb = c.page_blocks;
      int stage = 0;
      uint32_t phase = 0;
      int issued = 0;
      bool ok = true;
      while (left > 0 && ok) {
        const int here = (int)min(left, (int64_t)(cur.t1 - cur.tile));
        for (int tile = cur.tile; tile < cur.tile + here; ++tile) {
          // lane i < 8: block i of the tile
          const int key = tile * kKeys + (lane & 7) * 16;
          uint32_t at = 0xffffffffu;
          if (lane < 8 && key < cur.n) {
            const uint32_t blk = (uint32_t)key / 16;
            const uint32_t pi = (uint32_t)((uint64_t)blk * page_magic >> 36);
            const int page = a.page_table[(int64_t)cur.b * a.table_stride + pi];
            if (page >= 0 && page < c.num_pages)
              at = ((uint32_t)page * c.kv_heads + cur.kvh) * ppb + (blk - pi * ppb);
            else
              report_status(status, kStatusBadIndex);
          }
          const uint32_t have = __ballot_sync(kFull, at != 0xffffffffu);
          if (issued >= L::kStages && !__all_sync(kFull, mbar_wait_bounded(&raw_empty[stage], phase ^ 1u))) {
            if (lane == 0) give_up(kStatusEmptyWait);
            ok = false;
            break;
          }
          if (lane == 0) {
            raw_have[stage] = (int)have;
            if (have) mbar_arrive_expect_tx(&raw_full[stage], __popc(have) * L::kBlock);
            else mbar_arrive(&raw_full[stage]);
          }
          __syncwarp();
          if (at != 0xffffffffu)
            bulk_g2s(raw_ring + stage * L::kRaw + lane * L::kBlock, c.pages + (uint64_t)at * L::kBlock, L::kBlock,
                     &raw_full[stage]);
          ++issued;
          if (++stage == L::kStages) stage = 0, phase ^= 1u;
        }
        if (!next_piece(here)) break;
      }
      // every copy lands before the CTA can retire
      for (int i = max(0, issued - L::kStages); i < issued; ++i)
        (void)mbar_wait_bounded(&raw_full[i % L::kStages], (uint32_t)(i / L::kStages) & 1u);
    } else if (warp == 1) {
      // ------------------------------ MMA issuer ----------------------------------
      // The warp stays together and one elected lane issues: a product's descriptors are formed before its
      // first MMA, since the tensor pipe queues little and idles while addresses are made.
      const bool leader = tc::elect_one();
      const uint32_t idesc_s = tc::idesc_f16_f32(128, 128);
      const uint32_t idesc_o = tc::idesc_f16_f32(128, D) | tc::kIdescBMajorN;
      int item = 0;                       // K and V operands in order
      uint32_t kv_phase = 0, p_phase = 0, q_phase = 0;  // a bit for each barrier
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t ph) {
        if (__all_sync(kFull, mbar_wait_bounded(bar, ph))) return true;
        if (leader) give_up(kStatusMmaWait);
        ok = false;
        return false;
      };
      auto wait_kv = [&](int buf) {
        const bool r = wait(&kv_full[buf], kv_phase >> buf & 1u);
        kv_phase ^= 1u << buf;
        tc::fence_after_sync();
        return r;
      };
      const uint64_t dq0 = tc::smem_desc_k_sw128(q_at), dk0 = tc::smem_desc_k_sw128(buf_at);
      const uint64_t dv0 = tc::smem_desc_mn_sw128(buf_at, kKeys * 128);
      auto mma_s = [&](int x, int buf) {
        const uint64_t dq = dq0 + (uint32_t)(x * (L::kQ / 2) >> 4), dk = dk0 + (uint32_t)(buf * L::kOperand >> 4);
        const uint32_t d = tmem + kColS + x * 128;
        uint64_t qa[D / 16], ka[D / 16];
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t step = ((kk / 4) * (128 * 128) + (kk % 4) * 32) >> 4;
          qa[kk] = dq + step, ka[kk] = dk + step;
        }
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) tc::mma_f16(d, qa[kk], ka[kk], idesc_s, kk > 0);
          tc::mma_commit(&s_full[x]);
        }
        __syncwarp();
      };
      auto mma_o = [&](int x, int buf, bool first) {  // in the two halves in which P comes
        const uint64_t dv = dv0 + (uint32_t)(buf * L::kOperand >> 4);
        const uint32_t d = tmem + kColO + x * 128, p = tmem + kColS + x * 128;
        uint64_t va[kKeys / 16];
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk) va[kk] = dv + (uint32_t)(kk * 2048 >> 4);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (!wait(&p_full[x][half], p_phase >> x & 1u)) return false;
          tc::fence_after_sync();
          if (leader) {
#pragma unroll
            for (int kk = 4 * half; kk < 4 * half + 4; ++kk)
              tc::mma_f16_ts(d, p + kk * 8, va[kk], idesc_o, kk > 0 ? 1u : !first);
          }
          __syncwarp();
        }
        p_phase ^= 1u << x;
        return true;
      };
      auto commit = [&](uint64_t* bar) {
        if (leader) tc::mma_commit(bar);
        __syncwarp();
      };
      while (left > 0 && ok) {
        const int here = (int)min(left, (int64_t)(cur.t1 - cur.tile));
        if (!wait(&q_full[0], q_phase) || !wait(&q_full[1], q_phase)) break;
        q_phase ^= 1u;
        tc::fence_after_sync();
        int vbuf = 0;  // V of the tile before
        for (int j = 0; j < here; ++j) {
          const int kb = item % kBufs, vb = (item + 1) % kBufs;
          if (!wait_kv(kb)) break;
          mma_s(0, kb);
          if (j > 0) {
            if (!mma_o(1, vbuf, j == 1)) break;
            commit(&kv_empty[vbuf]);
          }
          mma_s(1, kb);
          commit(&kv_empty[kb]);
          if (!wait_kv(vb)) break;
          if (!mma_o(0, vb, j == 0)) break;
          vbuf = vb;
          item += 2;
        }
        if (!ok) break;
        if (!mma_o(1, vbuf, here == 1)) break;
        commit(&kv_empty[vbuf]);
        commit(&o_full);
        if (!next_piece(here)) break;
      }
      if (!ok) {
        // the tensor memory is given back only after the products in flight are done
        commit(&o_full);
        (void)mbar_wait_bounded(&o_full, 0);
        (void)mbar_wait_bounded(&o_full, 1);
      }
    }
  } else if (wg == 1) {
    tc::setmaxnreg_dec<104>();
    // ------------------------------ dequantisers -------------------------------------
    const int r = tid - 128;  // key of the tile
    const int row = r & 15;   // in its block
    int stage = 0, item = 0, tiles = 0, piece = 0;
    uint32_t phase = 0, e_phase = 0;  // e_phase: a bit for each buffer
    // A warp whose wait gave up is late: it does no more work but comes to the next tile's barrier, where all four see it and
    // stop together. Left alone, the others would wait there without a limit.
    bool ok = true, late = false;
    while (left > 0 && ok) {
      const int here = (int)min(left, (int64_t)(cur.t1 - cur.tile));
      for (int tile = cur.tile; tile < cur.tile + here; ++tile) {
        if (!late) late = !__all_sync(kFull, mbar_wait_bounded(&raw_full[stage], phase));
        const int have = raw_have[stage];
        const uint32_t blk = smem_u32(raw_ring + stage * L::kRaw + (r >> 4) * L::kBlock);
        const uint32_t par = blk + 16 * D + row * 4;
        // ---- parameters, zeros for keys that are not there or that no row sees; the four warps agree on the tile's powers ----
        uint32_t kpar[NG], vpar[NG], bad = 0, ksize = 0, vsize = 0;  // sizes: the larger of |offset| and 16 |scale|
        const bool there = tile * kKeys + r >= cur.lo && tile * kKeys + r < cur.hi && (have >> (r >> 4) & 1);
        auto finite = [](uint32_t p) { return (p & 0x7c00u) != 0x7c00u && (p & 0x7c000000u) != 0x7c000000u; };
#pragma unroll
        for (int gi = 0; gi < NG; ++gi) {
          kpar[gi] = there ? lds_u32_a(par + gi * 64) : 0u;
          vpar[gi] = there ? lds_u32_a(par + (NG + gi) * 64) : 0u;
          if (!finite(vpar[gi])) bad = 1u, vpar[gi] = 0u;
          if (finite(kpar[gi])) ksize = max(ksize, max((kpar[gi] & 0x7fffu) + 0x1000u, kpar[gi] >> 16 & 0x7fffu));
          vsize = max(vsize, max((vpar[gi] & 0x7fffu) + 0x1000u, vpar[gi] >> 16 & 0x7fffu));
        }
        ksize = __reduce_max_sync(kFull, ksize);
        vsize = __reduce_max_sync(kFull, vsize);
        if (lane == 0) sizes[tiles & 1][warp - 4] = make_uint2(late ? kLate : ksize, vsize);
        if (bad) odd_piece[piece % kMeta] = piece + 1;
        asm volatile("bar.sync 1, 128;" ::: "memory");
        for (int w = 0; w < 4; ++w) ksize = max(ksize, sizes[tiles & 1][w].x), vsize = max(vsize, sizes[tiles & 1][w].y);
        if (ksize == kLate) {
          ok = false;
          break;
        }
        const int ke = tile_power(ksize), ve = min(tile_power(vsize), 0);
        if (r == 0) tile_info[tiles % kMeta] = (uint32_t)have | (uint32_t)(ke + 64) << 8 | (uint32_t)(ve + 64) << 16;
        // ---- K ----
        int buf = item % kBufs;
        if (item >= kBufs) {
          if (!late) late = !__all_sync(kFull, mbar_wait_bounded(&kv_empty[buf], e_phase >> buf & 1u));
          e_phase ^= 1u << buf;
        }
        if (!late) {
          Group gr[NG];
#pragma unroll
          for (int gi = 0; gi < NG; ++gi) gr[gi] = group_of(kpar[gi], ke);
          const uint32_t dst = buf_at + buf * L::kOperand + r * 128 + ((r & 7) << 4);  // chunk c: dst ^ c << 4 (swizzled)
          // 16 bytes: words p = 4 ch .. of the row, word (t, w) = p / KW, p % KW; the starting chunk follows the
          // lane, so that eight rows are read from distinct banks. All loads come before the first store.
          uint4 v4[KW];
#pragma unroll
          for (int j = 0; j < KW; ++j) v4[j] = lds128_a(blk + row * (D / 2) + ((j + (lane >> 1)) & (KW - 1)) * 16);
#pragma unroll
          for (int j = 0; j < KW; ++j) {
            const int ch = (j + (lane >> 1)) & (KW - 1);
            const uint32_t w4[4] = {v4[j].x, v4[j].y, v4[j].z, v4[j].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int t = KW == 4 ? ch : ch * 2 + i / 2, w = KW == 4 ? i : i % 2;
              const int chunk = 4 * w + t;  // 16-byte chunk of the row
              sts128((dst ^ ((chunk & 7) << 4)) + (chunk >> 3) * (kKeys * 128), convert(w4[i], gr[w * NG / KW], gr[w * NG / KW]));
            }
          }
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && !late) mbar_arrive(&kv_full[buf]);
        ++item;
        // ---- V ----
        buf = item % kBufs;
        if (item >= kBufs) {
          if (!late) late = !__all_sync(kFull, mbar_wait_bounded(&kv_empty[buf], e_phase >> buf & 1u));
          e_phase ^= 1u << buf;
        }
        if (!late) {
          Group gr[KW];  // of each 32 elements
#pragma unroll
          for (int gi = 0; gi < NG; ++gi) {
            const Group y = group_of(vpar[gi], ve);
#pragma unroll
            for (int i = gi * (KW / NG); i < (gi + 1) * (KW / NG); ++i) gr[i] = y;
          }
          const uint32_t dst = buf_at + buf * L::kOperand + r * 128 + ((r & 7) << 4);
          uint32_t vw[8][VW];
#pragma unroll
          for (int g = 0; g < 8; ++g) {
            const uint32_t at = blk + 8 * D + v_word_byte<D>(g, row, 0);
            if constexpr (VW == 1) {
              vw[g][0] = lds_u32_a(at);
            } else {
              const uint2 v = lds_u64_a(at);
              vw[g][0] = v.x, vw[g][1] = v.y;
            }
          }
#pragma unroll
          for (int g = 0; g < 8; ++g) {
#pragma unroll
            for (int w = 0; w < VW; ++w) {
              // nibbles 0..3 and 4..7: elements 32 apart, of two groups when groups have 32
              sts128((dst ^ (g << 4)) + w * (kKeys * 128), convert(vw[g][w], gr[2 * w], gr[2 * w + 1]));
            }
          }
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && !late) {
          mbar_arrive(&kv_full[buf]);
          mbar_arrive(&raw_empty[stage]);
        }
        ++item;
        ++tiles;
        if (++stage == L::kStages) stage = 0, phase ^= 1u;
      }
      if (!ok || !next_piece(here)) break;
      ++piece;
    }
    if ((!ok || late) && lane == 0) give_up(kStatusFullWait);
  } else {
    tc::setmaxnreg_inc<168>();
    // ------------------------------ softmax -------------------------------------
    const int x = wg - 2;
    const int r = tid & 127;  // row of the row tile, tensor memory lane
    const uint32_t lane_at = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t s_at = lane_at + kColS + x * 128, o_at = lane_at + kColO + x * 128;
    const float c0 = fmaxf(fabsf(a.scale) * kLog2e, 1e-30f);
    const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;
    uint32_t s_phase = 0, o_phase = 0;
    int tiles = 0, piece = 0;
    bool ok = true;
    if (tid == 256) pieces[blockIdx.x].first = -1;
    while (left > 0) {
      const bool from_start = cur.tile == cur.t0;
      const int here = (int)min(left, (int64_t)(cur.t1 - cur.tile));
      const int rows = cur.qlen * G, row = cur.rt * kRows + x * 128 + r;
      const bool live = row < rows;
      const int tok = live ? row / G : 0, head = live ? row - tok * G : 0;
      const int wrow = r & ~31;  // first row of this warp
      {
        // whole rows of q by neighbouring lanes: a lane that reads its own row takes a line for every 16 bytes
        const int64_t own = (int64_t)(cur.q0 + tok) * a.q_stride + ((int64_t)cur.kvh * G + head) * D;
        constexpr int kChunks = D / 8, kAtOnce = 32 / kChunks, kLoads = 32 / kAtOnce;  // 16-byte chunks of a row, rows an instruction
        const int ch = lane % kChunks;
#pragma unroll 1
        for (int i0 = 0; i0 < 32; i0 += kLoads * kAtOnce) {
          uint4 v[kLoads];
#pragma unroll
          for (int i = 0; i < kLoads; ++i) {
            const int from = i0 + i * kAtOnce + lane / kChunks;
            const int64_t at = __shfl_sync(kFull, own, from);
            const bool there = __shfl_sync(kFull, (int)live, from) != 0;
            v[i] = there ? *reinterpret_cast<const uint4*>(static_cast<const __half*>(a.q) + at + ch * 8) : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int i = 0; i < kLoads; ++i) {
            const int to = wrow + i0 + i * kAtOnce + lane / kChunks;
            const uint4 p = in_code_order(v[i]);
            sts128(q_at + x * (L::kQ / 2) + tile_row_byte(to, ch),
                   make_uint4(p.x ^ flip, p.y ^ flip, p.z ^ flip, p.w ^ flip));
          }
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[x]);
      }
      const int pos = cur.n - cur.qlen + tok;
      const int lim_hi = a.causal ? min(cur.n, pos + 1) : cur.n;
      const int lim_lo = a.window > 0 ? pos - a.window + 1 : 0;
      float m = -FLT_MAX, l0 = 0.0f, l1 = 0.0f;
      int v_power = 0;  // O is held at 2^v_power, the power of the piece's largest V tile so far
      for (int j = 0; j < here; ++j) {
        const int base = (cur.tile + j) * kKeys;
        if (ok && !__all_sync(kFull, mbar_wait_bounded(&s_full[x], s_phase))) {
          if (lane == 0) give_up(kStatusMmaWait);
          ok = false;
        }
        s_phase ^= 1u;
        if (!ok) break;
        tc::fence_after_sync();
        // The second half of the scores is read twice, for its maximum and for its probabilities: the whole row
        // would not leave registers for the rest.
        float v[64];
        auto load_half = [&](int half) {
          tc::tmem_ld32(s_at + 64 * half, *reinterpret_cast<float(*)[32]>(&v[0]));
          tc::tmem_ld32(s_at + 64 * half + 32, *reinterpret_cast<float(*)[32]>(&v[32]));
        };
        load_half(1);
        const uint32_t in = tile_info[tiles % kMeta], have = in & 0xffu;
        const float c1 = c0 * pow2(64 - (int)(in >> 8 & 0xffu));
        const int ve = (int)(in >> 16) - 64;
        const bool masked = __any_sync(kFull, base < lim_lo || base + kKeys > lim_hi || have != 0xffu);
        ++tiles;
        // keys of a half that this row does not see, as bits (a block's 16 keys together when it was not read)
        auto mask_half = [&](int half) {
          const int lo = min(max(lim_lo - base - 64 * half, 0), 64), hi = min(max(lim_hi - base - 64 * half, 0), 64);
          uint64_t see = hi == 64 ? ~0ull : (1ull << hi) - 1;
          see = lo == 64 ? 0 : see >> lo << lo;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (!(have >> (4 * half + i) & 1)) see &= ~(0xffffull << (16 * i));
          const uint32_t s0 = (uint32_t)see, s1 = (uint32_t)(see >> 32);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            if (!(s0 >> i & 1)) v[i] = -INFINITY;
            if (!(s1 >> i & 1)) v[32 + i] = -INFINITY;
          }
        };
        auto top_half = [&]() {
          float t0 = v[0], t1 = v[1];
#pragma unroll
          for (int i = 2; i < 62; i += 4) t0 = max3(t0, v[i], v[i + 1]), t1 = max3(t1, v[i + 2], v[i + 3]);
          return fmaxf(max3(t0, v[62], v[63]), t1);
        };
        // Most loops that could be unrolled are not: the four roles' code has to stay in the instruction cache together (a chunk
        // of 2048 over 32768 keys, when this was chosen: 805 us; with this loop unrolled too 878, with the one below rolled 921).
        float top = -INFINITY;
#pragma unroll 1
        for (int half = 1; half >= 0; --half) {
          if (half == 0) load_half(0);
          tc::tmem_wait_ld();
          if (masked) mask_half(half);
          top = fmaxf(top, top_half());
        }
        top *= c1;
        if (__any_sync(kFull, top > m + kRise) || ve < v_power) {
          const float m2 = top > m + kRise ? top - kLift : m;
          float al = ex2(m - m2);
          m = m2;
          l0 *= al, l1 *= al;
          al *= pow2(min(ve - v_power, 0));
          v_power = min(v_power, ve);
          if (j > 0) {
#pragma unroll 1
            for (int i = 0; i < D / 32; ++i) {
              float o[32];
              tc::tmem_ld32(o_at + 32 * i, o);
              tc::tmem_wait_ld();
              uint32_t u[32];
#pragma unroll
              for (int k = 0; k < 32; ++k) u[k] = __float_as_uint(o[k] * al);
              tc::tmem_st32(o_at + 32 * i, u);
            }
          }
        }
        const float shift = -m - (float)(ve - v_power);
        float t0 = 0.0f, t1 = 0.0f;
        // P overlays S: keys 64 h .. 64 h + 63 go to columns 32 h .. 32 h + 31, whose scores are in registers
        // or used up. The products start on the first half while the second is made.
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (half == 1) {
            load_half(1);
            tc::tmem_wait_ld();
            if (masked) mask_half(1);
          }
          uint32_t p[32];
#pragma unroll
          for (int i = 0; i < 64; i += 2) {
            fma2(v[i], v[i + 1], c1, shift);
            v[i] = ex2(v[i]), v[i + 1] = ex2(v[i + 1]);
            add2(t0, t1, v[i], v[i + 1]);
            p[i / 2] = pack_half2(v[i], v[i + 1]);
          }
          tc::tmem_st32(s_at + 32 * half, p);
          tc::tmem_wait_st();
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[x][half]);
        }
        const float back = pow2(ve - v_power);
        l0 = fmaf(t0, back, l0), l1 = fmaf(t1, back, l1);
      }
      // ---- the end of this piece ----
      if (ok && !__all_sync(kFull, mbar_wait_bounded(&o_full, o_phase))) {
        if (lane == 0) give_up(kStatusMmaWait);
        ok = false;
      }
      o_phase ^= 1u;
      tc::fence_after_sync();
      // V values that are not finite: look for them again in the cache, 32 keys at a time
      uint32_t nan_groups = 0;
      if (odd_piece[piece % kMeta] == piece + 1) {
        const int ppb = c.page_blocks, end = min((cur.tile + here) * kKeys, cur.n);
        for (int k0 = cur.tile * kKeys; k0 < end; k0 += 32) {
          uint32_t bad = 0;
          if (k0 + lane < end) {
            const uint32_t blk = (uint32_t)(k0 + lane) / 16, pi = (uint32_t)((uint64_t)blk * page_magic >> 36);
            const int page = a.page_table[(int64_t)cur.b * a.table_stride + pi];
            if (page >= 0 && page < c.num_pages) {
              const uint8_t* at = c.pages + (((uint64_t)page * c.kv_heads + cur.kvh) * ppb + (blk - pi * ppb)) * L::kBlock;
              for (int gi = 0; gi < NG; ++gi) {
                const uint32_t p = *reinterpret_cast<const uint32_t*>(at + 16 * D + ((NG + gi) * 16 + (k0 + lane) % 16) * 4);
                if ((p & 0x7c00u) == 0x7c00u || (p & 0x7c000000u) == 0x7c000000u) bad |= 1u << gi;
              }
            }
          }
          if (__any_sync(kFull, bad != 0))
            for (int k = 0; k < 32; ++k) {
              const uint32_t w = __shfl_sync(kFull, bad, k);
              if (k0 + k >= lim_lo && k0 + k < lim_hi) nan_groups |= w;
            }
        }
      }
      const bool ends = cur.tile + here == cur.t1;
      const bool whole = from_start && ends;
      const float l = ok ? l0 + l1 : NAN;
      const bool none = l == 0.0f;
      const float f = (whole ? (none ? 0.0f : 1.0f / l) : 1.0f) * pow2(-v_power);
      float* slot = slots + ((int64_t)blockIdx.x * 2 + (from_start ? 1 : 0)) * kSlot;
      const int64_t out_row = (int64_t)(cur.q0 + tok) * a.q_heads + (int64_t)cur.kvh * G + head;
      // 64 elements of 32 rows at a time through the bytes of these rows' own q (the products have read it, and only this
      // warp writes it), so that neighbouring lanes store whole lines
      uint8_t* room = smem + x * (L::kQ / 2);
      constexpr bool kCutRoom = D == 128;  // 64 elements of a row in fp32 fit
#pragma unroll 1
      for (int w = 0; w < VW; ++w) {
        // column 64 w + 8 g + 4 (n & 1) + 2 h + n / 2 holds element 64 w + 32 h + 4 g + n
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {  // g of 4 half ..
          float o[32];
          if (ok) {
            tc::tmem_ld32(o_at + 64 * w + 32 * half, o);
            tc::tmem_wait_ld();
          }
          // 0 of a row that sees nothing (its l is 0 and so is f), NaN of groups that have one and of a call that gave up
          const float f0 = (nan_groups >> (2 * w * NG / KW) & 1) || !ok ? NAN : f;
          const float f1 = (nan_groups >> ((2 * w + 1) * NG / KW) & 1) || !ok ? NAN : f;
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = none && whole ? 0.0f : o[i] * (i & 2 ? f1 : f0);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int g2 = 0; g2 < 4; g2 += 2) {  // elements 32 h + 16 half + 4 g2 .. + 7 of the 64
              float y[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) y[k] = o[8 * (g2 + k / 4) + 4 * (k & 1) + 2 * h + k % 4 / 2];
              const int d8 = 4 * h + 2 * half + g2 / 2;  // eight elements
              if (whole) {
                *reinterpret_cast<uint4*>(room + tile_row_byte(wrow + lane, d8)) = make_uint4(
                    pack_half2(y[0], y[1]), pack_half2(y[2], y[3]), pack_half2(y[4], y[5]), pack_half2(y[6], y[7]));
              } else if (kCutRoom) {
                *reinterpret_cast<float4*>(room + tile_row_byte(wrow + lane, 2 * d8)) = make_float4(y[0], y[1], y[2], y[3]);
                *reinterpret_cast<float4*>(room + tile_row_byte(wrow + lane, 2 * d8 + 1)) =
                    make_float4(y[4], y[5], y[6], y[7]);
              } else if (live) {
                float4* s4 = reinterpret_cast<float4*>(slot + (x * 128 + r) * D + 64 * w + 8 * d8);
                s4[0] = make_float4(y[0], y[1], y[2], y[3]);
                s4[1] = make_float4(y[4], y[5], y[6], y[7]);
              }
            }
          }
        }
        __syncwarp();
        if (whole) {
#pragma unroll 2
          for (int i = 0; i < 8; ++i) {
            const int from = 4 * i + lane / 8, ch = lane % 8;
            const int64_t to = __shfl_sync(kFull, out_row, from);
            const bool there = __shfl_sync(kFull, (int)live, from) != 0;
            const uint4 y = *reinterpret_cast<const uint4*>(room + tile_row_byte(wrow + from, ch));
            if (there) *reinterpret_cast<uint4*>(static_cast<__half*>(a.out) + to * D + 64 * w + 8 * ch) = y;
          }
        } else if (kCutRoom) {
#pragma unroll 4
          for (int i = 0; i < 16; ++i) {
            const int from = 2 * i + lane / 16, ch = lane % 16;
            const bool there = __shfl_sync(kFull, (int)live, from) != 0;
            const float4 y = *reinterpret_cast<const float4*>(room + tile_row_byte(wrow + from, ch));
            if (there) *reinterpret_cast<float4*>(slot + (x * 128 + wrow + from) * D + 64 * w + 4 * ch) = y;
          }
        }
        __syncwarp();
      }
      if (live) {
        if (whole) {
          if (a.lse) a.lse[out_row] = none ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
        } else {
          *reinterpret_cast<float2*>(slot + kRows * D + (x * 128 + r) * 2) = make_float2(m, l);
        }
      }
      if (tid == 256 && !from_start && ends) {
        const int64_t s0 = range.u1 - left - (cur.tile - cur.t0);
        pieces[blockIdx.x] = {(int)range.cut.part_of(s0), cur.q0, cur.rt * kRows, rows, cur.kvh};
      }
      tc::fence_before_sync();
      if (!next_piece(here)) break;
      ++piece;
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 1) tc::tmem_dealloc(tmem, 512);
}

template <int D, int NG>
cudaError_t launch_tile(LaunchCtx& ctx, const Kv4Cache& c, const Kv4Attention& a) {
  auto kern = kv4_tile_kernel<D, NG>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(kern, TileSmem<D, NG>::kBytes, ctx.device, done);
  if (e != cudaSuccess) return e;
  const int grid = ctx.num_sms < 160 ? ctx.num_sms : 160;
  const uint64_t ppb = (uint64_t)(c.page_size / 16), magic = ((1ull << 36) + ppb - 1) / ppb;
  e = launch_kernel(ctx, kern, dim3(grid), dim3(kThreads), TileSmem<D, NG>::kBytes, c, a, magic, ctx.status);
  if (e != cudaSuccess) return e;
  const bool pdl = ctx.pdl;
  ctx.pdl = true;  // the joining kernel waits for this one on the device
  e = launch_kernel(ctx, kv4_join_kernel<D, kRows / 8, false>, dim3(ctx.num_sms), dim3(kJoinWarps * 32), 0, c, a, grid);
  ctx.pdl = pdl;
  return e;
}

}  // namespace

size_t kv4_tile_workspace_bytes(int D) {
  return (size_t)kMaxCtas * sizeof(Piece) + (size_t)160 * 2 * kRows * (D + 2) * 4;
}

cudaError_t launch_kv4_tile(LaunchCtx& ctx, const Kv4Cache& c, const Kv4Attention& a) {
  if (c.head_dim == 64) return c.group == 32 ? launch_tile<64, 2>(ctx, c, a) : launch_tile<64, 1>(ctx, c, a);
  if (c.group == 32) return launch_tile<128, 4>(ctx, c, a);
  return c.group == 64 ? launch_tile<128, 2>(ctx, c, a) : launch_tile<128, 1>(ctx, c, a);
}

}  // namespace mnb
