// Attention over the paged 4-bit key/value cache: one warp per (query token, query head).
//
// For each key the lanes form q . k over their D / 32 elements and add them by shuffles, then
// update a running maximum m, sum l and output o: with a = e^(m - m'), o' = o a + e^(s - m') v.
// A plain kernel that is right for every shape; latency-bound.
#include "kv4.cuh"
#include "mnb_device.cuh"
#include "mnb_internal.h"

namespace mnb {
namespace {

template <int D, bool F32>
__global__ void kv4_attention_plain(const Kv4Cache c, const Kv4Attention a, uint32_t* status) {
  pdl_wait();
  constexpr int E = D / 32;  // elements of a lane: d = lane * E ..
  const int lane = threadIdx.x % 32;
  const int64_t w = (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;
  if (w >= (int64_t)a.T * a.q_heads) return;
  const int t = (int)(w / a.q_heads), h = (int)(w % a.q_heads);
  int lo = 0, hi = a.batch;  // the last b with q_start[b] <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.q_start[mid] <= t) lo = mid; else hi = mid;
  }
  const int b = lo, q0 = a.q_start[b], q1 = min(a.q_start[b + 1], a.T);
  if (t < q0 || t >= q1) return;
  int n = max(a.kv_len[b], 0);
  if (n > a.table_stride * c.page_size) {
    n = a.table_stride * c.page_size;
    if (lane == 0) report_status(status, kStatusBadIndex);
  }
  const int kvh = h / (a.q_heads / c.kv_heads), ng = c.ng(), bb = c.block_bytes();
  const int pos = n - (q1 - q0) + (t - q0);
  const int end = a.causal ? min(n, pos + 1) : n;
  const int begin = a.window > 0 ? max(0, pos - a.window + 1) : 0;
  float q[E], o[E] = {};
  for (int i = 0; i < E; ++i) {
    const int64_t at = t * a.q_stride + (int64_t)h * D + lane * E + i;
    q[i] = (F32 ? static_cast<const float*>(a.q)[at] : __half2float(static_cast<const __half*>(a.q)[at])) * a.scale;
  }
  float m = -INFINITY, l = 0.0f;
  for (int j = begin; j < end; ++j) {
    const int page = a.page_table[(int64_t)b * a.table_stride + j / c.page_size];
    if (page < 0 || page >= c.num_pages) {
      if (lane == 0) report_status(status, kStatusBadIndex);
      continue;
    }
    const uint8_t* blk =
        c.pages + (((int64_t)page * c.kv_heads + kvh) * (c.page_size / 16) + j % c.page_size / 16) * bb;
    const int r = j % 16;
    float k[E], v[E], s = 0.0f;
    for (int i = 0; i < E; ++i) {
      const int d = lane * E + i, gi = d / c.group;
      const float2 kp = __half22float2(*reinterpret_cast<const __half2*>(blk + 16 * D + (gi * 16 + r) * 4));
      const float2 vp = __half22float2(*reinterpret_cast<const __half2*>(blk + 16 * D + ((ng + gi) * 16 + r) * 4));
      const uint32_t kw = *reinterpret_cast<const uint32_t*>(blk + kv4::k_word_byte<D>(r, d % 32 / 8, d / 32));
      const uint32_t vw =
          *reinterpret_cast<const uint32_t*>(blk + 8 * D + kv4::v_word_byte<D>(d % 32 / 4, r, d / 64));
      k[i] = fmaf((float)(kw >> (d % 8 * 4) & 15u), kp.x, kp.y);
      v[i] = fmaf((float)(vw >> (d % 4 * 4 + (d % 64 / 32) * 16) & 15u), vp.x, vp.y);
      s = fmaf(q[i], k[i], s);
    }
    for (int o2 = 16; o2; o2 >>= 1) s += __shfl_xor_sync(kFull, s, o2);
    const float m2 = fmaxf(m, s);
    const float al = m == -INFINITY ? 0.0f : expf(m - m2), p = s == -INFINITY ? 0.0f : expf(s - m2);
    l = l * al + p;
    for (int i = 0; i < E; ++i) o[i] = o[i] * al + p * v[i];
    m = m2;
  }
  for (int i = 0; i < E; ++i) {
    const int64_t at = ((int64_t)t * a.q_heads + h) * D + lane * E + i;
    const float y = l > 0.0f || l != l ? o[i] / l : 0.0f;
    if (F32) static_cast<float*>(a.out)[at] = y;
    else static_cast<__half*>(a.out)[at] = __float2half_rn(y);
  }
  if (a.lse && lane == 0) a.lse[(int64_t)t * a.q_heads + h] = l > 0.0f || l != l ? m + logf(l) : -INFINITY;
}

}  // namespace

size_t kv4_attention_workspace_bytes(int, int, int, int, int, int) { return 0; }

cudaError_t launch_kv4_attention(LaunchCtx& ctx, const Kv4Cache& c, const Kv4Attention& a) {
  ctx.variant = "kv4_attention_plain";
  const dim3 grid((unsigned)(((int64_t)a.T * a.q_heads + 3) / 4));
  auto go = [&](auto kern) { return launch_kernel(ctx, kern, grid, dim3(128), 0, c, a, ctx.status); };
  if (c.head_dim == 64) return a.f32 ? go(kv4_attention_plain<64, true>) : go(kv4_attention_plain<64, false>);
  if (c.head_dim == 128) return a.f32 ? go(kv4_attention_plain<128, true>) : go(kv4_attention_plain<128, false>);
  return a.f32 ? go(kv4_attention_plain<256, true>) : go(kv4_attention_plain<256, false>);
}

}  // namespace mnb
