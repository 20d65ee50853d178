// Attention over the paged 4-bit key/value cache: which kernel runs.
#include "kv4_stream.cuh"

namespace mnb {
namespace {

// Column groups (of 8 rows) of a row tile: the rows that an average sequence has for one key head, up to what the
// accumulators leave registers for.
int column_groups(int T, int batch, int G, int D, int f32) {
  const int64_t rows = ((int64_t)T + batch - 1) / batch * G;
  const int most = f32 || D == 256 ? 2 : 4;
  return rows <= 8 ? 1 : rows <= 16 || most == 2 ? 2 : 4;
}

// Whether the tcgen05 kernel takes the call: fp16, heads of 64 and 128, more rows a key head than the
// streaming kernel's widest row tile.
bool takes_tiles(int T, int batch, int G, int D, int f32) {
  return !f32 && D <= 128 && ((int64_t)T + batch - 1) / batch * G > 32;
}

}  // namespace

size_t kv4_tile_workspace_bytes(int D);
cudaError_t launch_kv4_tile(LaunchCtx& ctx, const Kv4Cache& c, const Kv4Attention& a);

size_t kv4_attention_workspace_bytes(int T, int batch, int q_heads, int kv_heads, int D, int f32) {
  if (takes_tiles(T, batch, q_heads / kv_heads, D, f32)) return kv4_tile_workspace_bytes(D);
  const int nt = column_groups(T, batch, q_heads / kv_heads, D, f32);
  return (size_t)kv4::kMaxCtas * (sizeof(kv4::Piece) + (size_t)2 * 8 * nt * (D + 2) * 4);
}

cudaError_t launch_kv4_attention(LaunchCtx& ctx, const Kv4Cache& c, const Kv4Attention& a) {
  if (takes_tiles(a.T, a.batch, a.q_heads / c.kv_heads, c.head_dim, a.f32)) {
    ctx.variant = "kv4_tile_tcgen05";
    return launch_kv4_tile(ctx, c, a);
  }
  const int nt = column_groups(a.T, a.batch, a.q_heads / c.kv_heads, c.head_dim, a.f32);
  static const char* names[2][3] = {{"kv4_stream_f16_rows8", "kv4_stream_f16_rows16", "kv4_stream_f16_rows32"},
                                    {"kv4_stream_f32_rows8", "kv4_stream_f32_rows16", ""}};
  ctx.variant = names[a.f32 ? 1 : 0][nt == 4 ? 2 : nt - 1];
  if (c.head_dim == 64) return a.f32 ? launch_kv4_stream_d64_f32(ctx, c, a, nt) : launch_kv4_stream_d64_f16(ctx, c, a, nt);
  if (c.head_dim == 128)
    return a.f32 ? launch_kv4_stream_d128_f32(ctx, c, a, nt) : launch_kv4_stream_d128_f16(ctx, c, a, nt);
  return a.f32 ? launch_kv4_stream_d256_f32(ctx, c, a, nt) : launch_kv4_stream_d256_f16(ctx, c, a, nt);
}

}  // namespace mnb
