// Attention over the paged 4-bit key/value cache: which kernel runs.
#include "kv4_stream.cuh"

namespace mnb {
namespace {

// Rows that an average sequence has for one key head.
int64_t rows_of(int T, int batch, int G) { return ((int64_t)T + batch - 1) / batch * G; }

// Column groups (of 8 rows) of the streaming kernel's row tile. Above 8 rows two: 16 rows of 16 x 4096, 4 x 32768 and 64 x 2048
// keys (8 key heads of 128) take 34, 54 and 65 us, with two tiles of one group 39, 65 and 75. More rows take more
// tiles of 16: at 32 rows 54, 90 and 110 us, where tiles of 32 (four groups) took 57, 94 and 110, and with heads of 64 40, 64 and 75
// against 44, 66 and 80.
int column_groups(int64_t rows) { return rows <= 8 ? 1 : 2; }

// Whether the tcgen05 kernel takes the call (fp16, heads of 64 and 128). Its time is that of 256 rows whatever their
// number, the streaming kernel's grows with every 16 rows and with the parameters of a key. At 48 rows, the same three key counts:
// heads of 64 in groups of 32 / 64: streaming 64, 106, 125 / 54, 87, 103 us, tcgen05 75, 108, 134 / 75, 107, 132;
// heads of 128, one group: streaming 75, 126, 154, tcgen05 82, 125, 169 (at 52 rows 95, 159, 196
// and 82, 124, 169); with groups of 64 at 36 rows: streaming 84, 140, 171, tcgen05 84, 124, 172; with groups of 32: streaming 114, 199, 234,
// tcgen05 90, 136, 187, at 32 rows streaming 82, 139, 165.
constexpr int kFewRows = 32, kMoreRows = 48;
bool takes_tiles(int64_t rows, int D, int f32, int group) {
  return !f32 && D <= 128 && rows > (D == 64 || group == D ? kMoreRows : kFewRows);
}

}  // namespace

size_t kv4_tile_workspace_bytes(int D);
cudaError_t launch_kv4_tile(LaunchCtx& ctx, const Kv4Cache& c, const Kv4Attention& a);

size_t kv4_attention_workspace_bytes(int T, int batch, int q_heads, int kv_heads, int D, int f32) {
  const int64_t rows = rows_of(T, batch, q_heads / kv_heads);
  // the larger of both kernels' where the cache's groups decide between them
  if (!f32 && D <= 128 && rows > kFewRows) return kv4_tile_workspace_bytes(D);
  const int nt = column_groups(rows);
  return (size_t)kv4::kMaxCtas * (sizeof(kv4::Piece) + (size_t)2 * 8 * nt * (D + 2) * 4);
}

cudaError_t launch_kv4_attention(LaunchCtx& ctx, const Kv4Cache& c, const Kv4Attention& a) {
  const int64_t rows = rows_of(a.T, a.batch, a.q_heads / c.kv_heads);
  if (takes_tiles(rows, c.head_dim, a.f32, c.group)) {
    ctx.variant = "kv4_tile_tcgen05";
    return launch_kv4_tile(ctx, c, a);
  }
  const int nt = column_groups(rows);
  static const char* names[2][2] = {{"kv4_stream_f16_rows8", "kv4_stream_f16_rows16"},
                                    {"kv4_stream_f32_rows8", "kv4_stream_f32_rows16"}};
  ctx.variant = names[a.f32 ? 1 : 0][nt - 1];
  if (c.head_dim == 64) return a.f32 ? launch_kv4_stream_d64_f32(ctx, c, a, nt) : launch_kv4_stream_d64_f16(ctx, c, a, nt);
  if (c.head_dim == 128)
    return a.f32 ? launch_kv4_stream_d128_f32(ctx, c, a, nt) : launch_kv4_stream_d128_f16(ctx, c, a, nt);
  return a.f32 ? launch_kv4_stream_d256_f32(ctx, c, a, nt) : launch_kv4_stream_d256_f16(ctx, c, a, nt);
}

}  // namespace mnb
