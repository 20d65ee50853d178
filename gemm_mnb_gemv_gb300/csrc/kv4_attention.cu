// Attention over the paged 4-bit key/value cache: which kernel runs.
#include "kv4_stream.cuh"

namespace mnb {
namespace {

// Rows that an average sequence has for one key head.
int64_t rows_of(int T, int batch, int G) { return ((int64_t)T + batch - 1) / batch * G; }

// Column groups (of 8 rows) of the streaming kernel's row tile. Above 8 rows two: 16 rows of 16 x 4096, 4 x 32768 and 64 x 2048
// keys (8 key heads of 128) take 34, 55 and 67 us, with two tiles of one group 39, 65 and 75. More rows take more
// tiles of 16: at 32 rows 56, 92 and 112 us; tiles of 32 (four groups), when last measured, took 57, 94 and 110 against 54, 90 and 110, and with
// heads of 64 44, 66 and 80 against 40, 64 and 75.
int column_groups(int64_t rows) { return rows <= 8 ? 1 : 2; }

// Whether the tcgen05 kernel takes the call (fp16, heads of 64 and 128). Its time is that of 256 rows whatever their
// number, the streaming kernel's grows with every 16 rows and with the parameters of a key. At 48 rows, the same three key counts:
// heads of 64 in groups of 32 / 64: streaming 67, 110, 129 / 57, 91, 107 us, tcgen05 77, 110, 138 / 76, 109, 134;
// heads of 128, one group: streaming 77, 129, 158, tcgen05 84, 125, 176 (at 52 rows 98, 164, 201
// and 84, 126, 176); with groups of 64 at 36 rows: streaming 86, 147, 180, tcgen05 86, 128, 181; with groups of 32: streaming 117, 204, 240,
// tcgen05 94, 132, 192, at 32 rows streaming 84, 144, 168.
// Those are uniform batches. The rows are an average, and a mixed batch goes through one kernel: 63 decode tokens (1000 to 7014 keys) with
// a chunk of 512 tokens over 3000 keys take 224 us on the streaming kernel (alone the decode tokens 71, the chunk 50 on
// the tcgen05 one), with a chunk of 1500 376 us on the tcgen05 kernel (71 and 91).
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
