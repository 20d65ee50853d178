// Streaming attention, fp16 activations (kv4_stream.cuh).
#include "kv4_stream.cuh"

namespace mnb {

cudaError_t launch_kv4_stream_f16(LaunchCtx& ctx, const Kv4Cache& c, const Kv4Attention& a, int nt) {
  using namespace kv4;
  switch (c.head_dim * 8 + nt) {
    case 64 * 8 + 1: return launch_stream<64, 1, false>(ctx, c, a);
    case 64 * 8 + 2: return launch_stream<64, 2, false>(ctx, c, a);
    case 64 * 8 + 4: return launch_stream<64, 4, false>(ctx, c, a);
    case 128 * 8 + 1: return launch_stream<128, 1, false>(ctx, c, a);
    case 128 * 8 + 2: return launch_stream<128, 2, false>(ctx, c, a);
    case 128 * 8 + 4: return launch_stream<128, 4, false>(ctx, c, a);
    case 256 * 8 + 1: return launch_stream<256, 1, false>(ctx, c, a);
    case 256 * 8 + 2: return launch_stream<256, 2, false>(ctx, c, a);
  }
  return cudaErrorInvalidValue;
}

}  // namespace mnb
