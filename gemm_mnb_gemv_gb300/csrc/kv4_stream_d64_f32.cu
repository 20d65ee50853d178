// Streaming attention (kv4_stream.cuh), heads of 64, fp32 activations.
#include "kv4_stream.cuh"

namespace mnb {
MNB_KV4_STREAM(d64_f32) { return kv4::launch_stream_d<64, true>(ctx, c, a, nt); }
}  // namespace mnb
