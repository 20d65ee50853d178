// Streaming attention (kv4_stream.cuh), heads of 128, fp32 activations.
#include "kv4_stream.cuh"

namespace mnb {
MNB_KV4_STREAM(d128_f32) { return kv4::launch_stream_d<128, true>(ctx, c, a, nt); }
}  // namespace mnb
