// Streaming attention (kv4_stream.cuh), heads of 256, fp16 activations.
#include "kv4_stream.cuh"

namespace mnb {
MNB_KV4_STREAM(d256_f16) { return kv4::launch_stream_d<256, false>(ctx, c, a, nt); }
}  // namespace mnb
