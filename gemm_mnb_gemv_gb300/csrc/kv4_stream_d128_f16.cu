// Streaming attention (kv4_stream.cuh), heads of 128, fp16 activations.
#include "kv4_stream.cuh"

namespace mnb {
MNB_KV4_STREAM(d128_f16) { return kv4::launch_stream_d<128, false>(ctx, c, a, nt); }
}  // namespace mnb
