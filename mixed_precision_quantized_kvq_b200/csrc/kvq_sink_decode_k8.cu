// Single-token attention with sinks: the kernels for 8-bit keys.
#include "kvq_sink_decode.cuh"

namespace kvq {

cudaError_t launch_sink_decode_k8(const Params& p, const sink::Args& a, int sms, cudaStream_t s) {
    return sink::launch_decode_bits<8>(p, a, sms, s);
}

}  // namespace kvq
