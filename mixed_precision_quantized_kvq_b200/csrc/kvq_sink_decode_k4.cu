// Single-token attention with sinks: the kernels for 4-bit keys.
#include "kvq_sink_decode.cuh"

namespace kvq {

cudaError_t launch_sink_decode_k4(const Params& p, const sink::Args& a, int sms, cudaStream_t s) {
    return sink::launch_decode_bits<4>(p, a, sms, s);
}

}  // namespace kvq
