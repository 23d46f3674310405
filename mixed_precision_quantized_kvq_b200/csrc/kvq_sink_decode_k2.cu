// Single-token attention with sinks: the kernels for 2-bit keys.
#include "kvq_sink_decode.cuh"

namespace kvq {

cudaError_t launch_sink_decode_k2(const Params& p, const sink::Args& a, int sms, cudaStream_t s) {
    return sink::launch_decode_bits<2>(p, a, sms, s);
}

}  // namespace kvq
