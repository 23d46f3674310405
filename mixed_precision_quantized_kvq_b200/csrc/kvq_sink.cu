// Dispatch of the attention with sinks and a sliding span.
#include "kvq_sink.cuh"

namespace kvq {

cudaError_t launch_sink_decode_k1(const Params&, const sink::Args&, int, cudaStream_t);
cudaError_t launch_sink_decode_k2(const Params&, const sink::Args&, int, cudaStream_t);
cudaError_t launch_sink_decode_k4(const Params&, const sink::Args&, int, cudaStream_t);
cudaError_t launch_sink_decode_k8(const Params&, const sink::Args&, int, cudaStream_t);
namespace sink {
cudaError_t launch_prefill(const Params&, const Args&, int, unsigned*, cudaStream_t);
}

cudaError_t launch_sink_attention(const Params& p, const sink::Args& a, int sms, cudaStream_t s) {
    // one query per sequence, scales shared by 32 channels or more
    if (!a.cu_q && !a.kpc && p.kg >= 32) {
        switch (p.kb) {
            case 1: return launch_sink_decode_k1(p, a, sms, s);
            case 2: return launch_sink_decode_k2(p, a, sms, s);
            case 4: return launch_sink_decode_k4(p, a, sms, s);
            default: return launch_sink_decode_k8(p, a, sms, s);
        }
    }
    unsigned* status = status_words();
    if (!status) return cudaErrorInvalidSymbol;
    return sink::launch_prefill(p, a, sms, status, s);
}

}  // namespace kvq
