// Attention with sinks and a sliding span over the quantized cache, and
// reading the cache back: arguments, the visibility rule and the launchers
// that the C-ABI layer (kvq_api.cu) calls.
#pragma once

#include "kvq_internal.cuh"

namespace kvq {
namespace sink {

// Arguments of one attention call.  A query at position t sees position x
// when x <= t and (x < sinks or t - x < span).
struct Args {
    const void* q;              // bf16 or fp32 rows of [Hq][d], q_stride elements apart
    int q_bf16;
    long long q_stride;
    const int32_t* cu_q;        // prefill: query row offsets [B+1]; decode: null (one row per sequence)
    const int32_t* lens;        // [B]
    int len_cap;                // lengths above it are clamped to it
    int max_q;                  // bound on the rows of a sequence (1 for decode)
    int sinks, span;
    float scale_log2;           // score scale * log2(e)
    __nv_bfloat16* out;         // rows of [Hq][d]
    float* lse;                 // rows of [Hq] (natural log), or null
    int kpc;                    // key groups run along positions
};

// ring slots per (sequence, kv-head)
__host__ __device__ __forceinline__ int ring_slots(const Params& p, int kpc) { return kpc ? p.W + p.kg - 1 : p.W; }

// positions of a length-L sequence that live in pages
__host__ __device__ __forceinline__ int paged_len(const Params& p, int kpc, int L) {
    const int q = L > p.W ? L - p.W : 0;
    return kpc ? q - q % p.kg : q;
}

// first position of the span of a query at position t
__host__ __device__ __forceinline__ int span_begin(int t, int span) { return t >= span ? t - span + 1 : 0; }

// The rows of sequence b: its length, its first query's row and position, and
// how many queries it has.  Returns false when the sequence is skipped.
struct Seq {
    int L, n, base;
    size_t row;
};
__device__ __forceinline__ bool sequence(const Args& a, int b, Seq& s) {
    s.L = max(0, min(__ldg(a.lens + b), a.len_cap));
    if (a.cu_q) {
        const int r0 = __ldg(a.cu_q + b);
        s.n = __ldg(a.cu_q + b + 1) - r0;
        s.row = size_t(r0);
        if (s.n <= 0 || s.n > s.L || s.n > a.max_q) return false;
    } else {
        s.n = 1;
        s.row = size_t(b);
    }
    s.base = s.L - s.n;
    return true;
}

}  // namespace sink

cudaError_t launch_sink_attention(const Params& p, const sink::Args& a, int sms, cudaStream_t s);

// kvq_read_back: rows [cu_rows[b], cu_rows[b+1]) get positions first[b] ...
struct ReadBackArgs {
    const int32_t* first;
    const int32_t* cu_rows;
    const int32_t* lens;
    int max_rows;
    void* k_out;
    void* v_out;
    int out_bf16;
    int kpc;
};
cudaError_t launch_read_back(const Params& p, const ReadBackArgs& a, cudaStream_t s);

}  // namespace kvq
