// Attention with sinks and a sliding span over the quantized cache on CUDA
// cores: one warp per (query, head) walks the positions the query sees with a
// running maximum and sum.  fp32 throughout.
#include "kvq_sink.cuh"

namespace kvq {
namespace {

// code of channel j at slot t of a channel-run block (values; keys with groups along positions)
__device__ __forceinline__ uint32_t run_code(const uint8_t* blk, int d, int ch, int bits, int t, int j) {
    const int bit = t * bits, byte = bit >> 3;
    return (uint32_t(blk[(byte / ch) * (d * ch) + j * ch + byte % ch]) >> (bit & 7)) & ((1u << bits) - 1u);
}

template <int D>
__global__ void sink_attention_kernel(Params p, sink::Args a) {
    constexpr int C = D / 32;
    const int b = blockIdx.z, h = blockIdx.y, i = blockIdx.x, lane = threadIdx.x % 32;
    const int head = h * p.g + threadIdx.x / 32;
    sink::Seq s;
    if (!sink::sequence(a, b, s) || i >= s.n) return;
    const int t = s.base + i, Lq = sink::paged_len(p, a.kpc, s.L), R = sink::ring_slots(p, a.kpc);
    const size_t row = s.row + i;
    float q[C], qr[C], o[C];
    for (int c = 0; c < C; ++c) {
        const size_t at = row * a.q_stride + size_t(head) * D + lane * C + c;
        q[c] = a.q_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[at])
                        : static_cast<const float*>(a.q)[at];
        qr[c] = q[c];
        o[c] = 0.f;
    }
    if (p.rotate) rotate_warp<D>(qr, p.signs, lane);
    float m = -INFINITY, l = 0.f;
    const int lo = sink::span_begin(t, a.span), ns = min(a.sinks, lo);
    for (int x = ns > 0 ? 0 : lo; x <= t; x = x + 1 == ns ? lo : x + 1) {
        float k[C], v[C];
        const bool paged = x < Lq;
        if (paged) {
            const int pg = phys_page(p, b, x / kPage), slot = x % kPage;
            if (pg < 0) continue;
            for (int c = 0; c < C; ++c) {
                const int j = lane * C + c;
                uint32_t code, meta;
                if (a.kpc) {
                    const int kb = kPage * p.kb / 8;
                    code = run_code(p.k_codes + (size_t(pg) * p.hkv + h) * size_t(D) * kb, D, kb < 16 ? kb : 16, p.kb, slot, j);
                    meta = p.k_meta[((size_t(pg) * p.hkv + h) * (kPage / p.kg) + slot / p.kg) * D + j];
                } else {
                    code = (*k_word(p, pg, h, slot, j * p.kb / 32) >> (j * p.kb % 32)) & ((1u << p.kb) - 1u);
                    meta = k_meta_row(p, pg, h, slot)[j / p.kg];
                }
                float2 f = meta_f2(meta);
                k[c] = fmaf(float(code), f.x, f.y);
                f = meta_f2(v_meta_row(p, pg, h, slot)[j / p.vg]);
                v[c] = fmaf(float(run_code(v_block(p, pg, h), D, p.vch, p.vb, slot, j)), f.x, f.y);
            }
        } else {
            const size_t w = ((size_t(b) * p.hkv + h) * R + x % R) * D + lane * C;
            for (int c = 0; c < C; ++c) {
                k[c] = __bfloat162float(p.k_win[w + c]);
                v[c] = __bfloat162float(p.v_win[w + c]);
            }
        }
        float dot = 0.f;
        for (int c = 0; c < C; ++c) dot = fmaf(paged ? qr[c] : q[c], k[c], dot);
        for (int w = 16; w; w >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, w);
        const float x2 = dot * a.scale_log2, mn = fmaxf(m, x2), f = exp2f(m - mn), e = exp2f(x2 - mn);
        m = mn;
        l = fmaf(l, f, e);
        for (int c = 0; c < C; ++c) o[c] = fmaf(o[c], f, e * v[c]);
    }
    for (int c = 0; c < C; ++c)
        a.out[(row * p.hq + head) * D + lane * C + c] = __float2bfloat16_rn(l > 0.f ? o[c] / l : 0.f);
    if (a.lse && lane == 0)
        a.lse[row * p.hq + head] = l > 0.f ? (m + log2f(l)) * 0.693147180559945309f : -INFINITY;
}

}  // namespace

cudaError_t launch_sink_decode_k1(const Params&, const sink::Args&, int, cudaStream_t);
cudaError_t launch_sink_decode_k2(const Params&, const sink::Args&, int, cudaStream_t);
cudaError_t launch_sink_decode_k4(const Params&, const sink::Args&, int, cudaStream_t);
cudaError_t launch_sink_decode_k8(const Params&, const sink::Args&, int, cudaStream_t);

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
    const dim3 grid(a.max_q, p.hkv, p.batch);
    if (p.d == 128)
        sink_attention_kernel<128><<<grid, 32 * p.g, 0, s>>>(p, a);
    else
        sink_attention_kernel<64><<<grid, 32 * p.g, 0, s>>>(p, a);
    return cudaGetLastError();
}

}  // namespace kvq
