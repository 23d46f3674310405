// Cached positions as dense rows in the model's basis (kvq_read_back).
//
// x^ = code*scale + zero (one fp32 fma) for quantized positions, and for
// rotated keys the inverse transform k = signs * (H x^) / sqrt(d) (the
// Sylvester matrix H is symmetric and H H = d I); the bf16 rows of the ring as
// they are.  Bound by memory: per position d*(kb+vb)/8 bytes of codes and the
// metadata in, 2*d values out (the larger part).
//
// One CTA per (64-position page, kv-head, key or value).  A thread makes
// eight channels of a position at a time, so that 16 (or 8) lanes write one
// whole row: its stores are 16 bytes wide and a warp's are contiguous.  Code
// rows along channels (keys) give a thread its eight codes in one load; code
// runs along positions (values, keys with groups along positions) are read as
// one word of eight channels each, which the thread keeps for the 32/bits
// positions that the words hold.
#include "kvq_sink.cuh"

namespace kvq {
namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
}

__device__ __forceinline__ void store8(const ReadBackArgs& a, void* out, size_t at, const float (&x)[8]) {
    if (a.out_bf16) {
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(out) + at) =
            make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
    } else {
        float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
        o[0] = make_float4(x[0], x[1], x[2], x[3]);
        o[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
}

// the inverse rotation of a row whose channels 8*oct .. 8*oct+7 lie in x; D/8 neighbouring lanes hold the row
template <int D>
__device__ __forceinline__ void rotate_back(float (&x)[8], const int8_t* signs, int oct, unsigned lanes) {
#pragma unroll
    for (int s = 1; s < 8; s <<= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (!(i & s)) {
                const float u = x[i], w = x[i + s];
                x[i] = u + w;
                x[i + s] = u - w;
            }
#pragma unroll
    for (int m = 1; m < D / 8; m <<= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float o = __shfl_xor_sync(lanes, x[i], m);
            x[i] = (oct & m) ? o - x[i] : x[i] + o;
        }
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * RotScale<D>::v * float(__ldg(signs + oct * 8 + i));
}

struct Tile {
    int b, h, pg;              // pg: physical page, -1 when absent
    int x0;                    // position of slot 0
    int lo, hi;                // rows wanted: positions [lo, hi)
    int L, Lq;
    long long row0;            // output row of position x is x + row0
};

template <int D>
__device__ __forceinline__ size_t out_at(const Params& p, const Tile& t, int x, int oct) {
    return (size_t(x + t.row0) * p.hkv + t.h) * D + oct * 8;
}

// eight codes of a token row: bits [8*oct*BITS, 8*(oct+1)*BITS)
template <int BITS>
__device__ __forceinline__ void row_codes(const uint8_t* blk, int ch, int slot, int oct, float (&c)[8]) {
    const int byte = oct * BITS;
    const uint8_t* at = blk + (byte / ch) * (kPage * ch) + slot * ch + byte % ch;
    uint64_t w;
    if (BITS == 8) w = __ldg(reinterpret_cast<const unsigned long long*>(at));
    if (BITS == 4) w = __ldg(reinterpret_cast<const uint32_t*>(at));
    if (BITS == 2) w = __ldg(reinterpret_cast<const uint16_t*>(at));
    if (BITS == 1) w = __ldg(at);
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = float(uint32_t(w >> (i * BITS)) & ((1u << BITS) - 1u));
}

// keys with groups along channels: one thread per (position, eight channels)
template <int BITS, int D>
__device__ __forceinline__ void token_rows(const Params& p, const ReadBackArgs& a, const Tile& t) {
    const uint8_t* blk = k_block(p, t.pg, t.h);
    for (int e = threadIdx.x; e < kPage * (D / 8); e += kThreads) {
        const int slot = e / (D / 8), oct = e % (D / 8), x = t.x0 + slot;
        // the D/8 lanes of one row take the same way
        const unsigned lanes = __ballot_sync(0xffffffffu, x >= t.lo && x < t.hi && x < t.Lq);
        if (x < t.lo || x >= t.hi || x >= t.Lq) continue;
        float c[8];
        row_codes<BITS>(blk, p.kch, slot, oct, c);
        const float2 f = meta_f2(__ldg(k_meta_row(p, t.pg, t.h, slot) + oct * 8 / p.kg));
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = fmaf(c[i], f.x, f.y);
        if (p.rotate) rotate_back<D>(c, p.signs, oct, lanes);
        store8(a, a.k_out, out_at<D>(p, t, x, oct), c);
    }
}

// channel runs: one thread per (word of 32/BITS positions, eight channels)
template <int BITS, int D, bool KEYS>
__device__ __forceinline__ void channel_runs(const Params& p, const ReadBackArgs& a, const Tile& t) {
    constexpr int N = 32 / BITS, WORDS = kPage / N, RUN = kPage * BITS / 8, CH = RUN < 16 ? RUN : 16;
    const uint8_t* blk = (KEYS ? p.k_codes : p.v_codes) + (size_t(t.pg) * p.hkv + t.h) * size_t(D) * RUN;
    for (int e = threadIdx.x; e < WORDS * (D / 8); e += kThreads) {
        const int w = e / (D / 8), oct = e % (D / 8);
        if (t.x0 + w * N >= min(t.hi, t.Lq) || t.x0 + (w + 1) * N <= t.lo) continue;
        uint32_t word[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            word[i] = __ldg(reinterpret_cast<const uint32_t*>(blk + (w * 4 / CH) * (D * CH) + (oct * 8 + i) * CH + w * 4 % CH));
#pragma unroll 4
        for (int n = 0; n < N; ++n) {
            const int slot = w * N + n, x = t.x0 + slot;
            if (x < t.lo || x >= t.hi || x >= t.Lq) continue;
            float c[8];
            if (KEYS) {
                const uint32_t* m = p.k_meta + ((size_t(t.pg) * p.hkv + t.h) * (kPage / p.kg) + slot / p.kg) * D + oct * 8;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 f = meta_f2(__ldg(m + i));
                    c[i] = fmaf(float((word[i] >> (n * BITS)) & ((1u << BITS) - 1u)), f.x, f.y);
                }
            } else {
                const float2 f = meta_f2(__ldg(v_meta_row(p, t.pg, t.h, slot) + oct * 8 / p.vg));
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    c[i] = fmaf(float((word[i] >> (n * BITS)) & ((1u << BITS) - 1u)), f.x, f.y);
            }
            store8(a, KEYS ? a.k_out : a.v_out, out_at<D>(p, t, x, oct), c);
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads) read_back_kernel(Params p, ReadBackArgs a) {
    Tile t;
    t.b = blockIdx.z;
    t.h = blockIdx.y >> 1;
    const bool keys = !(blockIdx.y & 1);
    const int r0 = __ldg(a.cu_rows + t.b), n = __ldg(a.cu_rows + t.b + 1) - r0;
    if (n <= 0 || n > a.max_rows) return;
    // positions in 64 bits until they are known to be near the cache
    const long long first = __ldg(a.first + t.b);
    const long long x0 = ((first >> 6) + blockIdx.x) * kPage;
    if (x0 >= first + n) return;
    t.L = max(0, __ldg(a.lens + t.b));
    t.Lq = sink::paged_len(p, a.kpc, t.L);
    t.row0 = (long long)r0 - first;
    const long long lo = max(x0, first), hi = min(x0 + kPage, first + n);
    t.x0 = int(max(min(x0, (long long)INT32_MAX - kPage), (long long)INT32_MIN));
    t.pg = -1;
    const bool near = x0 >= 0 && x0 < t.L;
    if (near && t.x0 < t.Lq) t.pg = phys_page(p, t.b, t.x0 / kPage);
    void* out = keys ? a.k_out : a.v_out;
    // ring rows, and zeros for positions that are not there
    const int R = sink::ring_slots(p, a.kpc);
    for (int e = threadIdx.x; e < kPage * (D / 8); e += kThreads) {
        const int oct = e % (D / 8);
        const long long x = x0 + e / (D / 8);
        if (x < lo || x >= hi) continue;
        float c[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (x >= 0 && x < t.L) {
            if (x < t.Lq) {
                if (t.pg >= 0) continue;
            } else {
                const uint4 w = __ldg(reinterpret_cast<const uint4*>(
                    (keys ? p.k_win : p.v_win) + ((size_t(t.b) * p.hkv + t.h) * R + int(x) % R) * D + oct * 8));
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    c[2 * i] = __uint_as_float(u[i] << 16);
                    c[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
                }
            }
        }
        store8(a, out, (size_t(x + t.row0) * p.hkv + t.h) * D + oct * 8, c);
    }
    if (t.pg < 0) return;
    t.lo = int(lo);
    t.hi = int(hi);
    if (!keys) {
        if (p.vb == 1) channel_runs<1, D, false>(p, a, t);
        if (p.vb == 2) channel_runs<2, D, false>(p, a, t);
        if (p.vb == 4) channel_runs<4, D, false>(p, a, t);
        if (p.vb == 8) channel_runs<8, D, false>(p, a, t);
    } else if (a.kpc) {
        if (p.kb == 1) channel_runs<1, D, true>(p, a, t);
        if (p.kb == 2) channel_runs<2, D, true>(p, a, t);
        if (p.kb == 4) channel_runs<4, D, true>(p, a, t);
        if (p.kb == 8) channel_runs<8, D, true>(p, a, t);
    } else {
        if (p.kb == 1) token_rows<1, D>(p, a, t);
        if (p.kb == 2) token_rows<2, D>(p, a, t);
        if (p.kb == 4) token_rows<4, D>(p, a, t);
        if (p.kb == 8) token_rows<8, D>(p, a, t);
    }
}

}  // namespace

cudaError_t launch_read_back(const Params& p, const ReadBackArgs& a, cudaStream_t s) {
    // a run of max_rows positions touches at most this many pages
    const dim3 grid((a.max_rows + 2 * (kPage - 1)) / kPage, 2 * p.hkv, p.batch);
    if (p.d == 128)
        read_back_kernel<128><<<grid, kThreads, 0, s>>>(p, a);
    else
        read_back_kernel<64><<<grid, kThreads, 0, s>>>(p, a);
    return cudaGetLastError();
}

}  // namespace kvq
