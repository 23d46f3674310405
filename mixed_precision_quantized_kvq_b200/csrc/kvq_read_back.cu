// Cached positions as dense rows in the model's basis (kvq_read_back).
//
// x^ = code*scale + zero (one fp32 fma) for quantized positions, and for
// rotated keys the inverse transform k = signs * (H x^) / sqrt(d) (the
// Sylvester matrix H is symmetric and H H = d I); the bf16 rows of the ring as
// they are.  Bound by memory: per position d*(kb+vb)/8 bytes of codes and the
// metadata in, 2*d values out (the larger part).
//
// One CTA per (64-position page, kv-head, key or value); CTAs of one page are
// neighbours, since their rows are in the output.  A thread owns eight channels
// and makes them for a few positions, so that 16 (or 8) lanes write one whole
// row: its stores are 16 bytes wide and a warp's are contiguous.  Code rows
// along channels (keys) give a thread its eight codes in one load; code runs
// along positions (values, keys with groups along positions) are read as one
// word of eight channels each, for D/16 neighbouring positions.
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

// Code n of a word as an fp32 number times 2^position(n): one mask puts it into the mantissa of 2^23, and taking 2^23 off
// is exact (integer conversions run at a quarter of the rate, shifts compete with the masks).  The power of two goes
// into the scale, also exactly; then one fp32 fma, as in the definition.
template <int BITS>
__device__ __forceinline__ constexpr int position(int n) { return n * BITS % 16; }
template <int BITS>
__device__ __forceinline__ float lifted(uint32_t w, int n) {
    const int at = position<BITS>(n);
    return __uint_as_float(((w >> (n * BITS - at)) & (((1u << BITS) - 1u) << at)) | 0x4b000000u) - 8388608.f;
}
template <int BITS>
__device__ __forceinline__ float lowered(float scale, int n) { return scale * (1.f / float(1 << position<BITS>(n))); }

struct Tile {
    int b, h, pg;              // pg: physical page, -1 when absent
    int x0;                    // position of slot 0
    int lo, hi;                // slots wanted that live in the page: [lo, hi)
};

// The output rows of a tile's slots, for this thread's channels.
template <int D>
struct Rows {
    static constexpr int kOct = D / 8, kGroups = kThreads / kOct;   // threads of a row, rows at a time
    int oct, group;
    size_t at, step;           // element of slot 0, elements between slots
};

// keys with groups along channels: eight codes of a position in one load
template <int BITS, int D>
__device__ __forceinline__ void token_rows(const Params& p, const ReadBackArgs& a, const Tile& t, const Rows<D>& r) {
    const int byte = r.oct * BITS;
    const uint8_t* codes = k_block(p, t.pg, t.h) + (byte / p.kch) * (kPage * p.kch) + byte % p.kch;
    const uint32_t* meta = k_meta_row(p, t.pg, t.h, 0) + (r.oct * 8 >> (__ffs(p.kg) - 1));
#pragma unroll 4
    for (int i = 0; i < kPage / Rows<D>::kGroups; ++i) {
        const int slot = i * Rows<D>::kGroups + r.group;
        const bool have = slot >= t.lo && slot < t.hi;
        // the lanes of one row take the same way
        const unsigned lanes = p.rotate ? __ballot_sync(0xffffffffu, have) : 0u;
        if (!have) continue;
        const uint8_t* at = codes + slot * p.kch;
        uint32_t w[2];
        if (BITS == 8) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(at));
            w[0] = v.x, w[1] = v.y;
        }
        if (BITS == 4) w[0] = __ldg(reinterpret_cast<const uint32_t*>(at));
        if (BITS == 2) w[0] = __ldg(reinterpret_cast<const uint16_t*>(at));
        if (BITS == 1) w[0] = __ldg(at);
        const float2 f = meta_f2(__ldg(meta + slot * p.nkg));
        float c[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int n = BITS == 8 ? k % 4 : k;
            c[k] = fmaf(lifted<BITS>(w[BITS == 8 ? k / 4 : 0], n), lowered<BITS>(f.x, n), f.y);
        }
        if (p.rotate) rotate_back<D>(c, p.signs, r.oct, lanes);
        store8(a, a.k_out, r.at + slot * r.step, c);
    }
}

// channel runs: D/16 neighbouring positions of eight channels
template <int BITS, int D, bool KEYS>
__device__ __forceinline__ void channel_runs(const Params& p, const ReadBackArgs& a, const Tile& t, const Rows<D>& r) {
    constexpr int N = 32 / BITS, RUN = kPage * BITS / 8, CH = RUN < 16 ? RUN : 16, T = kPage / Rows<D>::kGroups;
    constexpr int WORDS = (T + N - 1) / N;               // words a channel
    const int s0 = r.group * T;
    if (s0 >= t.hi || s0 + T <= t.lo) return;
    const uint8_t* blk = (KEYS ? p.k_codes : p.v_codes) + (size_t(t.pg) * p.hkv + t.h) * size_t(D) * RUN;
    uint32_t word[WORDS][8];
#pragma unroll
    for (int w = 0; w < WORDS; ++w) {
        const int byte = (s0 / N + w) * 4;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            word[w][k] = __ldg(reinterpret_cast<const uint32_t*>(blk + (byte / CH) * (D * CH) + (r.oct * 8 + k) * CH + byte % CH)) >>
                         (s0 % N * BITS);
    }
    const int gi = r.oct * 8 >> (__ffs(p.vg) - 1), kshift = __ffs(p.kg) - 1;
#pragma unroll
    for (int i = 0; i < T; ++i) {
        const int slot = s0 + i, n = i % N;
        if (slot < t.lo || slot >= t.hi) continue;
        float c[8];
        if (KEYS) {
            const uint4* m = reinterpret_cast<const uint4*>(
                p.k_meta + ((size_t(t.pg) * p.hkv + t.h) * (kPage >> kshift) + (slot >> kshift)) * D + r.oct * 8);
            const uint4 m0 = __ldg(m), m1 = __ldg(m + 1);
            const uint32_t mm[8] = {m0.x, m0.y, m0.z, m0.w, m1.x, m1.y, m1.z, m1.w};
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float2 f = meta_f2(mm[k]);
                c[k] = fmaf(lifted<BITS>(word[i / N][k], n), lowered<BITS>(f.x, n), f.y);
            }
        } else {
            const float2 f = meta_f2(__ldg(v_meta_row(p, t.pg, t.h, slot) + gi));
            const float scale = lowered<BITS>(f.x, n);
#pragma unroll
            for (int k = 0; k < 8; ++k) c[k] = fmaf(lifted<BITS>(word[i / N][k], n), scale, f.y);
        }
        store8(a, KEYS ? a.k_out : a.v_out, r.at + slot * r.step, c);
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads) read_back_kernel(Params p, ReadBackArgs a) {
    Tile t;
    t.b = blockIdx.y;
    // keys and values of all heads of a page side by side: their rows lie side by side in the output
    const unsigned part = blockIdx.x % (2 * p.hkv), tile = blockIdx.x / (2 * p.hkv);
    t.h = part >> 1;
    const bool keys = !(part & 1);
    const int r0 = __ldg(a.cu_rows + t.b), n = __ldg(a.cu_rows + t.b + 1) - r0;
    if (n <= 0 || n > a.max_rows) return;
    // positions in 64 bits until they are known to be near the cache
    const long long first = __ldg(a.first + t.b);
    const long long x0 = ((first >> 6) + tile) * kPage;
    if (x0 >= first + n) return;
    const int L = max(0, __ldg(a.lens + t.b)), Lq = sink::paged_len(p, a.kpc, L);
    // wanted slots of this tile, and those of them that live in the page
    const int lo = int(max(first - x0, 0ll)), hi = int(min(first + n - x0, (long long)kPage));
    const bool near = x0 >= 0 && x0 < L;
    t.x0 = near ? int(x0) : 0;
    t.pg = near && t.x0 < Lq ? phys_page(p, t.b, t.x0 / kPage) : -1;
    t.lo = lo;
    t.hi = t.pg >= 0 ? min(hi, Lq - t.x0) : 0;
    Rows<D> r;
    r.oct = threadIdx.x % Rows<D>::kOct;
    r.group = threadIdx.x / Rows<D>::kOct;
    r.step = size_t(p.hkv) * D;
    r.at = (size_t((long long)r0 + x0 - first) * p.hkv + t.h) * D + r.oct * 8;   // (wraps before the first row: lo > 0 then)
    if (t.hi > t.lo) {
        if (!keys) {
            if (p.vb == 1) channel_runs<1, D, false>(p, a, t, r);
            if (p.vb == 2) channel_runs<2, D, false>(p, a, t, r);
            if (p.vb == 4) channel_runs<4, D, false>(p, a, t, r);
            if (p.vb == 8) channel_runs<8, D, false>(p, a, t, r);
        } else if (a.kpc) {
            if (p.kb == 1) channel_runs<1, D, true>(p, a, t, r);
            if (p.kb == 2) channel_runs<2, D, true>(p, a, t, r);
            if (p.kb == 4) channel_runs<4, D, true>(p, a, t, r);
            if (p.kb == 8) channel_runs<8, D, true>(p, a, t, r);
        } else {
            if (p.kb == 1) token_rows<1, D>(p, a, t, r);
            if (p.kb == 2) token_rows<2, D>(p, a, t, r);
            if (p.kb == 4) token_rows<4, D>(p, a, t, r);
            if (p.kb == 8) token_rows<8, D>(p, a, t, r);
        }
    }
    // ring rows, and zeros for positions that are not there
    const int R = sink::ring_slots(p, a.kpc);
    void* out = keys ? a.k_out : a.v_out;
    for (int slot = max(t.hi, t.lo) + r.group; slot < hi; slot += Rows<D>::kGroups) {
        const long long x = x0 + slot;
        float c[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (x >= Lq && x < L) {
            const uint4 w = __ldg(reinterpret_cast<const uint4*>(
                (keys ? p.k_win : p.v_win) + ((size_t(t.b) * p.hkv + t.h) * R + int(x) % R) * D + r.oct * 8));
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                c[2 * i] = __uint_as_float(u[i] << 16);
                c[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
            }
        }
        store8(a, out, r.at + slot * r.step, c);
    }
}

}  // namespace

cudaError_t launch_read_back(const Params& p, const ReadBackArgs& a, cudaStream_t s) {
    // a run of max_rows positions touches at most this many pages
    const dim3 grid((a.max_rows + 2 * (kPage - 1)) / kPage * 2 * p.hkv, p.batch);
    if (p.d == 128)
        read_back_kernel<128><<<grid, kThreads, 0, s>>>(p, a);
    else
        read_back_kernel<64><<<grid, kThreads, 0, s>>>(p, a);
    return cudaGetLastError();
}

}  // namespace kvq
