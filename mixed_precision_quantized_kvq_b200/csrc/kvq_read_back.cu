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
// word of eight channels each, for D/16 neighbouring positions.  Measured on a
// B200: 88 us for 4096 rows of 16 sequences and 8 heads in bf16 (336 MB, 3.8
// TB/s, 58% of the copy rate).  Issue slots (about 70 for the reconstruction of
// a warp's 256 channels) are 42% busy: what is left above the bytes is a CTA's
// chain of loads (rows, first position, length, page number, codes).  Keys and
// values of a page in one CTA took 96.
#include "kvq_sink.cuh"

namespace kvq {
namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
}

template <typename Out>
__device__ __forceinline__ void store8(Out* o, const float (&x)[8]) {
    if (sizeof(Out) == 2) {
        *reinterpret_cast<uint4*>(o) =
            make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
    } else {
        reinterpret_cast<float4*>(o)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4*>(o)[1] = make_float4(x[4], x[5], x[6], x[7]);
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

// Code n of a word as an fp32 number plus 2^23, times 2^position(n): one mask puts it into the mantissa.  Taking 2^23 off
// is exact (integer conversions run at a quarter of the rate, shifts compete with the masks), the power of two goes into
// the scale, also exactly; then one fp32 fma, as in the definition.
template <int BITS>
__device__ __forceinline__ constexpr int position(int n) { return n * BITS % 16; }
template <int BITS>
__device__ __forceinline__ uint32_t lifted(uint32_t w, int n) {
    const int at = position<BITS>(n);
    return ((w >> (n * BITS - at)) & (((1u << BITS) - 1u) << at)) | 0x4b000000u;
}
template <int BITS>
__device__ __forceinline__ float lowered(float scale, int n) { return scale * (1.f / float(1 << position<BITS>(n))); }
// two lifted codes with their scales and zero points
__device__ __forceinline__ void reconstruct2(uint32_t a, uint32_t b, float s0, float s1, float z0, float z1, float& x, float& y) {
    asm("{\n\t.reg .b64 v, m, s, z;\n\t"
        "mov.b64 v, {%2, %3};\n\tmov.b64 m, {%8, %8};\n\tadd.rn.f32x2 v, v, m;\n\t"
        "mov.b64 s, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\tfma.rn.f32x2 v, v, s, z;\n\t"
        "mov.b64 {%0, %1}, v;\n\t}"
        : "=f"(x), "=f"(y)
        : "r"(a), "r"(b), "f"(s0), "f"(s1), "f"(z0), "f"(z1), "r"(0xcb000000u));
}

struct Tile {
    int b, h, pg;              // pg: physical page, -1 when absent
    int x0;                    // position of slot 0
    int lo, hi;                // slots wanted that live in the page: [lo, hi)
};

// A tile's output for this thread's channels: slot 0's place and the elements between slots.
template <int D, typename Out>
struct Rows {
    static constexpr int kOct = D / 8, kGroups = kThreads / kOct;   // threads of a row, rows at a time
    int oct, group;
    Out* at;
    size_t step;
};

// keys with groups along channels: eight codes of a position in one load.  ALL: every slot is wanted.
template <int BITS, bool ALL, int D, typename Out>
__device__ __forceinline__ void token_rows(const Params& p, const Tile& t, const Rows<D, Out>& r) {
    constexpr int G = Rows<D, Out>::kGroups;
    const int byte = r.oct * BITS;
    const uint8_t* codes = k_block(p, t.pg, t.h) + (byte / p.kch) * (kPage * p.kch) + byte % p.kch + r.group * p.kch;
    const uint32_t* meta = k_meta_row(p, t.pg, t.h, r.group) + (r.oct * 8 >> (__ffs(p.kg) - 1));
    Out* out = r.at + r.group * r.step;
#pragma unroll 4
    for (int slot = r.group; slot < kPage; slot += G, codes += G * p.kch, meta += G * p.nkg, out += G * r.step) {
        const bool have = ALL || (slot >= t.lo && slot < t.hi);
        // the lanes of one row take the same way
        const unsigned lanes = p.rotate ? __ballot_sync(0xffffffffu, have) : 0u;
        if (!have) continue;
        uint32_t w[2];
        if (BITS == 8) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(codes));
            w[0] = v.x, w[1] = v.y;
        }
        if (BITS == 4) w[0] = __ldg(reinterpret_cast<const uint32_t*>(codes));
        if (BITS == 2) w[0] = __ldg(reinterpret_cast<const uint16_t*>(codes));
        if (BITS == 1) w[0] = __ldg(codes);
        const float2 f = meta_f2(__ldg(meta));
        float c[8];
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
            const int n = BITS == 8 ? k % 4 : k;
            const uint32_t v = w[BITS == 8 ? k / 4 : 0];
            reconstruct2(lifted<BITS>(v, n), lifted<BITS>(v, n + 1), lowered<BITS>(f.x, n), lowered<BITS>(f.x, n + 1), f.y, f.y,
                         c[k], c[k + 1]);
        }
        if (p.rotate) rotate_back<D>(c, p.signs, r.oct, lanes);
        store8(out, c);
    }
}

// channel runs: D/16 neighbouring positions of eight channels
template <int BITS, bool KEYS, bool ALL, int D, typename Out>
__device__ __forceinline__ void channel_runs(const Params& p, const Tile& t, const Rows<D, Out>& r) {
    constexpr int N = 32 / BITS, RUN = kPage * BITS / 8, CH = RUN < 16 ? RUN : 16, T = kPage / Rows<D, Out>::kGroups;
    constexpr int WORDS = (T + N - 1) / N;               // words a channel
    const int s0 = r.group * T;
    if (!ALL && (s0 >= t.hi || s0 + T <= t.lo)) return;
    const uint8_t* blk = (KEYS ? p.k_codes : p.v_codes) + (size_t(t.pg) * p.hkv + t.h) * size_t(D) * RUN + r.oct * (8 * CH);
    uint32_t word[WORDS][8];
#pragma unroll
    for (int w = 0; w < WORDS; ++w) {
        const int byte = (s0 / N + w) * 4;
        const uint8_t* at = blk + (byte / CH) * (D * CH) + byte % CH;
#pragma unroll
        for (int k = 0; k < 8; ++k) word[w][k] = __ldg(reinterpret_cast<const uint32_t*>(at + k * CH)) >> (s0 % N * BITS);
    }
    const int kshift = __ffs(p.kg) - 1;
    const uint32_t* vmeta = v_meta_row(p, t.pg, t.h, s0) + (r.oct * 8 >> (__ffs(p.vg) - 1));
    const uint32_t* kmeta = p.k_meta + (size_t(t.pg) * p.hkv + t.h) * (kPage >> kshift) * D + r.oct * 8;
    Out* out = r.at + s0 * r.step;
#pragma unroll
    for (int i = 0; i < T; ++i, out += r.step) {
        const int slot = s0 + i, n = i % N;
        if (!ALL && (slot < t.lo || slot >= t.hi)) continue;
        const uint32_t(&w)[8] = word[i / N];
        float c[8];
        if (KEYS) {
            const uint4* m = reinterpret_cast<const uint4*>(kmeta + (slot >> kshift) * D);
            const uint4 m0 = __ldg(m), m1 = __ldg(m + 1);
            const uint32_t mm[8] = {m0.x, m0.y, m0.z, m0.w, m1.x, m1.y, m1.z, m1.w};
#pragma unroll
            for (int k = 0; k < 8; k += 2) {
                const float2 f = meta_f2(mm[k]), g = meta_f2(mm[k + 1]);
                reconstruct2(lifted<BITS>(w[k], n), lifted<BITS>(w[k + 1], n), lowered<BITS>(f.x, n), lowered<BITS>(g.x, n), f.y,
                             g.y, c[k], c[k + 1]);
            }
        } else {
            const float2 f = meta_f2(__ldg(vmeta + i * p.nvg));
            const float scale = lowered<BITS>(f.x, n);
#pragma unroll
            for (int k = 0; k < 8; k += 2)
                reconstruct2(lifted<BITS>(w[k], n), lifted<BITS>(w[k + 1], n), scale, scale, f.y, f.y, c[k], c[k + 1]);
        }
        store8(out, c);
    }
}

template <bool ALL, int D, typename Out>
__device__ __forceinline__ void page_rows(const Params& p, const Tile& t, const Rows<D, Out>& r, bool keys, bool kpc) {
    const int bits = keys ? p.kb : p.vb;
    if (!keys) {
        if (bits == 1) channel_runs<1, false, ALL>(p, t, r);
        if (bits == 2) channel_runs<2, false, ALL>(p, t, r);
        if (bits == 4) channel_runs<4, false, ALL>(p, t, r);
        if (bits == 8) channel_runs<8, false, ALL>(p, t, r);
    } else if (kpc) {
        if (bits == 1) channel_runs<1, true, ALL>(p, t, r);
        if (bits == 2) channel_runs<2, true, ALL>(p, t, r);
        if (bits == 4) channel_runs<4, true, ALL>(p, t, r);
        if (bits == 8) channel_runs<8, true, ALL>(p, t, r);
    } else {
        if (bits == 1) token_rows<1, ALL>(p, t, r);
        if (bits == 2) token_rows<2, ALL>(p, t, r);
        if (bits == 4) token_rows<4, ALL>(p, t, r);
        if (bits == 8) token_rows<8, ALL>(p, t, r);
    }
}

template <int D, typename Out>
__global__ void __launch_bounds__(kThreads) read_back_kernel(Params p, ReadBackArgs a) {
    Tile t;
    t.b = blockIdx.z;
    // keys and values of all heads of a page side by side: their rows lie side by side in the output
    t.h = blockIdx.x >> 1;
    const bool keys = !(blockIdx.x & 1);
    const int r0 = __ldg(a.cu_rows + t.b), n = __ldg(a.cu_rows + t.b + 1) - r0;
    if (n <= 0 || n > a.max_rows) return;
    // positions in 64 bits until they are known to be near the cache
    const long long first = __ldg(a.first + t.b);
    const long long x0 = ((first >> 6) + blockIdx.y) * kPage;
    if (x0 >= first + n) return;
    const int L = max(0, __ldg(a.lens + t.b)), Lq = sink::paged_len(p, a.kpc, L);
    // wanted slots of this tile, and those of them that live in the page
    const int lo = int(max(first - x0, 0ll)), hi = int(min(first + n - x0, (long long)kPage));
    const bool near = x0 >= 0 && x0 < L;
    t.x0 = near ? int(x0) : 0;
    t.pg = near && t.x0 < Lq ? phys_page(p, t.b, t.x0 / kPage) : -1;
    t.lo = lo;
    t.hi = t.pg >= 0 ? min(hi, Lq - t.x0) : 0;
    Rows<D, Out> r;
    r.oct = threadIdx.x % r.kOct;
    r.group = threadIdx.x / r.kOct;
    r.step = size_t(p.hkv) * D;
    // (slot 0 may lie before the first row; no slot below lo is touched)
    r.at = static_cast<Out*>(keys ? a.k_out : a.v_out) + ((long long)r0 + x0 - first) * (long long)r.step + t.h * D + r.oct * 8;
    if (t.hi > t.lo) {
        if (t.lo == 0 && t.hi == kPage)
            page_rows<true>(p, t, r, keys, a.kpc);
        else
            page_rows<false>(p, t, r, keys, a.kpc);
    }
    // ring rows, and zeros for positions that are not there
    const int R = sink::ring_slots(p, a.kpc);
    for (int slot = max(t.hi, t.lo) + r.group; slot < hi; slot += r.kGroups) {
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
        store8(r.at + slot * r.step, c);
    }
}

}  // namespace

cudaError_t launch_read_back(const Params& p, const ReadBackArgs& a, cudaStream_t s) {
    // a run of max_rows positions touches at most this many pages
    const dim3 grid(2 * p.hkv, (a.max_rows + 2 * (kPage - 1)) / kPage, p.batch);
    if (p.d == 128) {
        if (a.out_bf16)
            read_back_kernel<128, __nv_bfloat16><<<grid, kThreads, 0, s>>>(p, a);
        else
            read_back_kernel<128, float><<<grid, kThreads, 0, s>>>(p, a);
    } else {
        if (a.out_bf16)
            read_back_kernel<64, __nv_bfloat16><<<grid, kThreads, 0, s>>>(p, a);
        else
            read_back_kernel<64, float><<<grid, kThreads, 0, s>>>(p, a);
    }
    return cudaGetLastError();
}

}  // namespace kvq
