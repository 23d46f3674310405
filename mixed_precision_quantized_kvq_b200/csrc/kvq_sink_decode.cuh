// Single-token attention with sinks and a sliding span over the quantized
// cache (kvq_sink_decode_attention), for key groups of 32, 64 or 128 channels.
//
// With x^ = c*scale + zero per group of channels,
//     q . k^ = sum_u scale_u (q . c)_u + zero_u (sum q)_u     (u: 32 channels)
//     o_j    = sum_t (p_t vscale_t) c_tj + sum_t p_t vzero_t
// so the tensor cores take the codes as they lie in memory: a code of at most
// 8 bits, masked out of its word where it sits within the low ten bits of a
// half-word, IS an fp16 number, c * 2^(position - 24) (a subnormal one, exact).
// The power of two of its position is divided out of the other operand, 2^24
// out of the result.  One mask per two codes is all the unpacking there is,
// after a rotation of key words that puts 1- and 2-bit codes (and, where the
// query has a low part, 4-bit ones) high among the ten bits: sums are
// aligned to the exponents that the operands' fields name, so each zero above a
// subnormal's first bit costs them a bit (1-bit codes at bits 0 to 3: scores off
// by up to 2^-17 of sum |q k|, at bits 6 to 9 by 2^-22).
//
// What bounds it: latency.  It has to read the codes and metadata of the
// visible positions (116 bytes per position and kv-head for 4-bit keys and
// 2-bit values) and to issue about 1100 instructions a warp for 64 of them, and
// at the size below the two take about as long.  Hence the products on
// mma.sync.m16n8k16 with the positions
// (scores) or channels (values) as its 16 rows and the up to 8 query heads of
// a kv-head as its 8 columns: fragments are registers, the codes never go
// through shared memory a second time.  Measured on a B200: 28.8 us for 16
// sequences of 32 query and 8 kv-heads over 4096 positions (67.6 MB, 10.3 us at
// the copy rate): 12.5 whatever the span (dependent loads of length, page table
// and codes, first fetch of the instructions, the ring, the join) and 4.05 for
// each 1024 positions, 56% of the copy rate, up to a span of 16384.  Issue slots
// are 48% busy and DRAM 29%: 16 warps with a stage each for keys and for values do not
// cover the latency of a page.  Rotated keys and fp32 queries add a low part
// of the query, whose fragments make the head_dim-128 builds spill (76 to 124
// bytes a thread at 128 registers).
//
// Work split: one cluster of 1 to 16 CTAs per (sequence, kv-head); its warps
// take the 64-position pages in turn (warp w of W: pages w, w + W, ...), then
// 16-slot pieces of the bf16 ring, each with its own buffers for keys and
// values filled by cp.async (one stage each: with two stages of both, 12 warps
// fit an SM instead of 16 and 64 ragged sequences took 69 us instead of 48).
// The warps' partial sums meet in shared memory, across the cluster through
// distributed shared memory: no workspace, no atomics, the same result on every
// run.
//
// Fragment layouts (lane = 4*r + c): A rows r and r+8, B column r, D columns
// 2c and 2c+1.  A tile's scores come out as (position r, heads 2c, 2c+1);
// movmatrix turns the weights into the (positions, head r) fragments that the
// product with the values needs.  Which position sits in which row is chosen
// (row_position) so that the two weights of a register belong to the two codes
// that one mask takes out of a value word.
#pragma once

#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>

#include "kvq_sink.cuh"
#include "kvq_tc_ptx.cuh"

#include "kvq_mma_ptx.cuh"

namespace kvq {
namespace sink {

using namespace ptx;

constexpr int kMaxWarps = 16;        // what the registers of an SM hold, in one CTA or several
constexpr int kHeads = 8;            // columns of the products
constexpr int kRing = 16;            // ring slots per piece
constexpr float kRefNone = -1e30f;   // reference exponent before any position
constexpr float kCode = 16777216.f;  // 2^24: codes are fp16 numbers c * 2^-24
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_k8(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(b0));
}
// mma_bf16 without volatile, as the two above, so that the compiler may move loads and masks across it
__device__ __forceinline__ void mma_b16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void cp8(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// the kernels' view of shared memory: byte pointers
__device__ __forceinline__ uint32_t lds32(const unsigned char* a) { return *reinterpret_cast<const uint32_t*>(a); }
__device__ __forceinline__ uint2 lds64(const unsigned char* a) { return *reinterpret_cast<const uint2*>(a); }
__device__ __forceinline__ uint4 lds128(const unsigned char* a) { return *reinterpret_cast<const uint4*>(a); }
__device__ __forceinline__ void sts32(unsigned char* a, uint32_t v) { *reinterpret_cast<uint32_t*>(a) = v; }
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
    __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t bf162_bits(float lo, float hi) {
    __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    __half2 h = __hmul2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ float low_half(uint32_t w) { return __low2float(*reinterpret_cast<__half2*>(&w)); }

// Position of row x of the T-th eight rows of a page's scores.  Rows 2c and 2c + 1 are the positions of code pair T of
// the value words that lane column c holds (word c of a run's 16 bytes; half of word c >> 1 for 1-bit values): the
// weights of a pair then sit in one register after the transposition, and one mask takes the two codes out.
template <int VB>
__device__ __forceinline__ int row_position(int T, int x) {
    if (VB == 8) return 16 * (T >> 1) + 2 * x + (T & 1);
    if (VB == 4) return 32 * (T >> 2) + 4 * x + (T & 3);
    if (VB == 2) return 8 * x + T;
    return 32 * (x >> 2) + 8 * ((x >> 1) & 1) + 16 * (x & 1) + T;
}
// The bit at which pair T sits in its word (1-bit and the upper 2-bit pairs: after a shift) is value_bit.
// A lane column's 16 positions as four runs of four (the first position of run i), and where the words of pair T are
// among the 16 (the second kPairWords further).
template <int VB>
__device__ __forceinline__ int value_run(int c, int i) {
    if (VB == 8) return 16 * i + 4 * c;
    if (VB == 4) return 32 * (i >> 1) + 8 * c + 4 * (i & 1);
    if (VB == 2) return 16 * c + 4 * i;
    return 32 * (c >> 1) + 8 * (c & 1) + 16 * (i >> 1) + 4 * (i & 1);
}
template <int VB>
__device__ __forceinline__ constexpr int pair_word(int T) {
    return VB == 8 ? 4 * (T >> 1) + (T & 1) : VB == 4 ? 8 * (T >> 2) + (T & 3) : T;
}
template <int VB>
constexpr int kPairWords = VB == 8 ? 2 : VB == 4 ? 4 : 8;
template <int VB>
__device__ __forceinline__ constexpr int value_bit(int T) {
    return VB == 8 ? 0 : VB == 4 ? 4 * (T & 1) : VB == 2 ? (T < 5 ? 2 * T : 2 * T - 10) : T;
}
// Key rows and their metadata are stored with their 16-byte pieces exchanged within each 128 bytes, so that the eight
// positions of a score tile, whichever they are, lie in different banks.
__device__ __forceinline__ int key_slot(int t) { return t ^ ((t >> 3) & 7); }

// channels of code pair i (0..3) of lane column c within 32 channels, and the bit position of the pair
template <int KB>
__device__ __forceinline__ int pair_channel(int c, int i, int hi) {
    if (KB == 8) return (i >> 1) * 16 + 4 * c + (i & 1) + 2 * hi;
    if (KB == 4) return 8 * c + i + 4 * hi;
    if (KB == 2) return 16 * (c >> 1) + 4 * (c & 1) + i + 8 * hi;
    return 4 * c + i + 16 * hi;
}
template <int KB, bool LO>
__device__ __forceinline__ constexpr int pair_bit(int i) {
    return KB == 4 ? 4 * (i & 1) + (LO ? 2 : 0) : KB == 2 ? (LO ? 6 + 2 * (i & 1) : 2 + 2 * i) : KB == 1 ? 6 + i : 0;
}

// Shared memory of a CTA: what the query fragments are made of, then the
// warps' buffers; the partial sums take the buffers' place at the end.
template <int D, bool LO>
struct Head {
    __half qh[kHeads][D];                    // query, scaled to at most 2^8 per head, high and low part
    __half ql[kHeads][D];
    __nv_bfloat16 bq[LO ? 3 : 1][kHeads][D + 8];   // unrotated query for the ring: high part and, of fp32 queries, two low ones
    float qsum[kHeads][4];                   // sums over 32 channels
    float factor[kHeads];                    // score scale * log2(e) / query scaling
};

// A warp's buffers: keys (codes and metadata, or 16 ring rows) and values.  While the values are worked on, the next
// keys come in, and the other way round.
template <int D, int KB, int VB>
struct Buf {
    static constexpr int kK = kPage * D * KB / 8, kV = kPage * D * VB / 8, kRows = kRing * 2 * D;
    static constexpr int kUnits = D / 32;      // key metadata is kept for every 32 channels, value metadata by groups
    static constexpr int keys() { return max_of(kK + kPage * 4 * kUnits, kRows); }
    __host__ __device__ static int values(const Params& p) { return max_of(kV + kPage * 4 * p.nvg, kRows); }
    __host__ __device__ static constexpr int max_of(int a, int b) { return a > b ? a : b; }
};

// partial sums of a warp: [head][D] values, then reference exponents and sums of the weights
template <int D>
constexpr int kPartFloats = kHeads * D + 2 * kHeads;

// bytes of a warp's part of shared memory, and of a CTA's
template <int D, int KB, int VB>
__host__ __device__ int warp_smem(const Params& p) {
    const int both = Buf<D, KB, VB>::keys() + Buf<D, KB, VB>::values(p), part = kPartFloats<D> * 4;
    return both > part ? both : part;
}
template <int D, int KB, int VB, bool LO>
__host__ __device__ int decode_smem(const Params& p, int warps) {
    return int(sizeof(Head<D, LO>)) + warps * warp_smem<D, KB, VB>(p);
}

// The running state of a warp: fragments of the output (channels 16*i + r, 16*i + r + 8 of heads 2c, 2c+1; scaled by
// 2^-24), the zero points' share (value group r), weights' sums and reference exponents of the two heads.
template <int D>
struct Sums {
    float acc[D / 16][4];
    float zero[4];
    float l[2], ref[2];
};

template <int D>
__device__ __forceinline__ void raise_ref(Sums<D>& S, const float (&top)[2], int log_scale) {
    // Weights are 2^(score - ref), at most 2^15, and so are their products with the value scales (below
    // 2^log_scale): both round to fp16 without overflow, by up to 2^-11 of themselves.  After a rise the largest weight is
    // 2^(11 - log_scale), so half a step of the smallest fp16 numbers, 2^-25, is 2^(log_scale - 36) of it: that much of
    // a weight, and of a product times its code and 2^value_bit (divided out of it, a rounding of its own), may be lost.
    // log_scale is the largest over a page's groups: one group of large scales takes range from the others.
    const float need0 = top[0] - 15.f + float(log_scale), need1 = top[1] - 15.f + float(log_scale);
    if (__any_sync(kAll, need0 > S.ref[0] || need1 > S.ref[1])) {
        // four binades of room, so that the next rise seldom comes soon
        const float r0 = need0 > S.ref[0] ? need0 + 4.f : S.ref[0], r1 = need1 > S.ref[1] ? need1 + 4.f : S.ref[1];
        const float f0 = ex2(S.ref[0] - r0), f1 = ex2(S.ref[1] - r1);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            S.acc[i][0] *= f0;
            S.acc[i][1] *= f1;
            S.acc[i][2] *= f0;
            S.acc[i][3] *= f1;
        }
        S.zero[0] *= f0;
        S.zero[1] *= f1;
        S.l[0] *= f0;
        S.l[1] *= f1;
        S.ref[0] = r0;
        S.ref[1] = r1;
    }
}

__device__ __forceinline__ float max_rows(float x) {
    x = fmaxf(x, __shfl_xor_sync(kAll, x, 4));
    x = fmaxf(x, __shfl_xor_sync(kAll, x, 8));
    return fmaxf(x, __shfl_xor_sync(kAll, x, 16));
}
__device__ __forceinline__ float sum_rows(float x) {
    x += __shfl_xor_sync(kAll, x, 4);
    x += __shfl_xor_sync(kAll, x, 8);
    return x + __shfl_xor_sync(kAll, x, 16);
}

// visible to the query: position x below `limit` of the part it lives in
__device__ __forceinline__ bool visible(int x, int ns, int lo, int limit) { return x < limit && (x < ns || x >= lo); }

// Scores of one 64-position page whose keys are at `sk` (base = position of slot 0), to be multiplied by the head's
// factor: s[T][e] is position row_position(T, r), head 2c + e.
template <int D, int KB, int VB, bool LO>
__device__ __forceinline__ void page_scores(const Params& p, unsigned char* sk, int base, int ns, int lo, int Lq, bool edge,
                                            const uint32_t (&qh)[D / 8], const uint32_t (&ql)[LO ? D / 8 : 1], uint32_t qz,
                                            float (&s)[8][2]) {
    constexpr int NU = D / 32;
    const int lane = threadIdx.x % 32, r = lane >> 2, c = lane & 3;
    unsigned char* skm = sk + Buf<D, KB, VB>::kK;
    const auto meta = [&](int t) { return skm + key_slot(t) * (NU * 4); };
    if (edge) {   // positions that are not visible: finite scores (masked below)
        for (int t = lane; t < kPage; t += 32)
            if (!visible(base + t, ns, lo, Lq))
                for (int i = 0; i < NU; ++i) sts32(meta(t) + i * 4, 0);
        __syncwarp();
    }
#pragma unroll
    for (int b = 0; b < 4; ++b) {                       // 16 positions: rows r and r + 8
        const int t0 = row_position<VB>(2 * b, r), t1 = row_position<VB>(2 * b + 1, r);
        uint32_t m0[4], m1[4];                          // metadata of the 32-channel units
        if (NU == 4) {
            const uint4 x = lds128(meta(t0)), y = lds128(meta(t1));
            m0[0] = x.x, m0[1] = x.y, m0[2] = x.z, m0[3] = x.w;
            m1[0] = y.x, m1[1] = y.y, m1[2] = y.z, m1[3] = y.w;
        } else {
            const uint2 x = lds64(meta(t0)), y = lds64(meta(t1));
            m0[0] = x.x, m0[1] = x.y, m1[0] = y.x, m1[1] = y.y;
        }
        // zero points of units 2(c & 1), 2(c & 1) + 1 against the unit sums (high parts at c < 2, low at c >= 2)
        float z[4] = {0.f, 0.f, 0.f, 0.f};
        const bool odd = c & 1;
        if (NU == 4)
            mma_f16_k8(z, __byte_perm(odd ? m0[2] : m0[0], odd ? m0[NU - 1] : m0[1], 0x7632),
                       __byte_perm(odd ? m1[2] : m1[0], odd ? m1[NU - 1] : m1[1], 0x7632), qz);
        else
            mma_f16_k8(z, odd ? 0u : __byte_perm(m0[0], m0[1], 0x7632), odd ? 0u : __byte_perm(m1[0], m1[1], 0x7632), qz);
        float a[4] = {0.f, 0.f, 0.f, 0.f};
        const unsigned char *k0 = sk + key_slot(t0) * (KB == 1 ? D / 8 : 16), *k1 = sk + key_slot(t1) * (KB == 1 ? D / 8 : 16);
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            uint32_t e[4], f[4];                        // code pairs of rows r and r + 8
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const unsigned char* k = h ? k1 : k0;
                uint32_t(&x)[4] = h ? f : e;
                if (KB == 8) {
                    const uint32_t w0 = lds32(k + (2 * u) * (kPage * 16) + c * 4);
                    const uint32_t w1 = lds32(k + (2 * u + 1) * (kPage * 16) + c * 4);
                    x[0] = w0 & 0x00ff00ffu;
                    x[1] = (w0 >> 8) & 0x00ff00ffu;
                    x[2] = w1 & 0x00ff00ffu;
                    x[3] = (w1 >> 8) & 0x00ff00ffu;
                } else if (KB == 4) {
                    constexpr int kUp = pair_bit<KB, LO>(0);
                    const uint32_t word = lds32(k + u * (kPage * 16) + c * 4), w = word << kUp, v = word >> (8 - kUp);
                    x[0] = w & (0x000f000fu << kUp);
                    x[1] = w & (0x00f000f0u << kUp);
                    x[2] = v & (0x000f000fu << kUp);
                    x[3] = v & (0x00f000f0u << kUp);
                } else if (KB == 2) {
                    const uint32_t word = lds32(k + (u >> 1) * (kPage * 16) + (2 * (u & 1) + (c >> 1)) * 4);
                    const uint32_t v = __funnelshift_l(word, word, 2 - 8 * (c & 1));
                    const uint32_t w = LO ? __funnelshift_l(word, word, 6 - 8 * (c & 1)) : v;
                    x[0] = w & (0x00030003u << pair_bit<KB, LO>(0));
                    x[1] = w & (0x00030003u << pair_bit<KB, LO>(1));
                    x[2] = v & (0x00030003u << pair_bit<KB, LO>(2));
                    x[3] = v & (0x00030003u << pair_bit<KB, LO>(3));
                } else {
                    const uint32_t word = lds32(k + u * 4), w = __funnelshift_l(word, word, 6 - 4 * c);
                    x[0] = w & 0x00400040u;
                    x[1] = w & 0x00800080u;
                    x[2] = w & 0x01000100u;
                    x[3] = w & 0x02000200u;
                }
            }
            float d[4] = {0.f, 0.f, 0.f, 0.f};
            if (LO) {   // first: its sums are small, and so is what the products cut off them
                mma_f16(d, e[0], f[0], e[1], f[1], ql[LO ? 4 * u : 0], ql[LO ? 4 * u + 1 : 0]);
                mma_f16(d, e[2], f[2], e[3], f[3], ql[LO ? 4 * u + 2 : 0], ql[LO ? 4 * u + 3 : 0]);
            }
            mma_f16(d, e[0], f[0], e[1], f[1], qh[4 * u], qh[4 * u + 1]);
            mma_f16(d, e[2], f[2], e[3], f[3], qh[4 * u + 2], qh[4 * u + 3]);
            const float s0 = low_half(m0[u]), s1 = low_half(m1[u]);
            a[0] = fmaf(s0, d[0], a[0]);
            a[1] = fmaf(s0, d[1], a[1]);
            a[2] = fmaf(s1, d[2], a[2]);
            a[3] = fmaf(s1, d[3], a[3]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) s[2 * b + (i >> 1)][i & 1] = fmaf(a[i], kCode, z[i]);
        if (edge) {
            if (!visible(base + t0, ns, lo, Lq)) s[2 * b][0] = s[2 * b][1] = -INFINITY;
            if (!visible(base + t1, ns, lo, Lq)) s[2 * b + 1][0] = s[2 * b + 1][1] = -INFINITY;
        }
    }
}

// The weights of the scores and the product with the values at `sv`.
template <int D, int KB, int VB>
__device__ __forceinline__ void page_values(const Params& p, unsigned char* sv, int base, int ns, int lo, int Lq, bool edge,
                                            const float (&s)[8][2], const float (&factor)[2], Sums<D>& S) {
    const int lane = threadIdx.x % 32, r = lane >> 2, c = lane & 3, nvg = p.nvg;
    unsigned char* svm = sv + Buf<D, KB, VB>::kV;
    const int vshift = __ffs(p.vg) - 1;
    if (edge) {   // no values at positions that are not visible
        for (int t = lane; t < kPage; t += 32)
            if (!visible(base + t, ns, lo, Lq))
                for (int i = 0; i < nvg; ++i) sts32(svm + (i * kPage + t) * 4, 0);
        __syncwarp();
    }
    float top[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        float x = s[0][e];
#pragma unroll
        for (int T = 1; T < 8; ++T) x = fmaxf(x, s[T][e]);
        top[e] = max_rows(x) * factor[e];                // factors are not negative
    }
    uint32_t vmax = 0;                                   // largest value scale, as its fp16 bits
    for (int i = lane; i < kPage * nvg; i += 32) vmax = max(vmax, lds32(svm + i * 4) & 0x7fffu);
    vmax = __reduce_max_sync(kAll, vmax);
    raise_ref(S, top, max(0, int(vmax >> 10) - 14));     // a scale is below 2^(exponent field - 14)
    // (l sums the weights before they are rounded: lse is fp32's, and an output keeps the roundings of its weights)
    uint32_t w[8];                                       // weights of pair T, head r
#pragma unroll
    for (int T = 0; T < 8; ++T) {
        const float p0 = ex2(fmaf(s[T][0], factor[0], -S.ref[0])), p1 = ex2(fmaf(s[T][1], factor[1], -S.ref[1]));
        S.l[0] += p0;
        S.l[1] += p1;
        w[T] = transpose8(half2_bits(p0, p1));
    }
    uint32_t Z[8], pv[8];
#pragma unroll
    for (int T = 0; T < 8; ++T) Z[T] = 0;
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt) {
        if ((16 * mt & (p.vg - 1)) == 0) {
            const int gi = 16 * mt >> vshift;
            // metadata of this lane's 16 positions, four neighbours a load
            uint32_t m[16];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 x = lds128(svm + gi * (kPage * 4) + value_run<VB>(c, i) * 4);
                m[4 * i] = x.x, m[4 * i + 1] = x.y, m[4 * i + 2] = x.z, m[4 * i + 3] = x.w;
            }
#pragma unroll
            for (int T = 0; T < 8; ++T) {
                const uint32_t x = m[pair_word<VB>(T)], y = m[pair_word<VB>(T) + kPairWords<VB>];
                pv[T] = hmul2(w[T], __byte_perm(x, y, 0x5410));
                if (value_bit<VB>(T))                    // the power of two of the codes' position
                    pv[T] = hmul2(pv[T], uint32_t(15 - value_bit<VB>(T)) * 0x04000400u);
                if (r == gi) Z[T] = __byte_perm(x, y, 0x7632);
            }
        }
        uint32_t e[8], f[8];                             // code pairs of channels 16*mt + r and + 8
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int ch = 16 * mt + 8 * h + r;
            uint32_t(&x)[8] = h ? f : e;
            if (VB == 8) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t v = lds32(sv + j * (D * 16) + ch * 16 + c * 4);
                    x[2 * j] = v & 0x00ff00ffu;
                    x[2 * j + 1] = (v >> 8) & 0x00ff00ffu;
                }
            } else if (VB == 4) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t v = lds32(sv + j * (D * 16) + ch * 16 + c * 4), u = v >> 8;
                    x[4 * j] = v & 0x000f000fu;
                    x[4 * j + 1] = v & 0x00f000f0u;
                    x[4 * j + 2] = u & 0x000f000fu;
                    x[4 * j + 3] = u & 0x00f000f0u;
                }
            } else if (VB == 2) {
                const uint32_t v = lds32(sv + ch * 16 + c * 4), u = v >> 10;
#pragma unroll
                for (int T = 0; T < 8; ++T) x[T] = (T < 5 ? v : u) & (0x00030003u << value_bit<VB>(T));
            } else {
                const uint32_t v = lds32(sv + ch * 8 + (c >> 1) * 4) >> (8 * (c & 1));
#pragma unroll
                for (int T = 0; T < 8; ++T) x[T] = v & (0x00010001u << T);
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_f16(S.acc[mt], e[2 * k], f[2 * k], e[2 * k + 1], f[2 * k + 1], pv[2 * k], pv[2 * k + 1]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) mma_f16(S.zero, Z[2 * k], 0, Z[2 * k + 1], 0, w[2 * k], w[2 * k + 1]);
}

// Where 16-byte piece o of ring row i lies: exchanged within the row so that the same piece of eight rows falls into
// different banks (values, by columns) and four neighbouring pieces of rows 2k, 2k+1 do (keys, by rows).
template <int D>
__device__ __forceinline__ int ring_piece(int i, int o) {
    return i * (2 * D) + ((o ^ (((i & 1) << 2) | ((i >> 1) & 3))) << 4);
}

// Scores of 16 ring slots whose keys are at `sk`: s[h][e] is slot 8h + r, head 2c + e.  ok: bit i set when slot i holds
// a visible position (other rows are zeros).
template <int D, bool LO>
__device__ __forceinline__ void ring_scores(const Head<D, LO>& hd, const unsigned char* sk, uint32_t ok, bool lo_part,
                                            float scale_log2, float (&out)[8][2]) {
    const int lane = threadIdx.x % 32, r = lane >> 2, c = lane & 3;
    // (the low parts' sums of their own: what a product cuts off its sum is as small as the sum)
    float s[4] = {0.f, 0.f, 0.f, 0.f}, low[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {                   // channels 32*j + 8*c .. + 7 in one 16-byte piece
        const uint4 k0 = lds128(sk + ring_piece<D>(r, 4 * j + c)), k1 = lds128(sk + ring_piece<D>(r + 8, 4 * j + c));
        const uint4 q = *reinterpret_cast<const uint4*>(&hd.bq[0][r][32 * j + 8 * c]);
        uint32_t a[4] = {k0.x, k1.x, k0.y, k1.y}, b[4] = {k0.z, k1.z, k0.w, k1.w};
        mma_b16(s, a, q.x, q.y);
        mma_b16(s, b, q.z, q.w);
        if (LO && lo_part) {
#pragma unroll
            for (int part = LO ? 2 : 0; part >= 1; --part) {
                const uint4 ql = *reinterpret_cast<const uint4*>(&hd.bq[part][r][32 * j + 8 * c]);
                mma_b16(low, a, ql.x, ql.y);
                mma_b16(low, b, ql.z, ql.w);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i >> 1][i & 1] = (ok >> (r + 8 * (i >> 1))) & 1u ? (s[i] + low[i]) * scale_log2 : -INFINITY;
}

template <int D>
__device__ __forceinline__ void ring_values(const unsigned char* sv, const float (&s)[8][2], Sums<D>& S) {
    const int lane = threadIdx.x % 32;
    const float top[2] = {max_rows(fmaxf(s[0][0], s[1][0])), max_rows(fmaxf(s[0][1], s[1][1]))};
    raise_ref(S, top, 0);
    // weights as bf16 high and low parts, in the output's unit of 2^-24
    uint32_t wh[2], wl[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float p0 = ex2(s[h][0] - S.ref[0]), p1 = ex2(s[h][1] - S.ref[1]);
        S.l[0] += p0;
        S.l[1] += p1;
        const float x = p0 * (1.f / kCode), y = p1 * (1.f / kCode);
        const uint32_t hi = bf162_bits(x, y);
        wh[h] = transpose8(hi);
        wl[h] = transpose8(bf162_bits(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xffff0000u)));
    }
    // matrix i of the load: positions 8*(i >> 1) .., channels 16*mt + 8*(i & 1) ..
    const int row = (lane & 7) + 8 * (lane >> 4), piece = (lane >> 3) & 1;
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt) {
        uint32_t a[4];
        ldsm_x4_t(a, smem_u32(sv) + ring_piece<D>(row, 2 * mt + piece));
        mma_b16(S.acc[mt], a, wh[0], wh[1]);
        mma_b16(S.acc[mt], a, wl[0], wl[1]);
    }
}

template <int D, int KB, int VB, bool LO>
__global__ void __launch_bounds__(kMaxWarps * 32) sink_decode_kernel(const __grid_constant__ Params p, const __grid_constant__ Args a) {
    using G = Buf<D, KB, VB>;
    extern __shared__ __align__(16) unsigned char smem[];
    Head<D, LO>& hd = *reinterpret_cast<Head<D, LO>*>(smem);
    const int warps = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int r = lane >> 2, c = lane & 3;
    const int h = blockIdx.y, b = blockIdx.z, rank = blockIdx.x, ctas = gridDim.x;
    const int region = warp_smem<D, KB, VB>(p);
    unsigned char* mine = smem + sizeof(Head<D, LO>) + warp * region;
    unsigned char *sk = mine, *sv = mine + G::keys();

    // A negative score scale becomes the query's sign, so that the largest score is the largest product.
    const float sign = a.scale_log2 < 0.f ? -1.f : 1.f, scale_log2 = fabsf(a.scale_log2);

    // query rows of heads `warp` and `warp + warps`: under way while the length and the page table are read
    constexpr int C = D / 32;
    float q[2][C];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        const int x = warp + y * warps;
        const size_t at = size_t(b) * a.q_stride + size_t(h * p.g + x) * D + lane * C;
#pragma unroll
        for (int i = 0; i < C; ++i)
            q[y][i] = x >= p.g ? 0.f
                      : sign * (a.q_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[at + i])
                                         : static_cast<const float*>(a.q)[at + i]);
    }

    const int L = max(0, min(__ldg(a.lens + b), a.len_cap));
    const int Lq = paged_len(p, 0, L);                    // positions below Lq live in pages, the others in the ring
    const int lo = span_begin(L - 1, a.span), ns = min(a.sinks, lo);
    // items: pages with sinks, pages of the span, ring pieces
    const int n_sink = (min(ns, Lq) + kPage - 1) / kPage;
    const int first = max(n_sink, lo / kPage);
    const int n_page = n_sink + (lo < Lq ? max(0, (Lq + kPage - 1) / kPage - first) : 0);
    const int n_item = n_page + (p.W > 0 ? (min(p.W, L) + kRing - 1) / kRing : 0);
    const int step = warps * ctas, start = rank * warps + warp;
    auto logical = [&](int it) { return it < n_sink ? it : it - n_sink + first; };

    // physical pages of this warp's next 32 items, one per lane
    int table = -1, table_at = 0;
    auto look_up = [&](int k0) {
        const int it = start + (k0 + lane) * step;
        table = it < n_page ? phys_page(p, b, logical(it)) : -1;
        table_at = k0;
    };
    look_up(0);

    // What item number k of this warp is: -1 nothing to do, a page's block below 2^30, or 2^30 + the valid ring slots.
    constexpr int kIsRing = 1 << 30;
    auto item = [&](int k) -> int {
        const int it = start + k * step;
        if (k - table_at >= 32) look_up(k);
        const int pg = __shfl_sync(kAll, table, k - table_at);
        if (it < n_page) return pg;
        if (it >= n_item) return -1;
        const int slot = (it - n_page) * kRing + (lane & (kRing - 1)), q0 = Lq % p.W;
        const int x = Lq + (slot >= q0 ? slot - q0 : slot - q0 + p.W);
        const unsigned any = __ballot_sync(kAll, slot < p.W && visible(x, ns, lo, L)) & 0xffffu;
        return any ? kIsRing + int(any) : -1;
    };
    auto copy_ring = [&](unsigned char* to, const __nv_bfloat16* rows, int k, int what) {
        const size_t row = (size_t(b) * p.hkv + h) * p.W + (start + k * step - n_page) * kRing;
        const uint32_t at = smem_u32(to);
        for (int e = lane; e < kRing * (D / 8); e += 32) {
            const int i = e / (D / 8), o = e % (D / 8);
            const bool have = (what >> i) & 1;
            cp16_zfill(at + ring_piece<D>(i, o), rows + (have ? (row + i) * D + o * 8 : 0), have);
        }
    };
    auto copy_keys = [&](int k, int what) {
        if (what >= kIsRing) {
            copy_ring(sk, p.k_win, k, what);
        } else if (what >= 0) {
            const uint32_t at = smem_u32(sk);
            const size_t blk = size_t(what) * p.hkv + h;
            const uint8_t* kc = p.k_codes + blk * G::kK + lane * 16;
            if (KB == 1) {                               // rows of D/8 bytes: 8-byte pieces keep the exchange for D = 64
#pragma unroll
                for (int t = 0; t < kPage; t += 32)
                    if (D == 128)
                        cp16(at + key_slot(lane + t) * 16, kc + t * 16);
                    else
                        cp8(at + key_slot(lane + t) * 8, kc - lane * 8 + t * 8);
            } else {
#pragma unroll
                for (int e = 0; e < G::kK / 16; e += 32)   // chunk e / 64, positions e % 64 + lane
                    cp16(at + ((e & ~63) + key_slot((e & 63) + lane)) * 16, kc + e * 16);
            }
            const uint32_t am = at + G::kK;
            const uint32_t* km = p.k_meta + blk * kPage * p.nkg;
            if (D == 128 && p.nkg == 4) {
#pragma unroll
                for (int t = lane; t < kPage; t += 32) cp16(am + key_slot(t) * 16, km + t * 4);
            } else {                                     // one word for every 32 channels
                const int sh = __ffs(G::kUnits / p.nkg) - 1;
                for (int e = lane; e < kPage * G::kUnits; e += 32) {
                    const int t = e / G::kUnits, u = e % G::kUnits;
                    cp4(am + (key_slot(t) * G::kUnits + u) * 4, km + t * p.nkg + (u >> sh));
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const int vlog = __ffs(p.nvg) - 1;
    auto copy_values = [&](int k, int what) {
        if (what >= kIsRing) {
            copy_ring(sv, p.v_win, k, what);
        } else if (what >= 0) {
            const uint32_t at = smem_u32(sv);
            const size_t blk = size_t(what) * p.hkv + h;
            const uint8_t* vc = p.v_codes + blk * G::kV + lane * 16;
#pragma unroll
            for (int e = 0; e < G::kV; e += 512) cp16(at + e + lane * 16, vc + e);
            const uint32_t* vm = p.v_meta + blk * kPage * p.nvg;
            if (p.nvg == 1) {
                if (lane < 16) cp16(at + G::kV + lane * 16, vm + lane * 4);
            } else {                                     // group-major
                for (int e = lane; e < kPage * p.nvg; e += 32) {
                    const int t = e >> vlog, g = e & (p.nvg - 1);
                    cp4(at + G::kV + (g * kPage + t) * 4, vm + e);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int now = item(0);
    copy_keys(0, now);
    copy_values(0, now);

    // ---- queries to shared memory, a head's row by one warp ----
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        const int x = warp + y * warps;
        if (x >= kHeads) break;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            float left = q[y][i];
#pragma unroll
            for (int part = 0; part < (LO ? 3 : 1); ++part) {
                const __nv_bfloat16 b = __float2bfloat16_rn(left);
                hd.bq[part][x][lane * C + i] = b;
                left -= __bfloat162float(b);
                if (a.q_bf16) break;                     // (exact already)
            }
        }
        if (p.rotate) rotate_warp<D>(q[y], p.signs, lane);
        float m = 0.f, sum = 0.f;
#pragma unroll
        for (int i = 0; i < C; ++i) m = fmaxf(m, fabsf(q[y][i]));
        m = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(m)));
        // a power of two that brings the head's largest element into [2^7, 2^8)
        const int ex = max(-100, int(__float_as_uint(m) >> 23) - 127);
        const float up = __uint_as_float(uint32_t(127 + 7 - ex) << 23);
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const float v = q[y][i] * up;
            const __half hi = __float2half_rn(v);
            hd.qh[x][lane * C + i] = hi;
            hd.ql[x][lane * C + i] = __float2half_rn(v - __half2float(hi));
            sum += v;
        }
#pragma unroll
        for (int w = 1; w < 32 / C; w <<= 1) sum += __shfl_xor_sync(kAll, sum, w);
        if (lane % (32 / C) == 0) hd.qsum[x][lane / (32 / C)] = sum;
        // (never zero: -inf times it has to stay -inf)
        if (lane == 0) hd.factor[x] = fmaxf(scale_log2 * __uint_as_float(uint32_t(127 - 7 + ex) << 23), 1e-37f);
    }
    __syncthreads();
    uint32_t qh[D / 8], ql[LO ? D / 8 : 1];
#pragma unroll
    for (int u = 0; u < D / 32; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c0 = 32 * u + pair_channel<KB>(c, i, 0), c1 = 32 * u + pair_channel<KB>(c, i, 1);
            const float down = 1.f / float(1 << pair_bit<KB, LO>(i));
            qh[4 * u + i] = half2_bits(__half2float(hd.qh[r][c0]) * down, __half2float(hd.qh[r][c1]) * down);
            if (LO) ql[LO ? 4 * u + i : 0] = half2_bits(__half2float(hd.ql[r][c0]) * down, __half2float(hd.ql[r][c1]) * down);
        }
    uint32_t qz;
    {
        const int u = 2 * (c & 1);
        const bool have = u < D / 32;
        const float s0 = have ? hd.qsum[r][u] : 0.f, s1 = have ? hd.qsum[r][u + 1] : 0.f;
        const float h0 = __half2float(__float2half_rn(s0)), h1 = __half2float(__float2half_rn(s1));
        qz = c < 2 ? half2_bits(h0, h1) : half2_bits(s0 - h0, s1 - h1);
    }
    const float factor[2] = {hd.factor[2 * c], hd.factor[2 * c + 1]};
    const bool ring_lo = !a.q_bf16;

    Sums<D> S;
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) S.acc[i][j] = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) S.zero[j] = 0.f;
    S.l[0] = S.l[1] = 0.f;
    S.ref[0] = S.ref[1] = kRefNone;

    for (int k = 0; start + k * step < n_item; ++k) {
        const int next = item(k + 1);
        const bool page = now >= 0 && now < kIsRing;
        const int base = page ? logical(start + k * step) * kPage : 0;
        const bool edge = base + kPage > Lq || (base < lo && base + kPage > ns);
        float s[8][2];
        asm volatile("cp.async.wait_group 1;" ::: "memory");   // the keys are here, the values may not be
        __syncwarp();
        if (page)
            page_scores<D, KB, VB, LO>(p, sk, base, ns, lo, Lq, edge, qh, ql, qz, s);
        else if (now >= kIsRing)
            ring_scores<D, LO>(hd, sk, uint32_t(now), ring_lo, scale_log2, s);
        __syncwarp();
        copy_keys(k + 1, next);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncwarp();
        if (page)
            page_values<D, KB, VB>(p, sv, base, ns, lo, Lq, edge, s, factor, S);
        else if (now >= kIsRing)
            ring_values<D>(sv, s, S);
        __syncwarp();
        copy_values(k + 1, next);
        now = next;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();

    // ---- this warp's sums to its part of shared memory (its buffers are free) ----
    float* part = reinterpret_cast<float*>(mine);
    S.l[0] = sum_rows(S.l[0]);
    S.l[1] = sum_rows(S.l[1]);
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt) {
        const int gi = 16 * mt >> (__ffs(p.vg) - 1);     // all 16 channels of a tile are in one group
        const float z0 = __shfl_sync(kAll, S.zero[0], 4 * gi + c), z1 = __shfl_sync(kAll, S.zero[1], 4 * gi + c);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            part[(2 * c + (i & 1)) * D + 16 * mt + 8 * (i >> 1) + r] = fmaf(S.acc[mt][i], kCode, (i & 1) ? z1 : z0);
    }
    if (r == 0) {
        part[kHeads * D + 2 * c] = S.ref[0];
        part[kHeads * D + 2 * c + 1] = S.ref[1];
        part[kHeads * D + kHeads + 2 * c] = S.l[0];
        part[kHeads * D + kHeads + 2 * c + 1] = S.l[1];
    }

    // ---- the CTA's sums: weights of its warps' parts, then one part for the CTA in place of warp 0's ----
    __syncthreads();
    const auto parts = [&](int w) { return reinterpret_cast<float*>(smem + sizeof(Head<D, LO>) + w * region); };
    float* weight = reinterpret_cast<float*>(&hd.qh[0][0]);   // [warp][head]; the queries are in registers by now
    if (warp < kHeads / 4) {
        const int x = 4 * warp + r % 4;                       // lanes of one head: c + 4 * (r / 4), warps in steps of 8
        float top = kRefNone, l = 0.f;
        const int w0 = c + 4 * (r >> 2);
        float ref[2], sum[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int w = w0 + 8 * i;
            ref[i] = w < warps ? parts(w)[kHeads * D + x] : kRefNone;
            sum[i] = w < warps ? parts(w)[kHeads * D + kHeads + x] : 0.f;
            top = fmaxf(top, ref[i]);
        }
        top = fmaxf(top, __shfl_xor_sync(kAll, top, 1));
        top = fmaxf(top, __shfl_xor_sync(kAll, top, 2));
        top = fmaxf(top, __shfl_xor_sync(kAll, top, 16));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float f = ex2(ref[i] - top);
            weight[(w0 + 8 * i) * kHeads + x] = f;
            l = fmaf(sum[i], f, l);
        }
        l += __shfl_xor_sync(kAll, l, 1);
        l += __shfl_xor_sync(kAll, l, 2);
        l += __shfl_xor_sync(kAll, l, 16);
        if (w0 == 0) {
            hd.factor[x] = top;
            hd.qsum[x][0] = l;
        }
    }
    __syncthreads();
    namespace cg = cooperative_groups;
    cg::cluster_group cl = cg::this_cluster();
    for (int e = threadIdx.x; e < p.g * (D / 2); e += blockDim.x) {
        const int x = e / (D / 2);
        float2 o = make_float2(0.f, 0.f);
#pragma unroll 4
        for (int w = 0; w < warps; ++w) {
            const float2 v = reinterpret_cast<const float2*>(parts(w))[e];
            const float f = weight[w * kHeads + x];
            o.x = fmaf(v.x, f, o.x);
            o.y = fmaf(v.y, f, o.y);
        }
        if (ctas > 1) {
            reinterpret_cast<float2*>(parts(0))[e] = o;
        } else {
            const float l = hd.qsum[x][0], inv = l != 0.f ? 1.f / l : 0.f;   // (NaN stays)
            const size_t row = size_t(b) * p.hq + h * p.g + x;
            reinterpret_cast<__nv_bfloat162*>(a.out + row * D)[e % (D / 2)] = __floats2bfloat162_rn(o.x * inv, o.y * inv);
            if (a.lse && e % (D / 2) == 0)
                a.lse[row] = l != 0.f ? (hd.factor[x] + log2f(l)) * 0.693147180559945309f : -INFINITY;
        }
    }
    if (ctas == 1) return;
    // ---- the cluster's sums: each CTA finishes its share of the outputs ----
    cl.sync();
    for (int e = rank * blockDim.x + threadIdx.x; e < p.g * (D / 2); e += ctas * blockDim.x) {
        const int x = e / (D / 2);
        float top = kRefNone, l = 0.f;
        float2 o = make_float2(0.f, 0.f);
        for (int c0 = 0; c0 < ctas; c0 += 8) {           // eight CTAs' parts under way at a time
            float ref[8], sum[8];
            float2 v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const bool have = c0 + i < ctas;
                const unsigned char* at = cl.map_shared_rank(smem, have ? c0 + i : 0);
                const Head<D, LO>& other = *reinterpret_cast<const Head<D, LO>*>(at);
                ref[i] = have ? other.factor[x] : kRefNone;
                sum[i] = have ? other.qsum[x][0] : 0.f;
                v[i] = have ? reinterpret_cast<const float2*>(at + sizeof(Head<D, LO>))[e] : make_float2(0.f, 0.f);
            }
            const float before = top;
#pragma unroll
            for (int i = 0; i < 8; ++i) top = fmaxf(top, ref[i]);
            const float f0 = ex2(before - top);
            l *= f0;
            o.x *= f0;
            o.y *= f0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float f = ex2(ref[i] - top);
                l = fmaf(sum[i], f, l);
                o.x = fmaf(v[i].x, f, o.x);
                o.y = fmaf(v[i].y, f, o.y);
            }
        }
        const float inv = l != 0.f ? 1.f / l : 0.f;
        const size_t row = size_t(b) * p.hq + h * p.g + x;
        reinterpret_cast<__nv_bfloat162*>(a.out + row * D)[e % (D / 2)] = __floats2bfloat162_rn(o.x * inv, o.y * inv);
        if (a.lse && e % (D / 2) == 0) a.lse[row] = l != 0.f ? (top + log2f(l)) * 0.693147180559945309f : -INFINITY;
    }
    cl.sync();                                           // no CTA leaves while another reads its part
}

// ---------------------------------------------------------------- launch

// CTAs per (sequence, kv-head), at most 16: one sequence of 131072 positions at 8 bits takes 99 us with 16, 144 with 8.
// A CTA of a round costs about its items (pages or ring pieces, shared by its warps)
// plus one and a half for its start and its end; the rounds are what `slots` CTAs at a time make of all of them.
// (64 ragged sequences of 8 kv-heads: 48 us with the 512 CTAs that this gives, 63 with 1536, 100 with 4096; CTAs of two
// warps, which would fill the SMs more evenly, took 56.)
inline int split_ctas(long long pairs, int items, int warps, int slots, int most) {
    int best = 1;
    double least = 1e30;
    for (int n = 1; n <= most; ++n) {
        if (n > 1 && n * warps > items) break;
        const double rounds = double((pairs * n + slots - 1) / slots);
        const double cost = rounds * (double((items + n * warps - 1) / (n * warps)) + 1.5);
        if (cost < 0.97 * least) {
            least = cost;
            best = n;
        }
    }
    return best;
}

template <int D, int KB, int VB, bool LO>
cudaError_t launch_decode_one(const Params& p, const Args& a, int sms, cudaStream_t s) {
    auto* kernel = sink_decode_kernel<D, KB, VB, LO>;
    // per device, once: large shared memory, and the largest cluster that fits at it (16 is beyond what every device
    // has to offer, 8 is not); two threads may both find it
    static std::atomic<int> largest[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    constexpr int kMost = 227 * 1024;
    int most_ctas = largest[dev];
    if (!most_ctas) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t c{};
        cudaLaunchAttribute at{};
        at.id = cudaLaunchAttributeClusterDimension;
        at.val.clusterDim.x = 16;
        at.val.clusterDim.y = at.val.clusterDim.z = 1;
        c.gridDim = dim3(16);
        c.blockDim = dim3(256);
        c.dynamicSmemBytes = kMost;
        c.attrs = &at;
        c.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, kernel, &c) != cudaSuccess) {
            cudaGetLastError();
            n = 0;
        }
        most_ctas = n > 0 ? 16 : 8;
        largest[dev] = most_ctas;
    }
    // four warps a CTA, or as many up to eight as bring the most warps onto an SM (large buffers)
    int warps = 4, per_sm = 1;
    for (int w = 4, most = 0; w <= 8; ++w) {
        const int n = std::min(kMaxWarps / w, (228 * 1024) / (decode_smem<D, KB, VB, LO>(p, w) + 1024));
        if (n * w > most) {
            most = n * w;
            warps = w;
            per_sm = n;
        }
    }
    const int smem = decode_smem<D, KB, VB, LO>(p, warps);
    const long long bound = std::min<long long>(a.len_cap, (long long)a.sinks + a.span + 2 * kPage);
    const int items = int((bound + kPage - 1) / kPage) + (std::min(p.W, a.len_cap) + kRing - 1) / kRing;
    const int n = split_ctas((long long)p.batch * p.hkv, items, warps, sms * per_sm, most_ctas);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(n, p.hkv, p.batch);
    cfg.blockDim = dim3(32 * warps);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = n;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = n > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, p, a);
}

template <int KB>
cudaError_t launch_decode_bits(const Params& p, const Args& a, int sms, cudaStream_t s) {
    const bool low = p.rotate || !a.q_bf16;             // the query needs more than one fp16 part
#define KVQ_SINK_CASE(DD, VV)                                                    \
    if (p.d == DD && p.vb == VV)                                                 \
        return low ? launch_decode_one<DD, KB, VV, true>(p, a, sms, s)           \
                   : launch_decode_one<DD, KB, VV, false>(p, a, sms, s);
    KVQ_SINK_CASE(128, 1) KVQ_SINK_CASE(128, 2) KVQ_SINK_CASE(128, 4) KVQ_SINK_CASE(128, 8)
    KVQ_SINK_CASE(64, 1) KVQ_SINK_CASE(64, 2) KVQ_SINK_CASE(64, 4) KVQ_SINK_CASE(64, 8)
#undef KVQ_SINK_CASE
    return cudaErrorInvalidValue;
}

}  // namespace sink
}  // namespace kvq
