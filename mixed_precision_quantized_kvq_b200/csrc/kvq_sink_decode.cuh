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
// out of the result.  One mask per two codes is all the unpacking there is.
//
// What bounds it: the codes and metadata of the visible positions in (116
// bytes per position and kv-head for 4-bit keys and 2-bit values), and about
// 900 issue slots a warp for 64 of them, which at this many bytes is the
// larger part.  Hence the products on mma.sync.m16n8k16 with the positions
// (scores) or channels (values) as its 16 rows and the up to 8 query heads of
// a kv-head as its 8 columns: fragments are registers, the codes never go
// through shared memory a second time.
//
// Work split: one cluster of 1 to 8 CTAs per (sequence, kv-head); its warps
// take the 64-position pages in turn (warp w of W: pages w, w + W, ...), then
// 16-slot pieces of the bf16 ring, each warp with its own ring of kStages
// shared-memory stages filled by cp.async.  The warps' partial sums meet in
// shared memory, across the cluster through distributed shared memory: no
// workspace, no atomics, the same result on every run.
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

#include "kvq_sink.cuh"
#include "kvq_tc_ptx.cuh"

#include "kvq_mma_ptx.cuh"

namespace kvq {
namespace sink {

using namespace ptx;

constexpr int kStages = 2;
constexpr int kMaxWarps = 12;          // of a CTA, and what the registers of an SM hold
constexpr int kHeads = 8;            // columns of the products
constexpr int kRing = 16;            // ring slots per piece
constexpr float kRefNone = -1e30f;   // reference exponent before any position
constexpr float kCode = 16777216.f;  // 2^24: codes are fp16 numbers c * 2^-24
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_k8(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(b0));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void sts32(uint32_t a, uint32_t v) {
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
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

// position (of eight) in row x of a score tile
template <int VB>
__device__ __forceinline__ constexpr int row_position(int x) {
    return VB == 4 ? (x >> 1) + 4 * (x & 1) : VB == 8 ? 4 * (x >> 2) + ((x >> 1) & 1) + 2 * (x & 1) : x;
}

// channels of code pair i (0..3) of lane column c within 32 channels, and the bit position of the pair
template <int KB>
__device__ __forceinline__ int pair_channel(int c, int i, int hi) {
    if (KB == 8) return (i >> 1) * 16 + 4 * c + (i & 1) + 2 * hi;
    if (KB == 4) return 8 * c + i + 4 * hi;
    if (KB == 2) return 16 * (c >> 1) + 4 * (c & 1) + i + 8 * hi;
    return 4 * c + i + 16 * hi;
}
template <int KB>
__device__ __forceinline__ constexpr int pair_bit(int i) {
    return KB == 4 ? 4 * (i & 1) : KB == 2 ? 2 * i : KB == 1 ? i : 0;
}

// Shared memory of a CTA of W warps: query fragments' sources, then the
// warps' stages; the partial sums take the stages' place at the end.
template <int D>
struct Head {
    __half qh[kHeads][D];                    // query, scaled to at most 2^8 per head, high and low part
    __half ql[kHeads][D];
    __nv_bfloat16 bh[kHeads][D + 8];         // unrotated query for the ring, high and low part
    __nv_bfloat16 bl[kHeads][D + 8];
    float qsum[kHeads][4];                   // sums over 32 channels
    float factor[kHeads];                    // score scale * log2(e) / query scaling
};

template <int D, int KB, int VB>
struct Stage {
    static constexpr int kK = kPage * D * KB / 8, kV = kPage * D * VB / 8;
    static constexpr int kRingBytes = 2 * kRing * 2 * D;
    __host__ __device__ static int bytes(const Params& p) {
        const int page = kK + kV + kPage * 4 * (p.nkg + p.nvg);
        return page > kRingBytes ? page : kRingBytes;
    }
};

// partial sums of a warp: [head][D] values, then reference exponents and sums of the weights
template <int D>
constexpr int kPartFloats = kHeads * D + 2 * kHeads;

template <int D, int KB, int VB>
__host__ __device__ int decode_smem(const Params& p, int warps) {
    const int stage = Stage<D, KB, VB>::bytes(p) * kStages, part = kPartFloats<D> * 4;
    return int(sizeof(Head<D>)) + warps * (stage > part ? stage : part);
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
    // 2^log_scale): both round to fp16 without overflow, and what lies 2^-39 below the largest still counts.
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

// one 64-position page in the stage at `st`: base = position of slot 0
template <int D, int KB, int VB, bool LO>
__device__ __forceinline__ void page_tile(const Params& p, uint32_t st, int base, int ns, int lo, int Lq, bool edge,
                                          const uint32_t (&qh)[D / 8], const uint32_t (&ql)[LO ? D / 8 : 1],
                                          uint32_t qz, const float (&factor)[2], Sums<D>& S) {
    using G = Stage<D, KB, VB>;
    constexpr int NU = D / 32;
    const int lane = threadIdx.x % 32, r = lane >> 2, c = lane & 3;
    const int nkg = p.nkg, nvg = p.nvg;
    const uint32_t sk = st, sv = st + G::kK, skm = sv + G::kV, svm = skm + kPage * 4 * nkg;
    if (edge) {   // positions that are not visible: finite scores (masked below) and no values
        for (int t = lane; t < kPage; t += 32)
            if (!visible(base + t, ns, lo, Lq)) {
                for (int i = 0; i < nkg; ++i) sts32(skm + (t * nkg + i) * 4, 0);
                for (int i = 0; i < nvg; ++i) sts32(svm + (t * nvg + i) * 4, 0);
            }
        __syncwarp();
    }
    const int perm = row_position<VB>(r);
    // ---- scores: four tiles of 16 positions ----
    float s[4][4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const int t0 = 16 * b + perm, t1 = t0 + 8;      // positions of rows r and r + 8
        uint32_t m0[4], m1[4];                          // metadata of the 32-channel units
        if (nkg == 4) {
            const uint4 x = lds128(skm + t0 * 16), y = lds128(skm + t1 * 16);
            m0[0] = x.x, m0[1] = x.y, m0[2] = x.z, m0[3] = x.w;
            m1[0] = y.x, m1[1] = y.y, m1[2] = y.z, m1[3] = y.w;
        } else {
            const int sh = nkg == NU ? 0 : nkg * 2 == NU ? 1 : 2;
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                m0[u] = lds32(skm + (t0 * nkg + (u >> sh)) * 4);
                m1[u] = lds32(skm + (t1 * nkg + (u >> sh)) * 4);
            }
        }
        // zero points of units 2(c & 1), 2(c & 1) + 1 against the unit sums (high parts at c < 2, low at c >= 2)
        float z[4] = {0.f, 0.f, 0.f, 0.f};
        if (NU == 4) {
            const bool odd = c & 1;
            mma_f16_k8(z, __byte_perm(odd ? m0[2] : m0[0], odd ? m0[NU - 1] : m0[1], 0x7632),
                       __byte_perm(odd ? m1[2] : m1[0], odd ? m1[NU - 1] : m1[1], 0x7632), qz);
        } else {
            mma_f16_k8(z, (c & 1) ? 0u : __byte_perm(m0[0], m0[1], 0x7632), (c & 1) ? 0u : __byte_perm(m1[0], m1[1], 0x7632),
                       qz);
        }
        float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            uint32_t e[4], f[4];                        // code pairs of rows r and r + 8
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int t = h ? t1 : t0;
                uint32_t(&x)[4] = h ? f : e;
                if (KB == 8) {
                    const uint32_t w0 = lds32(sk + (2 * u) * (kPage * 16) + t * 16 + c * 4);
                    const uint32_t w1 = lds32(sk + (2 * u + 1) * (kPage * 16) + t * 16 + c * 4);
                    x[0] = w0 & 0x00ff00ffu;
                    x[1] = (w0 >> 8) & 0x00ff00ffu;
                    x[2] = w1 & 0x00ff00ffu;
                    x[3] = (w1 >> 8) & 0x00ff00ffu;
                } else if (KB == 4) {
                    const uint32_t w = lds32(sk + u * (kPage * 16) + t * 16 + c * 4), v = w >> 8;
                    x[0] = w & 0x000f000fu;
                    x[1] = w & 0x00f000f0u;
                    x[2] = v & 0x000f000fu;
                    x[3] = v & 0x00f000f0u;
                } else if (KB == 2) {
                    const uint32_t w = lds32(sk + (u >> 1) * (kPage * 16) + t * 16 + (2 * (u & 1) + (c >> 1)) * 4) >> (8 * (c & 1));
                    x[0] = w & 0x00030003u;
                    x[1] = w & 0x000c000cu;
                    x[2] = w & 0x00300030u;
                    x[3] = w & 0x00c000c0u;
                } else {
                    const uint32_t w = lds32(sk + t * (D / 8) + u * 4) >> (4 * c);
                    x[0] = w & 0x00010001u;
                    x[1] = w & 0x00020002u;
                    x[2] = w & 0x00040004u;
                    x[3] = w & 0x00080008u;
                }
            }
            float d[4] = {0.f, 0.f, 0.f, 0.f};
            mma_f16(d, e[0], f[0], e[1], f[1], qh[4 * u], qh[4 * u + 1]);
            mma_f16(d, e[2], f[2], e[3], f[3], qh[4 * u + 2], qh[4 * u + 3]);
            if (LO) {
                mma_f16(d, e[0], f[0], e[1], f[1], ql[LO ? 4 * u : 0], ql[LO ? 4 * u + 1 : 0]);
                mma_f16(d, e[2], f[2], e[3], f[3], ql[LO ? 4 * u + 2 : 0], ql[LO ? 4 * u + 3 : 0]);
            }
            const float s0 = low_half(m0[u]), s1 = low_half(m1[u]);
            a[0] = fmaf(s0, d[0], a[0]);
            a[1] = fmaf(s0, d[1], a[1]);
            a[2] = fmaf(s1, d[2], a[2]);
            a[3] = fmaf(s1, d[3], a[3]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) s[b][i] = fmaf(a[i], kCode, z[i]) * factor[i & 1];
        if (edge) {
            if (!visible(base + t0, ns, lo, Lq)) s[b][0] = s[b][1] = -INFINITY;
            if (!visible(base + t1, ns, lo, Lq)) s[b][2] = s[b][3] = -INFINITY;
        }
    }
    // ---- weights ----
    float top[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        float x = fmaxf(s[0][e], s[0][e + 2]);
#pragma unroll
        for (int b = 1; b < 4; ++b) x = fmaxf(x, fmaxf(s[b][e], s[b][e + 2]));
        top[e] = max_rows(x);
    }
    uint32_t vmax = 0;                                   // largest value scale, as its fp16 bits
    for (int i = lane; i < kPage * nvg; i += 32) vmax = max(vmax, lds32(svm + i * 4) & 0x7fffu);
    vmax = __reduce_max_sync(kAll, vmax);
    raise_ref(S, top, max(0, int(vmax >> 10) - 14));     // a scale is below 2^(exponent field - 14)
    uint32_t w[8];                                       // weights (positions of rows 2c, 2c+1; head r) of eight positions
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float p0 = ex2(s[b][2 * h] - S.ref[0]), p1 = ex2(s[b][2 * h + 1] - S.ref[1]);
            S.l[0] += p0;
            S.l[1] += p1;
            w[2 * b + h] = transpose8(half2_bits(p0, p1));
        }
    // B registers: the two positions whose codes one mask takes out of a value word
    uint32_t B[8];
    int tok[8];                                          // position of the low half; the high half is `gap` further
    constexpr int gap = VB == 8 ? 2 : VB == 4 ? 4 : VB == 2 ? 8 : 16;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (VB >= 4) {
            B[j] = w[j];
            tok[j] = 8 * j + (VB == 4 ? c : 4 * (c >> 1) + (c & 1));
        } else if (VB == 2) {
            B[j] = __byte_perm(w[j & ~1], w[j | 1], (j & 1) ? 0x7632 : 0x5410);
            tok[j] = 16 * (j >> 1) + 2 * c + (j & 1);
        } else {
            const int wd = j >> 2, hh = (j >> 1) & 1;
            B[j] = __byte_perm(w[4 * wd + hh], w[4 * wd + hh + 2], (j & 1) ? 0x7632 : 0x5410);
            tok[j] = 32 * wd + 8 * hh + 2 * c + (j & 1);
        }
    }
    // ---- values ----
    uint32_t Z[8], pv[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) Z[j] = 0;
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt) {
        if (16 * mt % p.vg == 0) {
            const int gi = 16 * mt / p.vg;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t x = lds32(svm + (tok[j] * nvg + gi) * 4), y = lds32(svm + ((tok[j] + gap) * nvg + gi) * 4);
                pv[j] = hmul2(B[j], __byte_perm(x, y, 0x5410));
                // odd pairs of 2-bit and 1-bit codes sit at bit 2 and bit 1
                if (VB == 2 && (j & 1)) pv[j] = hmul2(pv[j], 0x34003400u);
                if (VB == 1 && (j & 1)) pv[j] = hmul2(pv[j], 0x38003800u);
                if (r == gi) Z[j] = __byte_perm(x, y, 0x7632);
            }
        }
        uint32_t e[8], f[8];                             // code pairs of channels 16*mt + r and + 8
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int ch = 16 * mt + 8 * h + r;
            uint32_t(&x)[8] = h ? f : e;
            if (VB == 8) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    x[j] = (lds32(sv + (j >> 1) * (D * 16) + ch * 16 + (2 * (j & 1) + (c >> 1)) * 4) >> (8 * (c & 1))) & 0x00ff00ffu;
            } else if (VB == 4) {
                const uint4 u = lds128(sv + ch * 16), v = lds128(sv + D * 16 + ch * 16);
                const uint32_t wd[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = (wd[j] >> (4 * c)) & 0x000f000fu;
            } else if (VB == 2) {
                const uint4 u = lds128(sv + ch * 16);
                const uint32_t wd[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t v = wd[j] >> (4 * c);
                    x[2 * j] = v & 0x00030003u;
                    x[2 * j + 1] = v & 0x000c000cu;
                }
            } else {
                const uint2 u = lds64(sv + ch * 8);
                const uint32_t wd[2] = {u.x, u.y};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t v = wd[j >> 1] >> (2 * c + 8 * (j & 1));
                    x[2 * j] = v & 0x00010001u;
                    x[2 * j + 1] = v & 0x00020002u;
                }
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_f16(S.acc[mt], e[2 * k], f[2 * k], e[2 * k + 1], f[2 * k + 1], pv[2 * k], pv[2 * k + 1]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) mma_f16(S.zero, Z[2 * k], 0, Z[2 * k + 1], 0, B[2 * k], B[2 * k + 1]);
}

// Where 16-byte piece o of ring row i lies: exchanged within the row so that the same piece of eight rows falls into
// different banks (values, by columns) and four neighbouring pieces of rows 2k, 2k+1 do (keys, by rows).
template <int D>
__device__ __forceinline__ int ring_piece(int i, int o) {
    return i * (2 * D) + ((o ^ (((i & 1) << 2) | ((i >> 1) & 3))) << 4);
}

// 16 ring slots in the stage at `st`; ok: bit i set when slot i holds a visible position (other rows are zeros)
template <int D>
__device__ __forceinline__ void ring_tile(const Head<D>& hd, uint32_t st, uint32_t ok, bool lo_part, float scale_log2,
                                          Sums<D>& S) {
    const int lane = threadIdx.x % 32, r = lane >> 2, c = lane & 3;
    const uint32_t sv = st + kRing * 2 * D;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {                   // channels 32*j + 8*c .. + 7 in one 16-byte piece
        const uint4 k0 = lds128(st + ring_piece<D>(r, 4 * j + c)), k1 = lds128(st + ring_piece<D>(r + 8, 4 * j + c));
        const uint4 q = *reinterpret_cast<const uint4*>(&hd.bh[r][32 * j + 8 * c]);
        uint32_t a[4] = {k0.x, k1.x, k0.y, k1.y}, b[4] = {k0.z, k1.z, k0.w, k1.w};
        mma_bf16(s, a, q.x, q.y);
        mma_bf16(s, b, q.z, q.w);
        if (lo_part) {
            const uint4 ql = *reinterpret_cast<const uint4*>(&hd.bl[r][32 * j + 8 * c]);
            mma_bf16(s, a, ql.x, ql.y);
            mma_bf16(s, b, ql.z, ql.w);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = (ok >> (r + 8 * (i >> 1))) & 1u ? s[i] * scale_log2 : -INFINITY;
    const float top[2] = {max_rows(fmaxf(s[0], s[2])), max_rows(fmaxf(s[1], s[3]))};
    raise_ref(S, top, 0);
    float p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = ex2(s[i] - S.ref[i & 1]);
    S.l[0] += p[0] + p[2];
    S.l[1] += p[1] + p[3];
    // weights as bf16 high and low parts, in the output's unit of 2^-24
    uint32_t wh[2], wl[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float x = p[2 * h] * (1.f / kCode), y = p[2 * h + 1] * (1.f / kCode);
        const uint32_t hi = bf162_bits(x, y);
        wh[h] = transpose8(hi);
        wl[h] = transpose8(bf162_bits(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xffff0000u)));
    }
    // matrix i of the load: positions 8*(i >> 1) .., channels 16*mt + 8*(i & 1) ..
    const int row = (lane & 7) + 8 * (lane >> 4), piece = (lane >> 3) & 1;
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt) {
        uint32_t a[4];
        ldsm_x4_t(a, sv + ring_piece<D>(row, 2 * mt + piece));
        mma_bf16(S.acc[mt], a, wh[0], wh[1]);
        mma_bf16(S.acc[mt], a, wl[0], wl[1]);
    }
}

template <int D, int KB, int VB, bool LO>
__global__ void __launch_bounds__(kMaxWarps * 32) sink_decode_kernel(const __grid_constant__ Params p, const __grid_constant__ Args a) {
    using G = Stage<D, KB, VB>;
    extern __shared__ __align__(16) unsigned char smem[];
    Head<D>& hd = *reinterpret_cast<Head<D>*>(smem);
    const int warps = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int r = lane >> 2, c = lane & 3;
    const int h = blockIdx.y, b = blockIdx.z, rank = blockIdx.x, ctas = gridDim.x;
    const int stage_bytes = G::bytes(p);
    const int region = max(kStages * stage_bytes, kPartFloats<D> * 4);
    unsigned char* mine = smem + sizeof(Head<D>) + warp * region;
    const uint32_t st0 = smem_u32(mine);

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

    // start the copies of item number k of this warp; what: -1 nothing there, 0 page, else the valid ring slots
    auto issue = [&](int k, int stage) -> int {
        const int it = start + k * step;
        int what = -1;
        if (k - table_at >= 32) look_up(k);
        const int pg = __shfl_sync(kAll, table, k - table_at);
        if (it < n_page) {
            if (pg >= 0) {
                what = 0;
                const uint32_t st = st0 + stage * stage_bytes;
                const size_t blk = size_t(pg) * p.hkv + h;
                const uint8_t* kc = p.k_codes + blk * G::kK + lane * 16;
                const uint8_t* vc = p.v_codes + blk * G::kV + lane * 16;
#pragma unroll
                for (int e = 0; e < G::kK; e += 512) cp16(st + e + lane * 16, kc + e);
#pragma unroll
                for (int e = 0; e < G::kV; e += 512) cp16(st + G::kK + e + lane * 16, vc + e);
                const uint8_t* km = reinterpret_cast<const uint8_t*>(p.k_meta) + blk * (kPage * 4) * p.nkg;
                const uint8_t* vm = reinterpret_cast<const uint8_t*>(p.v_meta) + blk * (kPage * 4) * p.nvg;
                const uint32_t sm = st + G::kK + G::kV;
                const int nk = 16 * p.nkg, n = nk + 16 * p.nvg;
                for (int e = lane; e < n; e += 32) cp16(sm + e * 16, e < nk ? km + e * 16 : vm + (e - nk) * 16);
            }
        } else if (it < n_item) {
            const int slot = (it - n_page) * kRing + (lane & (kRing - 1)), q0 = Lq % p.W;
            const int x = Lq + (slot >= q0 ? slot - q0 : slot - q0 + p.W);
            const bool ok = slot < p.W && visible(x, ns, lo, L);
            const unsigned any = __ballot_sync(kAll, ok) & 0xffffu;
            if (any) {
                what = int(any);
                const uint32_t st = st0 + stage * stage_bytes;
                const size_t row = (size_t(b) * p.hkv + h) * p.W + (it - n_page) * kRing;
                for (int e = lane; e < 2 * kRing * (D / 8); e += 32) {
                    const int i = e / (D / 8), o = e % (D / 8), sl = i & (kRing - 1);
                    const bool have = (any >> sl) & 1u;
                    const __nv_bfloat16* src = (i < kRing ? p.k_win : p.v_win) + (have ? (row + sl) * D + o * 8 : 0);
                    cp16_zfill(st + (i < kRing ? 0 : kRing * 2 * D) + ring_piece<D>(sl, o), src, have);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        return what;
    };
    int what[kStages];
#pragma unroll
    for (int k = 0; k < kStages; ++k) what[k] = issue(k, k);

    // ---- queries: each head's row by one warp ----
    {
        constexpr int C = D / 32;
        const int g = p.g;
        for (int x = warp; x < kHeads; x += warps) {
            float q[C];
#pragma unroll
            for (int i = 0; i < C; ++i) q[i] = 0.f;
            if (x < g) {
                const size_t at = size_t(b) * a.q_stride + size_t(h * g + x) * D + lane * C;
#pragma unroll
                for (int i = 0; i < C; ++i)
                    q[i] = a.q_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[at + i])
                                    : static_cast<const float*>(a.q)[at + i];
            }
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const __nv_bfloat16 hi = __float2bfloat16_rn(q[i]);
                hd.bh[x][lane * C + i] = hi;
                hd.bl[x][lane * C + i] = __float2bfloat16_rn(q[i] - __bfloat162float(hi));
            }
            if (p.rotate) rotate_warp<D>(q, p.signs, lane);
            float m = 0.f, sum = 0.f;
#pragma unroll
            for (int i = 0; i < C; ++i) m = fmaxf(m, fabsf(q[i]));
            for (int w = 16; w; w >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, w));
            // a power of two that brings the head's largest element into [2^7, 2^8)
            const int ex = max(-100, int(__float_as_uint(m) >> 23) - 127);
            const float up = __uint_as_float(uint32_t(127 + 7 - ex) << 23);
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const float v = q[i] * up;
                const __half hi = __float2half_rn(v);
                hd.qh[x][lane * C + i] = hi;
                hd.ql[x][lane * C + i] = __float2half_rn(v - __half2float(hi));
                sum += v;
            }
#pragma unroll
            for (int w = 1; w < 32 / C; w <<= 1) sum += __shfl_xor_sync(kAll, sum, w);
            if (lane % (32 / C) == 0) hd.qsum[x][lane / (32 / C)] = sum;
            if (lane == 0) hd.factor[x] = a.scale_log2 * __uint_as_float(uint32_t(127 - 7 + ex) << 23);
        }
    }
    __syncthreads();
    uint32_t qh[D / 8], ql[LO ? D / 8 : 1];
#pragma unroll
    for (int u = 0; u < D / 32; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c0 = 32 * u + pair_channel<KB>(c, i, 0), c1 = 32 * u + pair_channel<KB>(c, i, 1);
            const float down = 1.f / float(1 << pair_bit<KB>(i));
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
        const int it = start + k * step, stage = k % kStages;
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        __syncwarp();
        int now = what[0];
#pragma unroll
        for (int i = 1; i < kStages; ++i)
            if (stage == i) now = what[i];
        const uint32_t st = st0 + stage * stage_bytes;
        if (now >= 0) {
            if (it < n_page) {
                const int base = logical(it) * kPage;
                const bool edge = base + kPage > Lq || (base < lo && base + kPage > ns);
                page_tile<D, KB, VB, LO>(p, st, base, ns, lo, Lq, edge, qh, ql, qz, factor, S);
            } else {
                ring_tile<D>(hd, st, uint32_t(now), ring_lo, a.scale_log2, S);
            }
        }
        __syncwarp();
        const int next = issue(k + kStages, stage);
#pragma unroll
        for (int i = 0; i < kStages; ++i)
            if (stage == i) what[i] = next;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();

    // ---- this warp's sums to its part of shared memory (its stages are free) ----
    float* part = reinterpret_cast<float*>(mine);
    S.l[0] = sum_rows(S.l[0]);
    S.l[1] = sum_rows(S.l[1]);
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt) {
        const int gi = 16 * mt / p.vg;                   // all 16 channels of a tile are in one group
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

    // ---- all parts of the cluster: each CTA finishes its share of the outputs ----
    namespace cg = cooperative_groups;
    cg::cluster_group cl = cg::this_cluster();
    if (ctas > 1)
        cl.sync();
    else
        __syncthreads();
    for (int e = rank * blockDim.x + threadIdx.x; e < p.g * (D / 2); e += ctas * blockDim.x) {
        const int x = e / (D / 2), j = 2 * (e % (D / 2));
        float top = kRefNone;
        for (int i = 0; i < ctas; ++i) {
            const unsigned char* base = ctas > 1 ? cl.map_shared_rank(smem, i) : smem;
            for (int w = 0; w < warps; ++w)
                top = fmaxf(top, reinterpret_cast<const float*>(base + sizeof(Head<D>) + w * region)[kHeads * D + x]);
        }
        float o0 = 0.f, o1 = 0.f, l = 0.f;
        for (int i = 0; i < ctas; ++i) {
            const unsigned char* base = ctas > 1 ? cl.map_shared_rank(smem, i) : smem;
            for (int w = 0; w < warps; ++w) {
                const float* q = reinterpret_cast<const float*>(base + sizeof(Head<D>) + w * region);
                const float f = ex2(q[kHeads * D + x] - top);
                const float2 v = *reinterpret_cast<const float2*>(q + x * D + j);
                o0 = fmaf(v.x, f, o0);
                o1 = fmaf(v.y, f, o1);
                l = fmaf(q[kHeads * D + kHeads + x], f, l);
            }
        }
        const float inv = l > 0.f ? 1.f / l : 0.f;
        const size_t row = size_t(b) * p.hq + h * p.g + x;
        *reinterpret_cast<__nv_bfloat162*>(a.out + row * D + j) = __floats2bfloat162_rn(o0 * inv, o1 * inv);
        if (a.lse && j == 0) a.lse[row] = l > 0.f ? (top + log2f(l)) * 0.693147180559945309f : -INFINITY;
    }
    if (ctas > 1) cl.sync();                             // no CTA leaves while another reads its part
}

// ---------------------------------------------------------------- launch

// CTAs per (sequence, kv-head).  A CTA of a round costs about its items (pages or ring pieces, shared by its warps)
// plus one and a half for its start and its end; the rounds are what `slots` CTAs at a time make of all of them.
inline int split_ctas(long long pairs, int items, int warps, int slots) {
    int best = 1;
    double least = 1e30;
    for (int n = 1; n <= 8; ++n) {
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
    static int opted[64];                               // largest dynamic shared memory asked for, per device
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    constexpr int kMost = 227 * 1024;
    if (!opted[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
        if (e != cudaSuccess) return e;
        opted[dev] = kMost;
    }
    // four warps, or two where the stages of 8-bit codes would leave room for one CTA only
    int warps = 4;
    if (2 * decode_smem<D, KB, VB>(p, 4) > kMost) warps = 2;
    const int smem = decode_smem<D, KB, VB>(p, warps);
    const int per_sm = std::max(1, std::min(12 / warps, (228 * 1024) / (smem + 1024)));
    const long long bound = std::min<long long>(a.len_cap, (long long)a.sinks + a.span + 2 * kPage);
    const int items = int((bound + kPage - 1) / kPage) + (std::min(p.W, a.len_cap) + kRing - 1) / kRing;
    const int n = split_ctas((long long)p.batch * p.hkv, items, warps, sms * per_sm);
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
