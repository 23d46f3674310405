// Attention of a chunk of new queries with sinks and a sliding span over the
// quantized cache (kvq_sink_prefill_attention) on the 5th-generation tensor
// cores (tcgen05, sm_100a).  Every layout; also the single-token form of the
// layouts whose scales are not shared by 32 channels (kvq_sink_decode.cuh): up
// to 8 of its 256 rows; one sequence, 8192 positions: 46 us with key groups
// along positions, 41 with groups of 16 channels.
//
//     S = Q K^T,  P = 2^(factor S - ref) where visible,  O += P V,  l += P 1
//
// over tiles of 64 positions (a page), with a running reference exponent per
// query row; O / l is rounded to bf16.  Bound by the tensor cores and the
// exponentials (one per visible pair: 16 a clock and SM, which takes as long as
// the two products at head_dim 128), in practice by the hand-overs of a tile:
// the tensor core works 46% of the time, issue slots are 62% busy, exponentials
// 35%.  Measured on a B200: 749 us for chunks of 512 queries of
// 16 sequences at 4096 positions, 32 query and 8 kv-heads (550 GFLOP: 735
// TFLOP/s, 44% of a library product's rate); a tile takes 2.4 us a CTA of which
// the tensor core works 0.7, a CTA's start and end about 15.
//
// One CTA per SM takes 256 rows of one (sequence, kv-head): two blocks of 128,
// each 128/g queries with their g heads.  Reconstructing a key or value costs
// about two issue slots an element, so a tile is reconstructed once, to fp16,
// for both blocks.  Tensor memory holds two score tiles and the output of each
// block: the next tile's scores are there before a tile's weights are done, so
// the weights seldom wait for a product (tiles of 128 positions with one score
// tile a block took 0.91 ms at the size above).  Warps:
//   0-3, 4-7   weights of block 0 and 1: thread = row.  S from tensor memory
//              once, P back over S as fp16; reference and O are adjusted only
//              when a score exceeds the reference by more than 15 binades.
//   8-11       reconstruct keys: thread = half the channels of a position
//              (groups along positions: two channels of half the positions).
//   12-19      values: thread = half the positions of a channel.  Codes and
//              metadata are loaded a tile ahead, page numbers two.
//   20, 21     issue the products of block 0 and 1 (22, 23 fill the warp group).
// The kernel is launched with 80 registers a thread, 1920 over its 24 warps; the
// roles then take 96, 112, 64 and 48: 8*96 + 4*112 + 8*64 + 4*48 = 1920.  (With
// fewer for the issuing warps they spill and everything waits for them.)
// Where few rows leave SMs idle and there are tiles enough, a cluster of 2, 4 or
// 8 CTAs shares the tiles of its rows (CTA c of n: tiles c, c + n, ...) and joins
// its outputs through distributed shared memory: 33 queries over 16000 positions
// of one sequence take 66 us.  A kernel of its own, since the arithmetic of the
// shared tiles costs the others 8%.
// Operands are 8x16-byte core matrices without swizzle, all 16-byte pieces of
// the same eight columns together, which makes the writers' 16-byte stores
// contiguous over a warp.  A word holds the codes (i, i + n/2) in the same
// bits of its halves, so reconstructed pairs come out in that order; instead of
// sorting them, the query's channels are stored in the same order (keys), and
// key rows, that is, the columns of S and P (values).
#include <math.h>

#include <algorithm>
#include <atomic>

#include <cooperative_groups.h>
#include <stddef.h>

#include "kvq_sink.cuh"
#include "kvq_tc_ptx.cuh"

#include "kvq_mma_ptx.cuh"

namespace kvq {
namespace sink {
namespace {

using namespace ptx;

constexpr int kRows = 128;                    // rows of a block
constexpr int kTile = kPage;                  // positions of a tile
constexpr int kThreads = 24 * 32;
constexpr int kKeyThreads = 128, kValueThreads = 256;
constexpr int kStages = 4;
constexpr uint64_t kLimitNs = 2000000000ull;  // a wait that takes longer gives up
constexpr float kRefNone = -1e30f;
constexpr float kTopWeight = 15.f, kLowTop = 8.f;   // the largest weight's exponent: at most, and after a rise
constexpr int kKeyPitch = kTile * 16 + 16;    // bytes between 16-byte columns of the key tile and of the queries: the
constexpr int kQueryPitch = kRows * 16 + 16;  // extra piece puts neighbouring columns of a row in different banks

// positions of the halves of pair p in a run of words of N codes
template <int N>
__device__ __forceinline__ constexpr int pair_low(int p) { return p / (N / 2) * N + p % (N / 2); }
// where code i of a run lies once the words are unpacked
__device__ __forceinline__ int slot_of(int i, int n) { return (i & ~(n - 1)) + 2 * (i & (n / 2 - 1)) + ((i & (n / 2)) ? 1 : 0); }

template <int D>
struct Smem {
    static constexpr int kQ = D / 8 * kQueryPitch;      // one block's queries
    static constexpr int kK = D / 8 * kKeyPitch;
    static constexpr int kV = kTile / 8 * D * 16;
    unsigned char q[2][(kQ + 127) / 128 * 128];
    unsigned char k[kStages][(kK + 127) / 128 * 128];
    unsigned char v[kStages][kV];
    alignas(16) __half vscale[2][8][kTile];             // value scales and zero points of two tiles: by group, in the
    alignas(16) __half vzero[2][8][kTile];              // order of the unpacked codes
    uint64_t kfull[kStages], kempty[kStages], vfull[kStages], vempty[kStages];
    uint64_t sfull[2][2], pfull[2][2];                  // block, tile % 2
    uint64_t odone[2], olast[2], qfull[2];              // a tile's values, the last tile's; the queries
    uint32_t tmem;
    int hidden[8];                                      // tile % 8: its page is absent
    int failed;
};

// One thread issues the products and their commits, in a branch of its own and without the optional operands: 64
// cycles for each 128x128x16 product, the tensor core's own time (112 to 130 with a predicate on each from the whole
// warp).
__device__ __forceinline__ bool elected() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(e)::"memory");
    return e != 0;
}
template <bool ADD>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "n"(ADD ? 1 : 0)
        : "memory");
}
template <bool ADD>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "n"(ADD ? 1 : 0)
        : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// floats between the rows of a CTA's part of a join: the output, reference, sum
template <int D>
constexpr int kPartPitch = D + 4;

// instruction descriptor: fp16 A and B (K-major), fp32 accumulator
constexpr uint32_t idesc_f16(int M, int N) { return (1u << 4) | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24); }

__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// two fp32 numbers in one register pair
__device__ __forceinline__ uint64_t pack2(float x, float y) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
    return v;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& x, float& y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t v;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
    return v;
}
// a load's registers are there once this has run; they pass through it so that nothing that reads them moves before it
__device__ __forceinline__ void tmem_loaded(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14])
                 :
                 : "memory");
    asm volatile("" : "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                      "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29])
                 :
                 : "memory");
    asm volatile("" : "+r"(r[30]), "+r"(r[31]) : : "memory");
}
__device__ __forceinline__ void arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 half2_of(uint32_t w) { return *reinterpret_cast<__half2*>(&w); }

// The 16/BITS pairs of a word as exact fp16 numbers.  With 0x6400 above them the ten low bits of a half-word are the
// mantissa of 1024 + code * 2^position; one exact operation takes both away.
template <int BITS>
__device__ __forceinline__ void unpack(uint32_t w, __half2 (&c)[16 / BITS]) {
    constexpr int kSpan = 10 / BITS * BITS;              // whole codes among the ten bits
    constexpr uint32_t kMask = ((1u << BITS) - 1u) * 0x00010001u;
#pragma unroll
    for (int i = 0; i < 16 / BITS; ++i) {
        const int at = i * BITS % kSpan, shift = i * BITS - at;
        const __half2 x = half2_of(((w >> shift) & (kMask << at)) | 0x64006400u);
        if (at == 0)
            c[i] = __hsub2(x, half2_of(0x64006400u));
        else
            c[i] = __hfma2(x, half2_of(uint32_t(15 - at) * 0x04000400u), half2_of(0x80008000u | uint32_t(25 - at) * 0x04000400u));
    }
}

// the lowest n bits, for any n
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }
// bits of 32 positions to the slots of their codes, n codes a word (slot_of for all of them)
__device__ __forceinline__ uint32_t slots_of(uint32_t v, int n) {
    const auto swap = [&](uint32_t mask, int by) {       // exchange the bits of `mask` with those `by` above
        const uint32_t t = ((v >> by) ^ v) & mask;
        v ^= t ^ (t << by);
    };
    if (n >= 32) swap(0x0000ff00u, 8);
    if (n >= 16) swap(0x00f000f0u, 4);
    if (n >= 8) swap(0x0c0c0c0cu, 2);
    swap(0x22222222u, 1);
    return v;
}

// What a CTA works on.  SPLIT: several CTAs share the tiles (the others' code does without).
template <bool SPLIT>
struct Work {
    int b, h, L, Lq, lo, p_max, sinks;          // lo: first position of the first query's span
    int n_sink, first, n_tile;                  // tiles of the sinks, first tile of the span, this CTA's tiles
    int rank, ctas;                             // this CTA takes tiles rank, rank + ctas, ...
    __device__ __forceinline__ int tile_start(int j) const {
        if (SPLIT) j = j * ctas + rank;
        return (j < n_sink ? j : j - n_sink + first) * kTile;
    }
    // seen by some row (a necessary condition; the rows' own masks are exact)
    __device__ __forceinline__ bool used(int x) const { return x <= p_max && (x < sinks || x >= lo); }
};

// eight bf16 numbers as fp32
__device__ __forceinline__ void widen(const uint4& w, float (&x)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}

// Two fp32 numbers as their nearest fp16 numbers and what those leave, in fp16 again: together 2^-22 of themselves off,
// or half a step of the smallest fp16 numbers.
struct Split {
    uint32_t high, low;
};
__device__ __forceinline__ Split split2(float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    return {bits(h), bits(__floats2half2_rn(x - __low2float(h), y - __high2float(h)))};
}
// code * scale + zero in fp32, split
__device__ __forceinline__ Split split_key(__half2 code, __half2 scale, __half2 zero) {
    return split2(fmaf(__low2float(code), __low2float(scale), __low2float(zero)),
                  fmaf(__high2float(code), __high2float(scale), __high2float(zero)));
}

// One row of D channels by D/8 neighbouring lanes, eight channels each, to column `row` of an operand of fp16 pieces
// `pitch` bytes apart; n: codes per word of the keys (channel order).  scaled: by `sign` and a power of two into
// [2^13, 2^14); returns that power's inverse.  EXACT: what the fp16 numbers leave goes `low` bytes further.  The whole warp
// calls it; nothing is stored where `to` is null.
template <int D, bool EXACT>
__device__ __forceinline__ float put_row(float (&x)[8], const int8_t* signs, bool scaled, float sign, unsigned char* to,
                                         int low, int pitch, int row, int n) {
    const int oct = threadIdx.x % (D / 8);
    if (signs) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= float(__ldg(signs + oct * 8 + i));
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
                const float o = __shfl_xor_sync(0xffffffffu, x[i], m);
                x[i] = (oct & m) ? o - x[i] : x[i] + o;
            }
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= RotScale<D>::v;
    }
    float up = 1.f, down = 1.f;
    if (scaled) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
#pragma unroll
        for (int w = 1; w < D / 8; w <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
        const int e = max(-100, int(__float_as_uint(m) >> 23) - 127);
        up = sign * __uint_as_float(uint32_t(127 + 13 - e) << 23);
        down = __uint_as_float(uint32_t(127 - 13 + e) << 23);
    }
    if (!to) return down;
#pragma unroll
    for (int part = 0; part < (EXACT ? 2 : 1); ++part) {
        if (n <= 8) {                                    // the lane's channels stay in one piece
            const auto pair = [&](int a, int b) { return bits(__floats2half2_rn(x[a] * up, x[b] * up)); };
            *reinterpret_cast<uint4*>(to + oct * pitch + row * 16) =
                n == 8   ? make_uint4(pair(0, 4), pair(1, 5), pair(2, 6), pair(3, 7))
                : n == 4 ? make_uint4(pair(0, 2), pair(1, 3), pair(4, 6), pair(5, 7))
                         : make_uint4(pair(0, 1), pair(2, 3), pair(4, 5), pair(6, 7));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int s = slot_of(oct * 8 + i, n);
                *reinterpret_cast<__half*>(to + (s >> 3) * pitch + row * 16 + (s & 7) * 2) = __float2half_rn(x[i] * up);
            }
        }
        if (EXACT && part == 0) {
            to += low;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[i] *= up;
                x[i] -= __half2float(__float2half_rn(x[i]));
            }
            up = 1.f;
        }
    }
    return down;
}

__device__ __forceinline__ void load8(const void* src, bool bf16, size_t at, float (&x)[8]) {
    if (bf16) {
        widen(__ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(src) + at)), x);
    } else {
        const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(src) + at);
        const float4 a = __ldg(f), b = __ldg(f + 1);
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
}

// where byte `from` of a row or run lies: `chunk` bytes together (16, or 8 for shorter rows and runs), `pitch` apart
__device__ __forceinline__ int part_offset(int from, int chunk, int pitch) { return from / chunk * pitch + from % chunk; }
// `bytes` (a power of two from 4 to 16 * M) of a row or run
template <int M>
__device__ __forceinline__ void load_part(uint4 (&to)[M], const uint8_t* at, int pitch, int bytes) {
    if (bytes >= 16) {
        to[0] = __ldg(reinterpret_cast<const uint4*>(at));
        if (M >= 2 && bytes >= 32) to[M >= 2 ? 1 : 0] = __ldg(reinterpret_cast<const uint4*>(at + pitch));
        if (M >= 4 && bytes >= 64) {
            to[M >= 4 ? 2 : 0] = __ldg(reinterpret_cast<const uint4*>(at + 2 * pitch));
            to[M >= 4 ? 3 : 0] = __ldg(reinterpret_cast<const uint4*>(at + 3 * pitch));
        }
    } else if (bytes == 8) {
        const uint2 x = __ldg(reinterpret_cast<const uint2*>(at));
        to[0].x = x.x;
        to[0].y = x.y;
    } else {
        to[0].x = __ldg(reinterpret_cast<const uint32_t*>(at));
    }
}

// ---------------------------------------------------------------- keys

__device__ __forceinline__ uint32_t word_of(const uint4& q, int w) { return w == 0 ? q.x : w == 1 ? q.y : w == 2 ? q.z : q.w; }

// half the channels of a position, codes in `raw`, metadata of their groups, to its row of the key tile (LOW bytes further
// what fp16 leaves of them, unless LOW is 0)
template <int BITS, int D, int KG, int LOW>
__device__ __forceinline__ void put_key(const uint4 (&raw)[4], const uint32_t (&meta)[4], unsigned char* to) {
    constexpr int N = 32 / BITS, W = D / 2 / N;          // codes a word, words
    uint32_t out[4], rest[4];
#pragma unroll
    for (int w = 0; w < W; ++w) {
        // groups of the word's low and high codes
        const uint32_t m0 = meta[w * N / KG % 4], m1 = meta[(w * N + N / 2) / KG % 4];
        const __half2 scale = half2_of(__byte_perm(m0, m1, 0x5410)), zero = half2_of(__byte_perm(m0, m1, 0x7632));
        __half2 c[N / 2];
        unpack<BITS>(word_of(raw[w / 4], w % 4), c);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const int s = w * (N / 2) + i;               // pair
            if (LOW) {
                const Split k = split_key(c[i], scale, zero);
                out[s & 3] = k.high, rest[s & 3] = k.low;
            } else {
                out[s & 3] = bits(__hfma2(c[i], scale, zero));
            }
            if ((s & 3) == 3) {
                *reinterpret_cast<uint4*>(to + (s >> 2) * kKeyPitch) = make_uint4(out[0], out[1], out[2], out[3]);
                if (LOW) *reinterpret_cast<uint4*>(to + LOW + (s >> 2) * kKeyPitch) = make_uint4(rest[0], rest[1], rest[2], rest[3]);
            }
        }
    }
}
template <int BITS, int D, int LOW>
__device__ __forceinline__ void put_key_of(int kg, const uint4 (&raw)[4], const uint32_t (&meta)[4], unsigned char* to) {
    if (kg == 16 || LOW)                                 // (single tokens over wider groups take the other kernel)
        put_key<BITS, D, 16, LOW>(raw, meta, to);
    else if (kg == 32 || D == 64)
        put_key<BITS, D, 32, LOW>(raw, meta, to);        // (D = 64: half a row is one group of 32 or part of one of 64)
    else
        put_key<BITS, D, 64, LOW>(raw, meta, to);        // half a row is one group of 64 or half of one of 128
}

// Keys with groups along positions: codes of channels 2*cp (raw[0..1]) and 2*cp + 1 (raw[2..3]) at half the positions of a
// page, 32 from t0 on, to rows of the key tile.  ALL: every one of them lives in the page (a check at each store instead:
// 564 us against 282 for two prompts of 3000 positions).  LOW: as above.
template <int BITS, int D, bool ALL, int LOW>
__device__ __forceinline__ void put_key_pairs(const uint4 (&raw)[4], const uint32_t* meta, int kshift, int t0, int valid, int vn,
                                              unsigned char* to) {
    constexpr int N = 32 / BITS, W = 32 / N;             // codes a word, words a channel
    int step[5];                                         // the slot of a position is the sum over its bits
#pragma unroll
    for (int b = 0; b < 5; ++b) step[b] = slot_of(1 << b, vn) * 16;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        __half2 ca[N / 2], cb[N / 2];
        unpack<BITS>(word_of(raw[w / 4], w % 4), ca);
        unpack<BITS>(word_of(raw[2 + w / 4], w % 4), cb);
        __half2 scale[2], zero[2];                       // of the words' low and high codes' groups
#pragma unroll
        for (int h = 0; h < (N > 16 ? 2 : 1); ++h) {
            const uint2 m = __ldg(reinterpret_cast<const uint2*>(meta + size_t((t0 + w * N + h * (N / 2)) >> kshift) * D));
            scale[h] = half2_of(__byte_perm(m.x, m.y, 0x5410));
            zero[h] = half2_of(__byte_perm(m.x, m.y, 0x7632));
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int h = i >= N / 2, t = w * N + i;
            const __half2 c = half2_of(__byte_perm(bits(ca[i % (N / 2)]), bits(cb[i % (N / 2)]), h ? 0x7632 : 0x5410));
            const Split k = LOW ? split_key(c, scale[N > 16 ? h : 0], zero[N > 16 ? h : 0])
                                : Split{bits(__hfma2(c, scale[N > 16 ? h : 0], zero[N > 16 ? h : 0])), 0u};
            int off = 0;
#pragma unroll
            for (int b = 0; b < 5; ++b)
                if (t & (1 << b)) off += step[b];
            if (ALL || t0 + t < valid) {
                *reinterpret_cast<uint32_t*>(to + off) = k.high;
                if (LOW) *reinterpret_cast<uint32_t*>(to + LOW + off) = k.low;
            }
        }
    }
}

template <int BITS, int D, int LOW>
__device__ __forceinline__ void put_key_pairs_of(const uint4 (&raw)[4], const uint32_t* meta, int kshift, int t0, int valid, int vn,
                                                 unsigned char* to) {
    if (t0 + 32 <= valid)
        put_key_pairs<BITS, D, true, LOW>(raw, meta, kshift, t0, valid, vn, to);
    else
        put_key_pairs<BITS, D, false, LOW>(raw, meta, kshift, t0, valid, vn, to);
}

// half a ring row to its row of the key tile, in the channel order of words of N codes.  LOW: as above.
template <int N, int D, int LOW>
__device__ __forceinline__ void put_ring_key(const __nv_bfloat16* src, unsigned char* to) {
    constexpr int C = N > 8 ? N : 8;                     // channels that are exchanged among themselves
#pragma unroll 2
    for (int c0 = 0; c0 < D / 2; c0 += C) {
        uint32_t u[C / 2];
#pragma unroll
        for (int i = 0; i < C / 8; ++i) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(src + c0) + i);
            u[4 * i] = v.x, u[4 * i + 1] = v.y, u[4 * i + 2] = v.z, u[4 * i + 3] = v.w;
        }
        const auto at = [&](int ch) { return __uint_as_float(ch & 1 ? u[ch / 2] & 0xffff0000u : u[ch / 2] << 16); };
        uint32_t out[C / 2], rest[C / 2];
#pragma unroll
        for (int q = 0; q < C / 2; ++q) {
            const int first = pair_low<N>(q);
            const Split k = LOW ? split2(at(first), at(first + N / 2))
                                : Split{bits(__floats2half2_rn(at(first), at(first + N / 2))), 0u};
            out[q] = k.high, rest[q] = k.low;
        }
#pragma unroll
        for (int i = 0; i < C / 8; ++i) {
            *reinterpret_cast<uint4*>(to + (c0 / 8 + i) * kKeyPitch) =
                make_uint4(out[4 * i], out[4 * i + 1], out[4 * i + 2], out[4 * i + 3]);
            if (LOW)
                *reinterpret_cast<uint4*>(to + LOW + (c0 / 8 + i) * kKeyPitch) =
                    make_uint4(rest[4 * i], rest[4 * i + 1], rest[4 * i + 2], rest[4 * i + 3]);
        }
    }
}

// One bf16 query row, as it came to its place among the queries, to fp16 in the channel order of words of N codes, times
// `sign` and a power of two that brings its largest element into [2^13, 2^14); returns that power's inverse.
template <int N, int D>
__device__ __forceinline__ float turn_query(unsigned char* row, float sign) {
    constexpr int C = N > 8 ? N : 8;                     // channels that are exchanged among themselves
    uint32_t top = 0;                                    // largest magnitude, as bf16 bits in either half
#pragma unroll 4
    for (int k = 0; k < D / 8; ++k) {
        const uint4 v = *reinterpret_cast<const uint4*>(row + k * kQueryPitch);
        top = __vmaxu2(__vmaxu2(top, v.x & 0x7fff7fffu), v.y & 0x7fff7fffu);
        top = __vmaxu2(__vmaxu2(top, v.z & 0x7fff7fffu), v.w & 0x7fff7fffu);
    }
    const int e = max(-100, int(max(top >> 16, top & 0xffffu) >> 7) - 127);
    const float up = sign * __uint_as_float(uint32_t(127 + 13 - e) << 23);
#pragma unroll 2
    for (int k0 = 0; k0 < D / 8; k0 += C / 8) {
        float x[C];
#pragma unroll
        for (int k = 0; k < C / 8; ++k) {
            float y[8];
            widen(*reinterpret_cast<const uint4*>(row + (k0 + k) * kQueryPitch), y);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[8 * k + i] = y[i] * up;
        }
#pragma unroll
        for (int k = 0; k < C / 8; ++k) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int low = pair_low<N>(4 * k + i);
                w[i] = bits(__floats2half2_rn(x[low], x[low + N / 2]));
            }
            *reinterpret_cast<uint4*>(row + (k0 + k) * kQueryPitch) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    return __uint_as_float(uint32_t(127 - 13 + e) << 23);
}

// ---------------------------------------------------------------- values

// half a channel's run of a page to the value tile: pieces of eight slots, D*16 bytes apart
template <int BITS, int D>
__device__ __forceinline__ void put_value(const __half* scale, const __half* zero, const uint4 (&raw)[2], unsigned char* to) {
    constexpr int N = 32 / BITS, W = 32 / N;
    const uint4 *sp = reinterpret_cast<const uint4*>(scale), *zp = reinterpret_cast<const uint4*>(zero);
    uint4 s4, z4, out;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        __half2 c[N / 2];
        unpack<BITS>(word_of(raw[w / 4], w % 4), c);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const int s = w * (N / 2) + i;               // pair
            if ((s & 3) == 0) {
                s4 = sp[s >> 2];
                z4 = zp[s >> 2];
            }
            const uint32_t v = bits(__hfma2(c[i], half2_of(word_of(s4, s & 3)), half2_of(word_of(z4, s & 3))));
            if ((s & 3) == 0) out.x = v;
            if ((s & 3) == 1) out.y = v;
            if ((s & 3) == 2) out.z = v;
            if ((s & 3) == 3) {
                out.w = v;
                *reinterpret_cast<uint4*>(to + (s >> 2) * (D * 16)) = out;
            }
        }
    }
}

// one channel of the ring positions among 32 positions from y0 on, in the order of words of N codes
template <int N, int D, bool SPLIT>
__device__ __forceinline__ void put_ring_value(const Work<SPLIT>& wk, const __nv_bfloat16* win, int R, int y0, unsigned char* to) {
    constexpr int C = N > 16 ? N : 16;                   // positions that are loaded at a time
#pragma unroll 1
    for (int o0 = 0; o0 < 32; o0 += C) {
        if (y0 + o0 + C <= wk.Lq || y0 + o0 > wk.p_max) continue;
        int slot = (y0 + o0) % R;
        __half f[C];
#pragma unroll
        for (int u = 0; u < C; ++u) {
            const int y = y0 + o0 + u;
            f[u] = __float2half_rn(y >= wk.Lq && wk.used(y) ? __bfloat162float(win[size_t(slot) * D]) : 0.f);
            slot = slot + 1 == R ? 0 : slot + 1;
        }
        unsigned char* col = to + o0 / 8 * (D * 16);
        if (y0 + o0 >= wk.Lq) {
#pragma unroll
            for (int k = 0; k < C / 8; ++k) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int low = pair_low<N>(4 * k + e);
                    w[e] = bits(__halves2half2(f[low], f[low + N / 2]));
                }
                *reinterpret_cast<uint4*>(col + k * (D * 16)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        } else {                                         // the page's last positions are among them
#pragma unroll
            for (int u = 0; u < C; ++u) {
                const int s = slot_of(u, N);
                if (y0 + o0 + u >= wk.Lq) *reinterpret_cast<__half*>(col + (s >> 3) * (D * 16) + (s & 7) * 2) = f[u];
            }
        }
    }
}

// ---------------------------------------------------------------- the kernel

// KPC: keys with groups along positions (with both forms of the keys in one build, chunks of 512 at 4096 positions took 752
// to 780 us against 738, as the compiler laid out the loop of the keys).
// EXACT: single tokens, whose scores and lse are to be fp32's as in the other kernel of that call: keys and queries as two fp16
// numbers each, the low parts in the place of the stages 2 and 3 and of block 1's queries, and S = Q K_low (+ Q_low K_high
// where queries are fp32 or rotated) + Q K_high.  (16 sequences, span 4096: 137 us with groups of 16 channels and 164 with
// groups along positions; 95 and 117 with fp16 alone, whose lse was off by 1e-4.)
template <int D, bool SPLIT, bool KPC, bool EXACT>
__global__ void __launch_bounds__(kThreads, 1) sink_prefill_kernel(const __grid_constant__ Params p,
                                                                   const __grid_constant__ Args a, int shared_by, unsigned* status) {
    const int ctas = SPLIT ? shared_by : 1;
    extern __shared__ unsigned char raw_smem[];
    Smem<D>& sm = *reinterpret_cast<Smem<D>*>((reinterpret_cast<uintptr_t>(raw_smem) + 127) & ~uintptr_t(127));
    // (the same in every lane, which the compiler knows after the exchange: operands of the products stay uniform)
    const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x) / 32, 0), lane = threadIdx.x % 32;
    Work<SPLIT> wk;
    wk.b = blockIdx.z;
    wk.h = blockIdx.y;
    Seq sq;
    if (!sequence(a, wk.b, sq)) return;
    const int g = p.g, QT = kRows / g;                    // queries of a block
    wk.rank = SPLIT ? blockIdx.x % ctas : 0;
    wk.ctas = ctas;
    const int i0 = int((gridDim.x - 1 - blockIdx.x) / ctas) * 2 * QT;   // the last queries see the most: first
    if (i0 >= sq.n) return;
    const int nq = min(2 * QT, sq.n - i0);
    const bool two = nq > QT;
    wk.L = sq.L;
    wk.Lq = paged_len(p, KPC, sq.L);
    wk.p_max = sq.base + i0 + nq - 1;
    wk.lo = span_begin(sq.base + i0, a.span);
    wk.sinks = a.sinks;
    // an empty sequence (decode) has no position at all
    wk.n_sink = (min(a.sinks, min(wk.lo, wk.p_max + 1)) + kTile - 1) / kTile;
    wk.first = max(wk.n_sink, wk.lo / kTile);
    const int all_tiles = wk.n_sink + max(0, (wk.p_max + kTile) / kTile - wk.first);
    wk.n_tile = all_tiles > wk.rank ? (all_tiles - wk.rank + ctas - 1) / ctas : 0;
    constexpr int kKeyStages = EXACT ? kStages / 2 : kStages;
    constexpr int kLow = EXACT ? kKeyStages * int(sizeof(sm.k[0])) : 0;   // bytes from a key tile to its low part
    constexpr int kQueryLow = EXACT ? int(sizeof(sm.q[0])) : 0;
    const int kn = KPC ? 2 : 32 / p.kb, vn = 32 / p.vb; // order of the key's channels (2: as they are) and of positions

    // ---- set up ----
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sm.kfull[i], kKeyThreads);
            mbar_init(&sm.vfull[i], kValueThreads);
            mbar_init(&sm.kempty[i], two ? 2 : 1);        // a commit of each block
            mbar_init(&sm.vempty[i], two ? 2 : 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&sm.sfull[i >> 1][i & 1], 1);
            mbar_init(&sm.pfull[i >> 1][i & 1], kRows);
        }
        mbar_init(&sm.odone[0], 1);
        mbar_init(&sm.odone[1], 1);
        mbar_init(&sm.olast[0], 1);
        mbar_init(&sm.olast[1], 1);
        mbar_init(&sm.qfull[0], kRows);
        mbar_init(&sm.qfull[1], kRows);
        sm.failed = 0;
        mbar_fence_init();
    }
    if (warp == 20) {
        tmem_alloc(&sm.tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;                        // S of block 0 (two of 64 columns) and 1, O of block 0 (D columns) and 1

    // A wait that gives up is remembered: every role stops at its next one that is not over at once.  The answer is the
    // warp's.
    auto late = [&](uint32_t bar, int parity) -> bool {
        const uint64_t begin = globaltimer();
        for (;;) {
            if (mbar_try_wait(bar, uint32_t(parity))) return true;
            if (*reinterpret_cast<volatile int*>(&sm.failed)) return false;
            if (globaltimer() - begin > kLimitNs) {
                if (atomicExch(&sm.failed, 1) == 0) atomicAdd(status, 1u);
                return false;
            }
        }
    };
    auto wait = [&](uint64_t* bar, int parity) -> bool {
        const uint32_t at = smem_u32(bar);
        bool done = mbar_try_wait(at, uint32_t(parity));
        if (!done) done = late(at, parity);
        return __all_sync(0xffffffffu, done);
    };

    if (warp < 8) {
        // ------------------------------------------------ weights
        asm volatile("setmaxnreg.inc.sync.aligned.u32 96;");
        const int m = warp >> 2, r = threadIdx.x & 127;
        if (m == 0 || two) {
            const uint32_t lanes = uint32_t(warp & 3) * 32u << 16;
            const uint32_t to = tmem + 256 + m * D + lanes;
            const int q_in = r / g;
            // ---- queries, while the first tiles come in ----
            // (A CTA of a cluster that has no tile has no use for them.  Its warps wait for no product, and so not for each
            // other, before they write their part of the join over the queries' place: nothing else may be written there.)
            const float scale = fabsf(a.scale_log2), sign = a.scale_log2 < 0.f ? -1.f : 1.f;
            float factor = 0.f;
            if (!SPLIT || wk.n_tile > 0) {
                constexpr int kPer = 32 / (D / 8);        // rows of the warp at a time, D/8 lanes each
                const int oct = lane % (D / 8), sub = lane / (D / 8), first = r - lane;
                // each lane knows its own row's place (-1: no such row)
                const bool have = r < QT * g && m * QT + q_in < nq;
                const long long own =
                    have ? (long long)(sq.row + i0 + m * QT + q_in) * a.q_stride + (long long)(wk.h * g + r % g) * D : -1ll;
                if (a.q_bf16) {                           // as they are to their place, all under way at once
                    const uint32_t to = smem_u32(sm.q[m]) + oct * kQueryPitch;
#pragma unroll
                    for (int r0 = 0; r0 < 32; r0 += kPer) {
                        const long long at = __shfl_sync(0xffffffffu, own, r0 + sub);
                        cp16_zfill(to + (first + r0 + sub) * 16, static_cast<const __nv_bfloat16*>(a.q) + (at >= 0 ? at + oct * 8 : 0),
                                   at >= 0);
                    }
                    cp_async_wait_all();
                    __syncwarp();
                }
                if (a.q_bf16 && !p.rotate) {              // in place, each lane its row
                    unsigned char* to = sm.q[m] + r * 16;
                    float down = 1.f;
                    if (kn == 8) down = turn_query<8, D>(to, sign);
                    if (kn == 2) down = turn_query<2, D>(to, sign);
                    if (kn == 4) down = turn_query<4, D>(to, sign);
                    if (kn == 16) down = turn_query<16, D>(to, sign);
                    if (kn == 32) down = turn_query<32, D>(to, sign);
                    factor = scale * down;
                } else {
#pragma unroll 2
                    for (int r0 = 0; r0 < 32; r0 += kPer) {
                        const int rr = first + r0 + sub;
                        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                        if (a.q_bf16) {
                            widen(*reinterpret_cast<const uint4*>(sm.q[m] + oct * kQueryPitch + rr * 16), x);
                        } else {
                            const long long at = __shfl_sync(0xffffffffu, own, r0 + sub);
                            if (at >= 0) load8(a.q, false, size_t(at) + oct * 8, x);
                        }
                        // (its exchanges come after every lane's read and before any lane's store)
                        const float down = put_row<D, EXACT>(x, p.rotate ? p.signs : nullptr, true, sign, sm.q[m], kQueryLow, kQueryPitch, rr, kn);
                        const int from = lane - r0;       // to the lane whose row it is
                        const float v = __shfl_sync(0xffffffffu, down, from >= 0 && from < kPer ? from * (D / 8) : 0);
                        if (from >= 0 && from < kPer) factor = scale * v;
                    }
                }
            }
            factor = fmaxf(factor, 1e-37f);               // (never zero: -inf times it has to stay -inf)
            fence_proxy_async();
            arrive(&sm.qfull[m]);
            const int t = sq.base + i0 + m * QT + min(q_in, QT - 1);
            const int t_first = sq.base + i0 + m * QT, t_last = min(t_first + QT - 1, wk.p_max);
            float ref = kRefNone, l = 0.f;
            bool ok = true;
            for (int j = 0; j < wk.n_tile && ok; ++j) {
                ok = wait(&sm.sfull[m][j & 1], (j >> 1) & 1);
                if (!ok) break;
                tc_fence_after();
                const uint32_t ts = tmem + (m * 2 + (j & 1)) * kTile + lanes;
                uint32_t s[2][32];
                tmem_ld32(ts, s[0]);
                tmem_ld32(ts + 32, s[1]);
                const int t0 = wk.tile_start(j), hidden = *reinterpret_cast<volatile int*>(&sm.hidden[j & 7]);
                // every row of the block sees the whole tile?
                const bool whole = !hidden && t0 + kTile - 1 <= t_first && (t_last - t0 < a.span || t0 + kTile <= a.sinks);
                tmem_loaded(s[0]);
                tmem_loaded(s[1]);
                if (!whole) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        // bit o: position x + o is visible to this row
                        const int x = t0 + 32 * c;
                        uint32_t v = below(t - x + 1) & (~below(max(t - a.span, -1) - x + 1) | below(a.sinks - x));
                        if (hidden) v &= ~below(wk.Lq - x);
                        v = slots_of(v, vn);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!(v & (1u << i))) s[c][i] = 0xff800000u;
                    }
                }
                float mx[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    mx[e] = __uint_as_float(s[e >> 2][(e & 3) * 8]);
#pragma unroll
                    for (int i = 1; i < 8; ++i) mx[e] = fmaxf(mx[e], __uint_as_float(s[e >> 2][(e & 3) * 8 + i]));
                }
                const float need = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7]))) * factor;
                // Weights are taken against the reference of the tiles before.  Should one exceed 2^15, the most that fp16
                // holds (the first tile's always do), the reference is raised and O brought down to it: to 2^8 below the
                // largest weight, which so lies from 2^8 to 2^15.  A weight then keeps 11 bits down to 2^-22 of the largest and
                // counts down to 2^-33, and what a sink leaves to many others is not lost.  (Room above for fewer rises
                // or range below: 16 chunks of 512 at 4096 positions take 756 us with the largest at 2^0, 761 at 2^6,
                // 765 at 2^8, 769 at 2^10.)
                if (__builtin_expect(__any_sync(0xffffffffu, need > ref + kTopWeight), 0)) {
                    const float up = fmaxf(ref, need - kLowTop), f = ex2(ref - up);
                    ref = up;
                    l *= f;
                    if (j > 0) {
                        // (S(j) came after the values of tile j - 2, so the barrier is in phase j - 1 or just past it)
                        ok = wait(&sm.odone[m], (j - 1) & 1);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int e = 0; e < D / 16; ++e) {
                            uint32_t o[16];
                            tmem_ld16(to + e * 16, o);
                            tc_wait_ld();
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tmem_st16(to + e * 16, o);
                        }
                    }
                }
                const uint64_t f2 = pack2(factor, factor), r2 = pack2(-ref, -ref);
                float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    uint32_t* q = &s[i >> 4][2 * (i & 15)];
                    float x, y;
                    unpack2(fma2(pack2(__uint_as_float(q[0]), __uint_as_float(q[1])), f2, r2), x, y);
                    x = ex2(x);
                    y = ex2(y);
                    part[i & 3] += x + y;                 // (before they are rounded: lse is fp32's)
                    s[0][i] = bits(__floats2half2_rn(x, y));   // (slot i has been read)
                }
                tmem_st32(ts, s[0]);                      // over S
                l += (part[0] + part[1]) + (part[2] + part[3]);
                tc_wait_st();
                tc_fence_before();
                arrive(&sm.pfull[m][j & 1]);
            }
            // ---- out ----
            if (ok && wk.n_tile > 0) ok = wait(&sm.olast[m], 0);
            tc_fence_after();
            const int qi = m * QT + q_in;
            const bool mine = r < QT * g && qi < nq;
            const size_t row = (sq.row + i0 + qi) * p.hq + wk.h * g + r % g;
            if (SPLIT) {
                // To this CTA's part of the join, over the operands.  With tiles, every product of both blocks is done by
                // then, and a block's products come after all of its queries and of the tiles that the other warps wrote;
                // without, neither queries nor tiles are written.
                if (ok && wk.n_tile > 0 && two) ok = wait(&sm.olast[1 - m], 0);
                float* part = reinterpret_cast<float*>(sm.q[0]) + (m * kRows + r) * kPartPitch<D>;
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = 0;
                    if (wk.n_tile > 0) {
                        tmem_ld32(to + c * 32, o);
                        tmem_loaded(o);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        reinterpret_cast<uint4*>(part + c * 32)[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                }
                part[D] = ref;
                part[D + 1] = ok ? l : NAN;
            } else {
                const float inv = !ok ? NAN : l != 0.f ? 1.f / l : 0.f;   // (NaN stays)
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = 0;
                    if (wk.n_tile > 0) {
                        tmem_ld32(to + c * 32, o);
                        tmem_loaded(o);
                    }
                    if (mine) {
                        uint4* dst = reinterpret_cast<uint4*>(a.out + row * D + c * 32);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(o[8 * i + 2 * e]) * inv,
                                                                               __uint_as_float(o[8 * i + 2 * e + 1]) * inv);
                                w[e] = *reinterpret_cast<const uint32_t*>(&h);
                            }
                            dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                }
                if (mine && a.lse) a.lse[row] = !ok ? NAN : l != 0.f ? (ref + log2f(l)) * 0.693147180559945309f : -INFINITY;
            }
        }
        if (SPLIT) {   // a warp a row, D/32 channels a lane; the rows are dealt to the CTAs
            cluster_sync();
            namespace cg = cooperative_groups;
            const cg::cluster_group cl = cg::this_cluster();
            constexpr int C = D / 32;
#pragma unroll 1
            for (int k = wk.rank + ctas * warp; k < 2 * kRows; k += ctas * 8) {
                const int mm = k / kRows, rr = k % kRows, qi = mm * QT + rr / g;
                if (rr >= QT * g || qi >= nq) continue;
                float ref[8], sum[8], v[8][C];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float* part = cl.map_shared_rank(reinterpret_cast<float*>(sm.q[0]), i < ctas ? i : 0) + k * kPartPitch<D>;
                    ref[i] = i < ctas ? part[D] : kRefNone;
                    sum[i] = i < ctas ? part[D + 1] : 0.f;
#pragma unroll
                    for (int c = 0; c < C; c += 2) {
                        const float2 x = *reinterpret_cast<const float2*>(part + lane * C + c);
                        v[i][c] = i < ctas ? x.x : 0.f;
                        v[i][c + 1] = i < ctas ? x.y : 0.f;
                    }
                }
                float top = ref[0], l = 0.f, o[C];
#pragma unroll
                for (int i = 1; i < 8; ++i) top = fmaxf(top, ref[i]);
#pragma unroll
                for (int c = 0; c < C; ++c) o[c] = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float f = ex2(ref[i] - top);
                    l = fmaf(sum[i], f, l);
#pragma unroll
                    for (int c = 0; c < C; ++c) o[c] = fmaf(v[i][c], f, o[c]);
                }
                const float inv = l != 0.f ? 1.f / l : 0.f;   // (NaN stays)
                const size_t row = (sq.row + i0 + qi) * p.hq + wk.h * g + rr % g;
#pragma unroll
                for (int c = 0; c < C; c += 2)
                    *reinterpret_cast<__nv_bfloat162*>(a.out + row * D + lane * C + c) = __floats2bfloat162_rn(o[c] * inv, o[c + 1] * inv);
                if (a.lse && lane == 0) a.lse[row] = l != 0.f ? (top + log2f(l)) * 0.693147180559945309f : -INFINITY;
            }
            cluster_sync();                               // no CTA leaves while another reads its part
        }
    } else if (warp < 20) {
        // ------------------------------------------------ keys (warps 8-11), values (12-19)
        const int R = ring_slots(p, KPC);
        // table entry of tile j's page (-1 past what any row sees); looked at a tile later, so nothing waits for it
        auto page_of = [&](int j) -> int {
            if (j >= wk.n_tile) return -1;
            const int lp = wk.tile_start(j) / kPage;
            return lp * kPage < wk.Lq && lp < p.max_pages ? __ldg(p.page_table + size_t(wk.b) * p.max_pages + lp) : -1;
        };
        auto present = [&](int pg) -> int { return pg < p.num_pages ? max(pg, -1) : -1; };
        bool ok = true;
        int pg = present(page_of(0)), pg_next = page_of(1);
        if (warp < 12) {
            asm volatile("setmaxnreg.inc.sync.aligned.u32 112;");
            const int i = threadIdx.x - 256;
            const int half = i >> 6, slot = i & 63;       // kpc: half of the positions, channel pair
            const int run_bytes = kPage * p.kb / 8, ch = min(16, run_bytes), kshift = __ffs(p.kg) - 1;
            uint4 raw[4];
            uint32_t meta[4];
            // this thread's codes and metadata in page 0, and what lies between pages
            const int part = KPC ? run_bytes / 2 : p.krow_bytes / 2, groups = min(4, max(1, D / 2 >> kshift));
            const size_t code_step = size_t(p.hkv) * kPage * p.krow_bytes, meta_step = size_t(p.hkv) * kPage * p.nkg;
            const uint8_t* codes = p.k_codes + size_t(wk.h) * kPage * p.krow_bytes +
                                   (KPC ? 2 * slot * ch + part_offset(half * part, ch, D * 16)
                                          : slot * p.kch + part_offset(half * part, p.kch, kPage * 16));
            // (tokens: groups from that of channel half * D/2 on: D/2 / kg of them, or the one that holds them all)
            const uint32_t* metas = p.k_meta + (size_t(wk.h) * kPage + slot) * p.nkg + (half * (D / 2) >> kshift);
            auto load = [&]() {
                if (pg < 0) return;
                const uint8_t* at = codes + pg * code_step;
                if (KPC) {
                    if (slot >= D / 2) return;
                    uint4 x[2], y[2];
                    load_part<2>(x, at, D * 16, part);
                    load_part<2>(y, at + ch, D * 16, part);
                    raw[0] = x[0], raw[1] = x[1], raw[2] = y[0], raw[3] = y[1];
                } else {
                    load_part<4>(raw, at, kPage * 16, part);
                    const uint32_t* m = metas + pg * meta_step;
                    meta[0] = __ldg(m);
                    if (groups >= 2) meta[1] = __ldg(m + 1);
                    if (groups >= 4) {
                        meta[2] = __ldg(m + 2);
                        meta[3] = __ldg(m + 3);
                    }
                }
            };
            load();
#pragma unroll 1
            for (int j = 0; j < wk.n_tile; ++j) {
                const int st = j % kKeyStages, t0 = wk.tile_start(j), x = t0 + slot;
                if (j >= kKeyStages) ok = wait(&sm.kempty[st], (j / kKeyStages + 1) & 1);
                if (!ok) break;
                unsigned char* sk = sm.k[st];
                unsigned char* row = sk + slot_of(slot, vn) * 16 + half * (D / 16) * kKeyPitch;
                if (KPC) {
                    if (slot < D / 2 && pg >= 0) {
                        const uint32_t* m = p.k_meta + (size_t(pg) * p.hkv + wk.h) * size_t(kPage >> kshift) * D + 2 * slot;
                        unsigned char* col = sk + (slot >> 2) * kKeyPitch + (slot & 3) * 4 + half * (32 * 16);
                        if (p.kb == 4) put_key_pairs_of<4, D, kLow>(raw, m, kshift, half * 32, wk.Lq - t0, vn, col);
                        if (p.kb == 8) put_key_pairs_of<8, D, kLow>(raw, m, kshift, half * 32, wk.Lq - t0, vn, col);
                        if (p.kb == 2) put_key_pairs_of<2, D, kLow>(raw, m, kshift, half * 32, wk.Lq - t0, vn, col);
                        if (p.kb == 1) put_key_pairs_of<1, D, kLow>(raw, m, kshift, half * 32, wk.Lq - t0, vn, col);
                    }
                } else if (pg >= 0 && x < wk.Lq) {
                    if (p.kb == 4) put_key_of<4, D, kLow>(p.kg, raw, meta, row);
                    if (p.kb == 8) put_key_of<8, D, kLow>(p.kg, raw, meta, row);
                    if (p.kb == 2) put_key_of<2, D, kLow>(p.kg, raw, meta, row);
                    if (p.kb == 1) put_key_of<1, D, kLow>(p.kg, raw, meta, row);
                }
                __syncwarp();
                if (t0 + kTile > wk.Lq && !p.rotate) {    // ring rows
                    if (x >= wk.Lq && x < wk.L) {
                        const __nv_bfloat16* src = p.k_win + ((size_t(wk.b) * p.hkv + wk.h) * R + x % R) * D + half * (D / 2);
                        if (kn == 8) put_ring_key<8, D, kLow>(src, row);
                        if (kn == 2) put_ring_key<2, D, kLow>(src, row);
                        if (kn == 4) put_ring_key<4, D, kLow>(src, row);
                        if (kn == 16) put_ring_key<16, D, kLow>(src, row);
                        if (kn == 32) put_ring_key<32, D, kLow>(src, row);
                    }
                } else if (t0 + kTile > wk.Lq) {          // rotated first: D/8 lanes a row, two loads under way at a time
                    constexpr int kPer = 32 / (D / 8);
                    const int oct = lane % (D / 8);
#pragma unroll 1
                    for (int s0 = (warp - 8) * 16; s0 < (warp - 8) * 16 + 16; s0 += 2 * kPer) {
                        if (t0 + s0 + 2 * kPer <= wk.Lq || t0 + s0 >= wk.L) continue;
                        float f[2][8];
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const int y = t0 + s0 + u * kPer + lane / (D / 8);
#pragma unroll
                            for (int e = 0; e < 8; ++e) f[u][e] = 0.f;
                            if (y >= wk.Lq && y < wk.L)
                                load8(p.k_win, true, ((size_t(wk.b) * p.hkv + wk.h) * R + y % R) * D + oct * 8, f[u]);
                        }
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const int s = s0 + u * kPer + lane / (D / 8), y = t0 + s;
                            put_row<D, EXACT>(f[u], p.signs, false, 1.f, y >= wk.Lq && y < wk.L ? sk : nullptr, kLow, kKeyPitch, slot_of(s, vn),
                                              kn);
                        }
                    }
                }
                if (i == 0) sm.hidden[j & 7] = pg < 0 && t0 < wk.Lq;
                fence_proxy_async();
                arrive(&sm.kfull[st]);
                pg = present(pg_next);
                load();
                pg_next = page_of(j + 2);
            }
        } else {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
            const int i = threadIdx.x - 384, vrun = p.vchan_bytes;
            const int ch = i & (D - 1), gi = ch / p.vg, half = (i / D) & 1;  // channel, half of the positions
            const bool active = i < 2 * D;
            const int position = i & 63, g0 = i >> 6;     // metadata: position, groups g0 and g0 + 4
            const int at = slot_of(position, vn);
            uint4 raw[2];
            uint32_t meta[2];
            const size_t code_step = size_t(p.hkv) * D * vrun, meta_step = size_t(p.hkv) * kPage * p.nvg;
            const uint8_t* codes = p.v_codes + size_t(wk.h) * D * vrun + ch * p.vch + part_offset(half * (vrun / 2), p.vch, D * 16);
            const uint32_t* metas = p.v_meta + (size_t(wk.h) * kPage + position) * p.nvg + g0;
            auto load = [&](int j) {
                raw[0] = raw[1] = make_uint4(0, 0, 0, 0);
                meta[0] = meta[1] = 0;
                if (pg < 0) return;
                if (active) load_part<2>(raw, codes + pg * code_step, D * 16, vrun / 2);
                const int y = wk.tile_start(j) + position;
                if (g0 < p.nvg && y < wk.Lq && wk.used(y)) {
                    const uint32_t* m = metas + pg * meta_step;
                    meta[0] = __ldg(m);
                    if (g0 + 4 < p.nvg) meta[1] = __ldg(m + 4);
                }
            };
            load(0);
#pragma unroll 1
            for (int j = 0; j < wk.n_tile; ++j) {
                const int st = j % kStages, y0 = wk.tile_start(j) + half * 32;
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (g0 + 4 * e < p.nvg) {
                        sm.vscale[j & 1][g0 + 4 * e][at] = __ushort_as_half(uint16_t(meta[e]));
                        sm.vzero[j & 1][g0 + 4 * e][at] = __ushort_as_half(uint16_t(meta[e] >> 16));
                    }
                if (j >= kStages) ok = wait(&sm.vempty[st], (j / kStages + 1) & 1);
                {   // the metadata is there (the other tile's may still be read); and do all the warps go on?
                    uint32_t all;
                    asm volatile(
                        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
                        "barrier.cta.red.and.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}\n"
                        : "=r"(all)
                        : "r"(uint32_t(ok)), "n"(kValueThreads)
                        : "memory");
                    ok = all != 0;
                    if (!ok) break;
                }
                if (active) {
                    unsigned char* to = sm.v[st] + ch * 16 + half * 4 * (D * 16);
                    const __half *vs = &sm.vscale[j & 1][gi][half * 32], *vz = &sm.vzero[j & 1][gi][half * 32];
                    if (p.vb == 2) put_value<2, D>(vs, vz, raw, to);
                    if (p.vb == 4) put_value<4, D>(vs, vz, raw, to);
                    if (p.vb == 8) put_value<8, D>(vs, vz, raw, to);
                    if (p.vb == 1) put_value<1, D>(vs, vz, raw, to);
                    if (y0 + 32 > wk.Lq && wk.Lq < wk.L) {   // ring positions (the page's codes gave zeros there)
                        const __nv_bfloat16* win = p.v_win + (size_t(wk.b) * p.hkv + wk.h) * R * D + ch;
                        if (p.vb == 2) put_ring_value<16, D>(wk, win, R, y0, to);
                        if (p.vb == 4) put_ring_value<8, D>(wk, win, R, y0, to);
                        if (p.vb == 8) put_ring_value<4, D>(wk, win, R, y0, to);
                        if (p.vb == 1) put_ring_value<32, D>(wk, win, R, y0, to);
                    }
                }
                fence_proxy_async();
                arrive(&sm.vfull[st]);
                pg = present(pg_next);
                load(j + 1);
                pg_next = page_of(j + 2);
            }
        }
    } else {
        // ------------------------------------------------ products
        asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
        const int m = warp - 20;
        // One thread a block (two warps, so two schedulers): a hand-over then costs a dozen instructions, and the
        // instructions around a product, not the tensor core, are what limits a thread.
        if (m < (two ? 2 : 1) && wk.n_tile > 0 && elected()) {
            constexpr uint32_t kS = idesc_f16(kRows, kTile), kO = idesc_f16(kRows, D);
            const uint64_t qd = smem_desc(smem_u32(sm.q[m]), kQueryPitch, 128);
            const uint64_t kd = smem_desc(smem_u32(sm.k[0]), kKeyPitch, 128), vd = smem_desc(smem_u32(sm.v[0]), D * 16, 128);
            constexpr int kKStep = int(sizeof(sm.k[0])) >> 4, kVStep = int(sizeof(sm.v[0])) >> 4;
            const uint32_t d = tmem + 256 + m * D;
            auto reached = [&](uint64_t* bar, int parity) -> bool {
                const uint32_t at = smem_u32(bar);
                return mbar_try_wait(at, uint32_t(parity)) || late(at, parity);
            };
            bool ok = reached(&sm.qfull[m], 0);
            // S of the first two tiles, then for each tile: O += P V, S of the tile after the next
#pragma unroll 1
            for (int j = -2; j < wk.n_tile && ok; ++j) {
                const int ahead = j + 2, vs = j & (kStages - 1), ks = ahead & (kKeyStages - 1);
                const uint32_t tile = tmem + (m * 2 + (j & 1)) * kTile;
                if (j >= 0) {
                    ok = reached(&sm.vfull[vs], (j / kStages) & 1) && reached(&sm.pfull[m][j & 1], (j >> 1) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t v = vd + uint64_t(vs * kVStep);
                    if (j == 0)
                        mma_ts<false>(d, tile, v, kO);
                    else
                        mma_ts<true>(d, tile, v, kO);
#pragma unroll
                    for (int s = 1; s < kTile / 16; ++s) mma_ts<true>(d, tile + s * 8, v + s * (2 * D * 16 >> 4), kO);
                    // (Only barriers that someone waits for: an arrival at one that nobody does could come after the CTA's end.)
                    commit(j + 1 == wk.n_tile ? &sm.olast[m] : &sm.odone[m]);
                    if (j + kStages < wk.n_tile) commit(&sm.vempty[vs]);
                }
                if (ahead >= wk.n_tile) continue;
                ok = reached(&sm.kfull[ks], (ahead / kKeyStages) & 1);
                if (!ok) break;
                tc_fence_after();
                const uint64_t k = kd + uint64_t(ks * kKStep);
                const auto product = [&](uint64_t qa, uint64_t kb) {
#pragma unroll
                    for (int s = 1; s < D / 16; ++s) mma_ss<true>(tile, qa + s * (2 * kQueryPitch >> 4), kb + s * (2 * kKeyPitch >> 4), kS);
                };
                if (EXACT) {                              // the low parts first: their sums are small, and so is what is cut off them
                    mma_ss<false>(tile, qd, k + (kLow >> 4), kS);
                    product(qd, k + (kLow >> 4));
                    if (!a.q_bf16 || p.rotate) {
                        mma_ss<true>(tile, qd + (kQueryLow >> 4), k, kS);
                        product(qd + (kQueryLow >> 4), k);
                    }
                    mma_ss<true>(tile, qd, k, kS);
                } else {
                    mma_ss<false>(tile, qd, k, kS);
                }
                product(qd, k);
                commit(&sm.sfull[m][j & 1]);
                if (ahead + kKeyStages < wk.n_tile) commit(&sm.kempty[ks]);
            }
        }
    }
    if (SPLIT && warp >= 8) {
        __syncwarp();
        cluster_sync();
        cluster_sync();
    }
    // every product has been waited for by the weights' warps, or the waits have given up
    tc_fence_before();
    __syncthreads();
    if (warp == 20) tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t launch_d(const Params& p, const Args& a, int sms, unsigned* status, cudaStream_t s) {
    static std::atomic<bool> opted[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    constexpr int kBytes = int(sizeof(Smem<D>)) + 128;
    if (!opted[dev]) {
        for (auto* kernel : {sink_prefill_kernel<D, false, false, false>, sink_prefill_kernel<D, true, false, false>,
                             sink_prefill_kernel<D, false, true, false>, sink_prefill_kernel<D, true, true, false>,
                             sink_prefill_kernel<D, false, false, true>, sink_prefill_kernel<D, true, false, true>,
                             sink_prefill_kernel<D, false, true, true>, sink_prefill_kernel<D, true, true, true>}) {
            const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
            if (e != cudaSuccess) return e;
        }
        opted[dev] = true;
    }
    static_assert(2 * kRows * kPartPitch<D> * 4 <= int(offsetof(Smem<D>, vscale)), "a join's part lies over the operands");
    const int per = 2 * (kRows / p.g), blocks = (a.max_q - 1) / per + 1;
    // CTAs that share the tiles of a block of rows: as many as there are SMs for, with four tiles each at least if a
    // sequence fills the page table.  (Lengths are on the device: a shorter sequence leaves some without a tile and joins
    // empty parts.  Eight kv-heads, 100 positions: 33 queries take 18 us and 100 queries 38 under a table of 512 pages, 12
    // and 13 under one of 2 pages, where nothing is shared.)
    const long long cached = std::min<long long>((long long)p.max_pages * kPage + ring_slots(p, a.kpc), a.len_cap);
    const long long tiles = std::min(cached, (long long)a.sinks + a.span + per + 2 * kPage) / kTile;
    const long long all = (long long)blocks * p.hkv * p.batch;
    int ctas = 1;
    while (ctas < 8 && all * ctas * 2 <= sms && tiles >= 4 * ctas * 2) ctas *= 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(blocks * ctas, p.hkv, p.batch);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kBytes;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ctas;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = ctas > 1 ? 1 : 0;
    auto* kernel = !a.cu_q ? a.kpc ? ctas > 1 ? sink_prefill_kernel<D, true, true, true> : sink_prefill_kernel<D, false, true, true>
                             : ctas > 1 ? sink_prefill_kernel<D, true, false, true> : sink_prefill_kernel<D, false, false, true>
                   : a.kpc ? ctas > 1 ? sink_prefill_kernel<D, true, true, false> : sink_prefill_kernel<D, false, true, false>
                           : ctas > 1 ? sink_prefill_kernel<D, true, false, false> : sink_prefill_kernel<D, false, false, false>;
    return cudaLaunchKernelEx(&cfg, kernel, p, a, ctas, status);
}

}  // namespace

cudaError_t launch_prefill(const Params& p, const Args& a, int sms, unsigned* status, cudaStream_t s) {
    return p.d == 128 ? launch_d<128>(p, a, sms, status, s) : launch_d<64>(p, a, sms, status, s);
}

}  // namespace sink
}  // namespace kvq
