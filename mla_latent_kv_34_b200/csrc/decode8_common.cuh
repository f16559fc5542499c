// What the two attend kernels of the 8-bit cache share: the split of the (sequence, tile) space into pieces, the
// block lookup, and the two-term e4m3 form of queries and probabilities.
//
// Two terms.  The tensor cores multiply 8-bit values, so the codes of the cache go into them as they stand.  The other
// operand, a bf16 query or an fp32 probability, is written as hi + lo: hi (e4m3) holds 4 significant bits, lo what is
// left.  For the query lo is e4m3 too, the next 4 bits: a bf16 value (8 significant bits) is held exactly as long as its
// last bit is at least 2^-9 (the e4m3 step near 0); scaled by a power of two so that the row's largest value lies in
// (224, 448], that is every element down to 2^-10 of the largest, and an absolute 2^-19 of the largest below.
#pragma once

#include <cuda_fp16.h>

#include "mla_internal.cuh"
#include "sm100.cuh"

namespace mla {
namespace d8 {

using namespace sm100;

constexpr uint64_t kLimitNs = 2000000000ull;  // 2 s per wait
constexpr int kTile = kBlockTokens;
constexpr int kCopyA = 2 * kBlock8Chunk;                        // latent chunks 0, 1: 32 KB
constexpr int kCopyB = 2 * kBlock8Chunk + kBlockTokens * kDr;   // latent chunks 2, 3 and the RoPE columns: 40 KB
constexpr int kTileBytes = kCopyA + kCopyB;                     // codes of a block, contiguous in it
static_assert(kTileBytes == kBlock8Scales, "a block's codes are its first bytes");

struct Params {
    const uint16_t* q;
    const uint8_t* cache;
    const int32_t* block_table;
    const int32_t* kv_len;
    float* o_part;
    float4* ml_part;  // a piece's R, sum of P' / s, the same sum of P' as the MMAs have it
    int32_t* dev_status;
    int64_t cap_blocks;
    int max_blocks;
    int B, n_q, H, R, G, P_g, slots, rs;
    float scale_log2;
};

__device__ __forceinline__ int seq_tiles(const Params& p, int b) {
    return valid_seq_tiles(p.kv_len[b], p.n_q, p.max_blocks);
}

struct Seg {
    int b, t0, t1, L, slot;
    const int32_t* tab;  // the sequence's row of the block table
};

// Pool block of a table entry; one outside the pool is reported and replaced by block 0 (that sequence's result is
// then unspecified, but no access leaves the pool).
__device__ __forceinline__ const uint8_t* block_of(const Params& p, int32_t e, bool report_it) {
    if (e < 0 || e >= p.cap_blocks) {
        if (report_it) report(p.dev_status, MLA_DEVERR_ROW_RANGE);
        e = 0;
    }
    return p.cache + static_cast<int64_t>(e) * kBlock8Bytes;
}

// Walks the segments of one work unit's tile range [lo, hi), starting at sequence b whose first tile has global
// index tb.
struct SegWalk {
    int b, tb, lo, hi, pidx;
    __device__ bool next(const Params& p, Seg& s) {
        while (b < p.B && tb < hi) {
            const int nt = seq_tiles(p, b);
            const int cb = b, ctb = tb;
            tb += nt;
            ++b;
            const int a = max(lo, ctb), e = min(hi, ctb + nt);
            if (a < e) {
                s.b = cb;
                s.t0 = a - ctb;
                s.t1 = e - ctb;
                s.L = p.kv_len[cb];
                s.tab = p.block_table + static_cast<int64_t>(cb) * p.max_blocks;
                s.slot = cb + pidx;
                return true;
            }
        }
        return false;
    }
};

// One warp: total tiles, and (by a warp scan) the sequence that holds the first tile of work unit pidx of P_g; the
// first block of the grid reports sequences that are not processed.  out: [total, first sequence, its first tile].
__device__ __forceinline__ void find_first(const Params& p, int pidx, int lane, int* out) {
    int s = 0;
    for (int b = lane; b < p.B; b += 32) {
        s += seq_tiles(p, b);
        if (blockIdx.x == 0) {
            const int L = p.kv_len[b];
            if (L < p.n_q) report(p.dev_status, MLA_DEVERR_KV_LEN);
            else if (seq_tiles(p, b) == 0) report(p.dev_status, MLA_DEVERR_ROW_RANGE);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const int lo = static_cast<int>((static_cast<int64_t>(pidx) * s) / p.P_g);
    int b0 = p.B, tb0 = s, run = 0;
    for (int base = 0; base < p.B; base += 32) {
        const int b = base + lane;
        const int nt = b < p.B ? seq_tiles(p, b) : 0;
        int inc = nt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, b < p.B && run + inc > lo);
        if (hit) {
            const int f = __ffs(hit) - 1;
            b0 = base + f;
            tb0 = run + __shfl_sync(0xffffffffu, inc - nt, f);
            break;
        }
        run += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) {
        out[0] = s;
        out[1] = b0;
        out[2] = tb0;
    }
}

// Exponent a of a query row whose largest magnitude has bf16 bits `top`: 2^a is the least power of two (>= 2^-120)
// with largest <= 448 * 2^a.  0 for a row of zeros.
__device__ __forceinline__ int row_exp(uint32_t top) {
    if (top == 0) return 0;
    return max(static_cast<int>(top >> 7) - 127 - 8 + ((top & 0x7Fu) > 0x60u ? 1 : 0), -120);
}
__device__ __forceinline__ float exp2_int(int k) { return __uint_as_float(static_cast<uint32_t>(127 + k) << 23); }

// Two packed bf16 times inv (a power of two; magnitudes at most 448) -> hi and lo codes, two each.  The scaled value is
// exact in fp16 down to steps of 2^-24, far below e4m3's 2^-9.
__device__ __forceinline__ void split2_q(uint32_t w, float inv, uint16_t& hi, uint16_t& lo) {
    const float x0 = __uint_as_float(w << 16) * inv, x1 = __uint_as_float(w & 0xFFFF0000u) * inv;
    uint32_t h, d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(x1), "f"(x0));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(hi) : "r"(h));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(h), "r"(e4m3x2_to_f16x2(hi)));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(lo) : "r"(d));
}

// Four packed bf16 -> a word of hi codes and a word of lo codes.
__device__ __forceinline__ void split4_q(uint32_t w0, uint32_t w1, float inv, uint32_t& hi, uint32_t& lo) {
    uint16_t h0, l0, h1, l1;
    split2_q(w0, inv, h0, l0);
    split2_q(w1, inv, h1, l1);
    hi = h0 | (static_cast<uint32_t>(h1) << 16);
    lo = l0 | (static_cast<uint32_t>(l1) << 16);
}

// Two packed bf16 as fp32.
__device__ __forceinline__ float2 bf16x2_f32(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// Packed fp32 arithmetic (two lanes an instruction).
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 c, a, b;\n\t"
        "mov.b64 {%0, %1}, c;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 c, a, b;\n\t"
        "mov.b64 {%0, %1}, c;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}

// Four probabilities 0 <= p <= 2^8.75 of 8 significant bits (a bf16's) as hi (e4m3) and lo (e5m2) codes.  hi rounds to
// nearest; what it leaves, at most 8 units of the last bit, has 3 significant bits, which e5m2 holds: exact down to
// p = 2^-6.  Below, hi's steps are 2^-9 and lo goes on to 2^-16, and many equal small probabilities (a long tail behind one
// dominant token) would move their sum by up to an eighth if each were rounded to nearest.  So lo's rounding is dithered
// over the tokens, which keeps the sum: e5m2 is the upper half of an fp16, the dither is added to the lower byte before it
// is cut off, and changes nothing where that byte is 0.
__device__ __forceinline__ void split4_p(float p0, float p1, float p2, float p3, uint32_t dither01, uint32_t dither23,
                                         uint32_t& hi, uint32_t& lo) {
    uint32_t h01, h23, d01, d23;
    uint16_t a, b;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h01) : "f"(p1), "f"(p0));
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h23) : "f"(p3), "f"(p2));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(a) : "r"(h01));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(b) : "r"(h23));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d01) : "r"(h01), "r"(e4m3x2_to_f16x2(a)));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d23) : "r"(h23), "r"(e4m3x2_to_f16x2(b)));
    hi = a | (static_cast<uint32_t>(b) << 16);
    lo = __byte_perm(d01 + dither01, d23 + dither23, 0x7531);
}
// The same, for any p, with lo * 2^4 in e4m3, for accumulators that keep the lo part in columns of their own: 4 significant
// bits down to 2^-10 and steps of 2^-13 below.  With the one bit more, a dithered rounding (`dither`: seven bits for each half)
// of a probability down to 2^-5 still holds it within 2^-8.  An e4m3 code of x has the bits of the fp16 of 2^-8 x, less its top
// exponent bit and its last seven.
__device__ __forceinline__ void split4_p16(float p0, float p1, float p2, float p3, uint32_t dither, uint32_t& hi,
                                           uint32_t& lo) {
    uint32_t h01, h23, d01, d23;
    uint16_t a, b;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h01) : "f"(p1), "f"(p0));
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h23) : "f"(p3), "f"(p2));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(a) : "r"(h01));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(b) : "r"(h23));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d01) : "r"(h01), "r"(e4m3x2_to_f16x2(a)));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d23) : "r"(h23), "r"(e4m3x2_to_f16x2(b)));
    asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(d01) : "r"(0x2C002C00u));  // 2^-4
    asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(d23) : "r"(0x2C002C00u));
    d01 += dither;
    d23 += dither;
    hi = a | (static_cast<uint32_t>(b) << 16);
    lo = __byte_perm(((d01 << 1) & 0x7F007F00u) | (d01 & 0x80008000u), ((d23 << 1) & 0x7F007F00u) | (d23 & 0x80008000u), 0x7531);
}
// The dither of token `tok` of tile t is an eight-bit number, base(tok % 16) + mask(tok / 16, t), the base a multiple of 16 and
// the mask below it: the 256 tokens of two tiles have each of the 256 values once, so that even equal probabilities keep
// their sum down to 2^-24 (dithers of 16 levels, the same in every tile, lost whole tails of equal probabilities below 2^-20).
__host__ __device__ constexpr uint32_t rev4(uint32_t k) { return (k & 1) << 3 | (k & 2) << 1 | (k & 4) >> 1 | (k & 8) >> 3; }
// base of tokens 2 k and 2 k + 1 of a run of 16, one in each half's lower byte.
__host__ __device__ constexpr uint32_t dither_pair(int k) { return rev4(2 * k) << 4 | rev4(2 * k + 1) << 20; }
// mask of run g (of 8) of tile t, in both halves.
__device__ __forceinline__ uint32_t dither_mask(int g, int t) {
    return rev4(static_cast<uint32_t>(g)) * 0x00010001u + (static_cast<uint32_t>(t) & 1u) * 0x00010001u;
}

// The reference exponent of a row's probabilities, P' = 2^(y - R) with y = log2(p s_t) (s_t, the token's scale, is
// folded into P because V's rows are codes).  O and the sums are kept relative to R, an integer, so moving it multiplies
// them by an exact power of two.  The terms' steps are absolute (2^-16 and 2^-13), P' has to stay below 448, and one token
// may be far above tens of thousands that share the rest of the sum.  So the largest P' belongs near the top, where the
// steps are 2^-21 of it and less; but a row whose first units are its first of many alike needs room to rise, since every
// move costs the whole tile a pass over O.  A row's units (the tokens whose largest y is known at once) follow one another:
//   first  its largest P' goes to (2^(First - 1), 2^First];
//   up     when a unit's largest y passes R + 8.75 (kRoom): its largest P' goes to (2^(Up - 1), 2^Up];
//   down   when the largest P' of two units running (two of the same warp's turns, R the same at both) lies below 2^-Low, what
//          set R was a peak: R moves down, First powers of two below the larger one, but only until the peak is at 2^Up;
//   eager  (TileAsks) the first such unit moves R, at most 2^kLift below the highest R of the piece: O and the sums,
//          P' / s with s >= 2^-40 among them, then stay finite in fp32, and what is lost is below 2^-kLift of the largest.
// With R fixed at the first unit's largest P' in (1, 2], 32 K tokens 2^9 below the first cost 0.007 of the result in the 2-norm
// (0.013 with the 2^-13 steps), and 0.03 (0.07) where the first token's scale was 8 times theirs; now 0.004 at most.
constexpr uint32_t kMinusInf = 0xFF800000u;
constexpr float kNoRef = -3.402823466e38f;  // no reference yet: the lowest float; y - kNoRef is -inf where y is
constexpr uint32_t kNoTile = 0xFFFFFFFEu;
struct LowUnit {  // a warp's last low unit of a row: its largest y, its tile (counted over the work unit; kNoTile: none)
    float top;
    uint32_t at;
};
// A row's scale covers its RoPE columns, and is 1 for a row of zeros, so a token may have a large y and add little or nothing to
// O, while the others in its unit are held in steps set by it.  So one warp looks at the rows ahead of the softmax: at 16 of
// each token's latent codes, and at all of them where those are below 448 * 2^-3.8.
//   lift   m, for tokens whose latent codes are small beside the largest in the tile: the power of two by which they may be
//          multiplied, up to 2^15.  In the aggregation such a token's codes are multiplied by 2^m (exactly; in shared memory) and its
//          scale divided by it.  A token whose latents are all zero has m = kZeroLift, and no codes to multiply.
//   eager  what set R may have been large by its scale alone: tokens are lifted, or were in the tile before, or its latents were
//          all small against their scales, or the scales have fallen by 2^4 since this last was so.  Low units move R at once.
// 511 rows of standard deviation a and one of zeros in their midst lost 0.06 of the result at a = 0.01, all of it at 1e-5.
constexpr float kRoom = 8.75f;
constexpr int kFar = 4;
constexpr int kMostLift = 15, kZeroLift = 40;
struct TileAsks {
    uint32_t lift, eager;
};
constexpr int kNoLatent = -99;
constexpr uint32_t kNoScale = 0x0D800000u;  // 2^-100, for tokens that do not exist (their scores are masked)
// The exponent of a token's largest latent code against 448 (kNoLatent: all are zero), by one thread of a warp that takes
// 32 rows in order: `row` is the token's, r its index.
__device__ __forceinline__ int latent_exp(const uint8_t* row, int r) {
    uint32_t m = 0;
#pragma unroll 8
    for (int u = 0; u < 32; ++u) {  // (each lane its own unit of a column block: no two of eight lanes meet in a bank)
        const uint4 x = *reinterpret_cast<const uint4*>(row + (u >> 3) * kBlock8Chunk + (((u + r) & 7) << 4));
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m = __vmaxu2(m, w[i] & 0x7F007F00u);
            m = __vmaxu2(m, (w[i] << 8) & 0x7F007F00u);
        }
    }
    const uint32_t top = max((m >> 8) & 0x7Fu, m >> 24);
    // (0x7E is 448)
    return top == 0 ? kNoLatent : min(static_cast<int>(top >> 3) - 15 + ((top & 7u) == 7u ? 1 : 0), 0);
}
// 16 codes with 0 for NaN, in place: a token that some query of the step does not see has P = 0 there, and 0 * NaN would
// reach it; the queries that see it have a NaN score.
__device__ __forceinline__ void nan_to_zero16(uint8_t* at) {
    uint4 x = *reinterpret_cast<const uint4*>(at);
    uint32_t w[4] = {x.x, x.y, x.z, x.w}, any = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t n = ((w[i] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;  // the top bit of each byte that is NaN
        any |= n;
        w[i] &= ~((n >> 7) * 0xFFu);
    }
    if (any) *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
}
// For rows first .. last - 1 of a tile, by a warp; for one row, by a thread.  (Not inlined: seldom needed, and the loops that call
// them fill the instruction cache.)
static __device__ __noinline__ void nan_to_zero_rows(uint8_t* tile, int first, int last, int lane) {
    uint8_t* at = tile + (lane >> 3) * kBlock8Chunk + (lane & 7) * 16;
    uint32_t any = 0;
#pragma unroll 8
    for (int r = first; r < last; ++r) {
        const uint4 x = *reinterpret_cast<const uint4*>(at + r * 128);
        any |= ((x.x & 0x7F7F7F7Fu) + 0x01010101u) | ((x.y & 0x7F7F7F7Fu) + 0x01010101u) | ((x.z & 0x7F7F7F7Fu) + 0x01010101u) |
               ((x.w & 0x7F7F7F7Fu) + 0x01010101u);
    }
    if ((any & 0x80808080u) == 0) return;
    for (int r = first; r < last; ++r) nan_to_zero16(at + r * 128);
}
static __device__ __noinline__ void nan_to_zero_row(uint8_t* row) {
#pragma unroll 1
    for (int u = 0; u < 32; ++u) nan_to_zero16(row + (u >> 3) * kBlock8Chunk + (u & 7) * 16);
}

// 16 codes times 2^m, in place (no result passes 448).
__device__ __forceinline__ void lift16(uint8_t* at, uint32_t pow2_f16x2) {
    const uint4 x = *reinterpret_cast<const uint4*>(at);
    uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h[2];
        uint16_t c[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(h[k]) : "r"(e4m3x2_to_f16x2(static_cast<uint16_t>(w[i] >> (16 * k)))), "r"(pow2_f16x2));
            asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c[k]) : "r"(h[k]));
        }
        w[i] = c[0] | static_cast<uint32_t>(c[1]) << 16;
    }
    *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
}
// A token's row of latent codes times 2^m, by a thread.
static __device__ __noinline__ void lift_row(uint8_t* row, int m) {
    if (m < 1 || m > kMostLift) return;
    const uint32_t p = static_cast<uint32_t>(15 + m) << 10;
#pragma unroll 1
    for (int u = 0; u < 32; ++u) lift16(row + (u >> 3) * kBlock8Chunk + (u & 7) * 16, p | p << 16);
}

// Bit i: of 16 codes of token 32 i + lane none is 2^5 = 448 * 2^-3.8 or more (the upper two exponent bits are not both set).
__device__ __forceinline__ uint32_t small_tokens(const uint8_t* codes, int n, int lane) {
    const uint8_t* at = codes + lane * 128;
    uint32_t small = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // units that spread over the banks, and over the columns
        const uint4 x = *reinterpret_cast<const uint4*>(at + i * 4096 + (((lane + (lane >> 3) + 4 * i) & 7) << 4));
        const uint32_t m = (x.x & (x.x << 1)) | (x.y & (x.y << 1)) | (x.z & (x.z << 1)) | (x.w & (x.w << 1));
        if ((m & 0x40404040u) == 0 && 32 * i + lane < n) small |= 1u << i;
    }
    return small;
}
// The lifts of tokens 32 i + lane of a tile (byte i of the first; 0 for those not in `small`); the second: whether any is lifted (1),
// whether all latents are small (2).
static __device__ __noinline__ uint2 tile_lifts(const uint8_t* codes, int n, uint32_t small, int lane) {
    int f[4], g = kNoLatent;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 32 * i + lane;
        f[i] = 0;
        if (__any_sync(0xffffffffu, (small >> i & 1u) != 0)) {
            const int e = latent_exp(codes + r * 128, r);
            if (small >> i & 1u) f[i] = e;
        }
        if (r < n) g = max(g, f[i]);
    }
    g = __reduce_max_sync(0xffffffffu, g);
    uint32_t lifts = 0;
    bool use = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int m = f[i] == kNoLatent ? kZeroLift : min(g - f[i], kMostLift);
        use = use || ((small >> i & 1u) != 0 && m >= kFar);
        if (small >> i & 1u) lifts |= static_cast<uint32_t>(max(m, 0)) << (8 * i);
    }
    use = __any_sync(0xffffffffu, use);
    return make_uint2(use ? lifts : 0u, (use ? 1u : 0u) | (g <= -kFar ? 2u : 0u));
}

// A tile's lifts, applied to a copy of its codes by a warp; whether there are any.
static __device__ __noinline__ bool lift_tile(uint8_t* codes, int n, uint32_t small, int lane) {
    const uint2 l = tile_lifts(codes, n, small, lane);
    __syncwarp();
#pragma unroll 1
    for (int i = 0; i < 4; ++i)
        if (32 * i + lane < n) lift_row(codes + (32 * i + lane) * 128, static_cast<int>(l.x >> (8 * i) & 0xFFu));
    __syncwarp();
    return (l.y & 1u) != 0;
}

// One warp scans the tiles of a segment one after another, from the codes that the copies brought to shared memory.  (The
// code of the common case is kept short: the loops of a block's warps share an instruction cache that they fill.)
struct TileScan {
    int run;      // largest scale since the last eager tile
    bool before;  // the tile before may have set R by its scales
    __device__ __forceinline__ void reset() {
        run = -1000;
        before = false;
    }
    // A tile's codes are at `codes`, its first n >= 1 tokens exist; `bits`: the scales of tokens 4 lane .. 4 lane + 3 (kNoScale for
    // those that do not).  Where tokens are lifted, the tile's lifts go to `to` (a byte each, in shared memory).
    __device__ __forceinline__ TileAsks tile(const uint8_t* codes, int n, const uint32_t (&bits)[4], int lane, uint8_t* to) {
        const uint32_t small = small_tokens(codes, n, lane);
        const int hi = static_cast<int>(__reduce_max_sync(0xffffffffu, max(max(bits[0], bits[1]), max(bits[2], bits[3]))) >> 23);
        TileAsks ask = {0u, before || hi + kFar <= run ? 1u : 0u};
        before = false;
        if (__any_sync(0xffffffffu, small != 0)) {
            const uint2 l = tile_lifts(codes, n, small, lane);
            ask.lift = l.y & 1u;
            ask.eager |= ask.lift;
            before = l.y != 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) to[32 * i + lane] = static_cast<uint8_t>(l.x >> (8 * i));
            __syncwarp();
        }
        run = ask.eager ? hi : max(run, hi);
        return ask;
    }
};

constexpr float kLift = 48.f;
struct RowPeak {  // of a row's piece: the y (rounded up) that the last first, up or eager move was for; the highest R
    float peak, high;
};
template <int First, int Up, int Low>
struct RowRef {
    // The common case, in one comparison: neither up nor low.
    static constexpr float kMiddle = 0.5f * (kRoom - Low), kHalf = 0.5f * (kRoom + Low);
    __device__ static bool stays(float top, float R) { return !(fabsf(top - R - kMiddle) > kHalf); }
    __device__ static bool is_up(float top, float R) { return top > R + kRoom; }
    // (not for a unit with nothing visible, nor before the first)
    __device__ static bool is_low(float top, float R) {
        return top < R - static_cast<float>(Low) && top != __uint_as_float(kMinusInf);
    }
    // The reference after a piece's first unit (by itself: the code of all other moves is long, and seldom there when a piece
    // starts).
    __device__ static float first(float top, RowPeak& pk) {
        if (top == __uint_as_float(kMinusInf)) return kNoRef;
        pk.peak = ceilf(top);
        return pk.high = pk.peak - First;
    }
    // The reference after a unit of tile n whose largest y is `top`; `same`: R has not changed since this warp's last unit, of
    // tile n - 1.  `low` is the warp's for the row.
    __device__ static float moved(float top, float R, bool same, uint32_t n, bool eager, LowUnit& low, RowPeak& pk) {
        if (is_up(top, R)) {
            const bool first = R == kNoRef;
            pk.peak = ceilf(top);
            R = pk.peak - (first ? First : Up);
            pk.high = first ? R : fmaxf(pk.high, R);
        } else if (is_low(top, R)) {
            if (eager) {
                pk.peak = ceilf(top);
                R = fminf(R, fmaxf(pk.peak - First, pk.high - kLift));
                low.at = kNoTile;
            } else if (same && low.at == n - 1) {
                R = fminf(R, fmaxf(ceilf(fmaxf(top, low.top)) - First, pk.peak - Up));
                low.at = kNoTile;
            } else {
                low.top = top;
                low.at = n;
            }
        }
        return R;
    }
};
// The exponent by which O and the sums are multiplied when R moves (<= -126: they vanish; 0 too where there was none).
__device__ __forceinline__ int ref_exp(float from, float to) {
    return from == kNoRef ? 0 : static_cast<int>(fmaxf(from - to, -127.f));
}
__device__ __forceinline__ float ref_factor(int d) { return d <= -126 ? 0.f : exp2_int(d); }
// The factor from one reference to another (1 where there was none: the sum is then 0).
__device__ __forceinline__ float ref_step(float from, float to) {
    return from == kNoRef ? 1.f : ref_factor(static_cast<int>(fmaxf(from - to, -127.f)));
}

// Instruction descriptor for kind::f8f6f4 with e4m3 operands (a_e5m2, b_e5m2: that one e5m2) and fp32 D.
__host__ __device__ constexpr uint32_t idesc_f8_f32(int M, int N, bool a_mn_major, bool b_mn_major, bool a_e5m2 = false,
                                                    bool b_e5m2 = false) {
    return (1u << 4) | (static_cast<uint32_t>(a_e5m2) << 7) | (static_cast<uint32_t>(b_e5m2) << 10) |
           (static_cast<uint32_t>(a_mn_major) << 15) | (static_cast<uint32_t>(b_mn_major) << 16) |
           (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

}  // namespace d8
}  // namespace mla
