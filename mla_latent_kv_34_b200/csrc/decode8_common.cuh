// What the two attend kernels of the 8-bit cache share: the split of the (sequence, tile) space into pieces, the
// block lookup, and the two-term e4m3 form of queries and probabilities.
//
// Two terms.  The tensor cores multiply e4m3 by e4m3, so the codes of the cache go into them as they stand.  The other
// operand, a bf16 query or an fp32 probability, is written as hi + lo, both e4m3: hi holds 4 significant bits, lo the
// next 4 of what is left.  A bf16 value (8 significant bits) is represented exactly as long as its last bit is at
// least 2^-9 (the e4m3 step near 0); scaled by a power of two so that the row's largest value lies in (224, 448], that
// is every element down to 2^-10 of the largest, and an absolute 2^-19 of the largest below.
#pragma once

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
    float2* ml_part;
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

// Largest magnitude bits of two packed bf16 into the running packed maximum.
__device__ __forceinline__ uint32_t max_abs2(uint32_t m, uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b32 a;\n\tand.b32 a, %2, 0x7fff7fff;\n\tmax.u16x2 %0, %1, a;\n\t}" : "=r"(r) : "r"(m), "r"(w));
    return r;
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

// hi part of a probability 0 <= p <= 2^8.75: p rounded to 4 significant bits (half up), still fp32.  p - hi is exact.
__device__ __forceinline__ float hi_part(float p) {
    return __uint_as_float((__float_as_uint(p) + 0x00080000u) & 0xFFF00000u);
}

// The reference exponent of a row's probabilities, P' = 2^(y - R) with y = log2(p s_t) (s_t, the token's scale, is
// folded into P because V's rows are codes).  O and the sum are kept relative to R, an integer, so moving it multiplies
// them by an exact power of two.  P' has to stay below 448 (e4m3) and its largest values well above the smallest step:
//   up    when a tile's largest y - R exceeds 8.75;
//   down  when it is below 5 and what came before is small too (`mass`, the sum over earlier tiles of their largest P',
//         below 32 a tile): then the steps of 2^-9 could add up to more than 2^-8 of the row's sum.
// Either way R is put where the tile's largest P' lies in (2^5, 2^6].  It does not go further down than 2^32 below its
// highest place: what is that small no longer counts.
struct RowRef {
    float R, high, mass;
    __device__ __forceinline__ void reset() {
        R = __uint_as_float(0xFF800000u);
        high = R;
        mass = 0.f;
    }
    // Takes a tile's largest y (-inf: nothing visible) and the tiles before it; returns the exponent by which O and
    // the sum are to be multiplied (<= -126: they vanish), 0 for none.
    __device__ __forceinline__ int move(float top, int tiles_before) {
        int d = 0;
        if (top > R + 8.75f || (top < R + 5.f && top != __uint_as_float(0xFF800000u) && mass < 32.f * tiles_before)) {
            float to = ceilf(top) - 6.f;
            to = fmaxf(to, high - 32.f);
            if (to != R) {
                // (no O yet: R is -inf, and nothing is multiplied)
                d = (R == __uint_as_float(0xFF800000u)) ? 0 : static_cast<int>(fmaxf(fminf(R - to, 126.f), -127.f));
                R = to;
                high = fmaxf(high, to);
            }
        }
        mass = mass * factor(d) + (R == __uint_as_float(0xFF800000u) ? 0.f : ex2_approx(top - R));
        return d;
    }
    __device__ __forceinline__ static float factor(int d) { return d <= -126 ? 0.f : exp2_int(d); }
    __device__ __forceinline__ float minus() const { return R == __uint_as_float(0xFF800000u) ? 0.f : -R; }
};

// Instruction descriptor for kind::f8f6f4 with e4m3 A/B and fp32 D.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N, bool a_mn_major, bool b_mn_major) {
    return (1u << 4) | (static_cast<uint32_t>(a_mn_major) << 15) | (static_cast<uint32_t>(b_mn_major) << 16) |
           (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

}  // namespace d8
}  // namespace mla
