// The 8-bit latent cache: quantising rows as they are written, and bringing them back to bf16.
//
// A token's row x = [c^KV (512) | R_pos k^R (64)] is the bf16 row that append_cache.cu stores; its 8-bit form is
//   s = 2^k, the least power of two >= 2^-40 with max |x_i| <= 448 s over the finite x_i (1 if none is nonzero),
//   code_i = e4m3(x_i / s), round to nearest, ties to even; NaN and infinities become NaN.
// x_i / s and code_i * s only move the exponent, so the one rounding is e4m3's (relative 2^-4 at most, down to
// 2^-6 s; steps of 2^-9 s below).  One scale serves all 576 columns: e4m3 is a floating-point type, so a finer
// scale would gain precision only for values more than 2^14 below the row's largest.
//
// Layout of a block (mla.h): column c of row r at byte (c / 128) * 16384 + r * 128 + (((c % 128) / 16) ^ (r % 8)) * 16
// + c % 16 for the latent part, 65536 + r * 64 + (((c - 512) / 16) ^ (r / 2 % 4)) * 16 + c % 16 for the RoPE part, and
// the fp32 scale of row r at 73728 + 4 r.
#include "mla_internal.cuh"
#include "sm100.cuh"

namespace mla {

namespace {

// Bits of |x| of two packed bf16, 0 where not finite; their maximum.
__device__ __forceinline__ uint32_t top_bits(uint32_t w) {
    const uint32_t lo = w & 0x7FFFu, hi = (w >> 16) & 0x7FFFu;
    return max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u);
}

// fp32 value of a bf16; infinities as NaN.
__device__ __forceinline__ float finite_or_nan(uint32_t bits16) {
    return __uint_as_float((bits16 & 0x7FFFu) == 0x7F80u ? 0x7FC00000u : bits16 << 16);
}

// Four bf16 (two words) times inv -> four e4m3 codes.
__device__ __forceinline__ uint32_t codes4(uint32_t w0, uint32_t w1, float inv) {
    const uint32_t a = sm100::cvt_e4m3x2(finite_or_nan(w0 & 0xFFFFu) * inv, finite_or_nan(w0 >> 16) * inv);
    const uint32_t b = sm100::cvt_e4m3x2(finite_or_nan(w1 & 0xFFFFu) * inv, finite_or_nan(w1 >> 16) * inv);
    return a | (b << 16);
}

// The same where every value is finite: the products are exact in bf16 (down to steps far below e4m3's).
__device__ __forceinline__ uint32_t codes2_finite(uint32_t w, uint32_t inv2) {
    uint32_t v;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(v) : "r"(w), "r"(inv2));
    return sm100::cvt_e4m3x2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t codes4_finite(uint32_t w0, uint32_t w1, uint32_t inv2) {
    return __byte_perm(codes2_finite(w0, inv2), codes2_finite(w1, inv2), 0x5410);
}

// A warp per token: lane i has latent columns 16 i .. 16 i + 15 (32 bytes read, one 16-byte unit written) and the RoPE
// pair i.  The row's maximum is an integer maximum of bf16 magnitudes, so the scale has no rounding; a row with a NaN or an
// infinity takes the longer way.
// Has to move 1416 bytes in and 580 out a token, 10 us for 32749 tokens at a copy's rate; takes 15: DRAM is at 39 % of its peak
// (the writes stay in L2), the integer pipe of the busiest SM at 73 %, so it is the instructions of packing, and the ramp.
// At decode sizes the launch: 2.6 us.  Half a warp per token, with half the address arithmetic, took as long.
__global__ void __launch_bounds__(256) append_cache8_kernel(
    uint8_t* __restrict__ cache, int64_t cap_blocks, const int32_t* __restrict__ block_table, int num_seqs,
    int max_blocks, const int32_t* __restrict__ seq_idx, const int32_t* __restrict__ pos,
    const uint16_t* __restrict__ c_kv, const uint16_t* __restrict__ k_rope, const float* __restrict__ rope_table,
    int64_t rope_len, int T, int32_t* dev_status) {
    const int64_t tok = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    if (tok >= T) return;
    const int32_t p = pos[tok];
    const int32_t sq = seq_idx[tok];
    const uint4* src = reinterpret_cast<const uint4*>(c_kv + tok * kDc) + 2 * lane;
    const uint4 x0 = src[0], x1 = src[1];
    const uint32_t x[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
    const uint32_t xr = reinterpret_cast<const uint32_t*>(k_rope + tok * kDr)[lane];
    int64_t blk = -1;
    if (p >= 0 && sq >= 0 && sq < num_seqs && p / kBlockTokens < max_blocks)
        blk = block_table[static_cast<int64_t>(sq) * max_blocks + p / kBlockTokens];
    float2 cs = make_float2(0.f, 0.f);  // (asked for beside the table entry, not after it)
    if (p >= 0 && p < rope_len) cs = reinterpret_cast<const float2*>(rope_table + static_cast<int64_t>(p) * kDr)[lane];
    if (blk < 0 || blk >= cap_blocks) {
        if (lane == 0) report(dev_status, MLA_DEVERR_ROW_RANGE);
        return;
    }
    if (p >= rope_len) {
        if (lane == 0) report(dev_status, MLA_DEVERR_POS_RANGE);
        return;
    }
    // the RoPE pair, rotated and rounded to bf16 with append_cache.cu's arithmetic
    const float r0 = bf16_to_f32(static_cast<uint16_t>(xr & 0xFFFFu));
    const float r1 = bf16_to_f32(static_cast<uint16_t>(xr >> 16));
    const uint32_t y = pack_bf16x2(__fsub_rn(__fmul_rn(r0, cs.x), __fmul_rn(r1, cs.y)),
                                   __fadd_rn(__fmul_rn(r0, cs.y), __fmul_rn(r1, cs.x)));
    uint32_t m2 = y & 0x7FFF7FFFu;
#pragma unroll
    for (int w = 0; w < 8; ++w) m2 = sm100::max_abs2(m2, x[w]);
    uint32_t top = __reduce_max_sync(0xffffffffu, max(m2 & 0xFFFFu, m2 >> 16));
    const bool finite = top < 0x7F80u;
    if (!finite) {
        top = top_bits(y);
#pragma unroll
        for (int w = 0; w < 8; ++w) top = max(top, top_bits(x[w]));
        top = __reduce_max_sync(0xffffffffu, top);
    }
    // 448 = 1.75 * 2^8: with top = f * 2^e, k = e - 8, or e - 7 where f > 1.75
    int k = static_cast<int>(top >> 7) - 127 - 8 + ((top & 0x7Fu) > 0x60u ? 1 : 0);
    k = top == 0 ? 0 : max(k, kScale8MinExp);
    const uint32_t inv = static_cast<uint32_t>(127 - k) << 23;  // (k <= 120: a normal number)
    const int r = p % kBlockTokens;
    uint8_t* dst = cache + blk * kBlock8Bytes;
    uint32_t c[4], cy;
    if (finite) {
        const uint32_t inv2 = inv | (inv >> 16);
#pragma unroll
        for (int w = 0; w < 4; ++w) c[w] = codes4_finite(x[2 * w], x[2 * w + 1], inv2);
        cy = codes2_finite(y, inv2);
    } else {
#pragma unroll
        for (int w = 0; w < 4; ++w) c[w] = codes4(x[2 * w], x[2 * w + 1], __uint_as_float(inv));
        cy = codes4(y, 0, __uint_as_float(inv));
    }
    *reinterpret_cast<uint4*>(dst + (lane >> 3) * kBlock8Chunk + r * 128 + (((lane & 7) ^ (r & 7)) << 4)) =
        make_uint4(c[0], c[1], c[2], c[3]);
    *reinterpret_cast<uint16_t*>(dst + kBlock8Rope + r * 64 + (((lane >> 3) ^ ((r >> 1) & 3)) << 4) + (lane & 7) * 2) =
        static_cast<uint16_t>(cy);
    if (lane == 0)
        *reinterpret_cast<float*>(dst + kBlock8Scales + 4 * r) = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
}

// Two e4m3 codes times s, as packed bf16 (exact unless the product leaves bf16's normal range).
__device__ __forceinline__ uint32_t two_back(uint32_t codes, float s) {
    const float2 v = sm100::e4m3x2_to_f32(static_cast<uint16_t>(codes));
    return pack_bf16x2(v.x * s, v.y * s);
}

constexpr int kReadRows = 32;     // rows of a work unit: a quarter of a block
constexpr int kReadThreads = 288; // nine warps: 36 units of 16 codes a row x 32 rows / 288 = 4 units a thread
constexpr int kReadUnitsPerTile = kBlockTokens / kReadRows;

// Tiles of sequence b to copy; 0 (reported by the caller's flag) where it does not fit its table rows.
__device__ __forceinline__ int read_tiles(const int32_t* kv_len, int b, int mb8, int mb16, int32_t* bad) {
    const int L = kv_len[b];
    if (L < 0) {
        *bad |= MLA_DEVERR_KV_LEN;
        return 0;
    }
    const int nt = L / kBlockTokens + (L % kBlockTokens != 0);
    if (nt > mb8 || nt > mb16) {
        *bad |= MLA_DEVERR_ROW_RANGE;
        return 0;
    }
    return nt;
}

// The (sequence, quarter block) units are cut into equal ranges, one per CTA, so ragged lengths balance; a thread
// takes four 16-byte units of codes (all four loads in flight) and writes two neighbouring 16-byte units of bf16 for
// each.  Bound: HBM, 580 bytes read and 1152 written a token: 173 us for 520 K tokens, 5.1 TB/s (a copy 6.6, writes alone
// 3.8).  Seven ranges an SM, of which four run at once: with 3, 4, 14 or 28 it took 178, 177, 177 and 183 us, with more
// CTAs at once (fewer registers) 220 and more; with the addresses computed unit by unit 188.
__global__ void __launch_bounds__(kReadThreads) read_cache8_kernel(
    const uint8_t* __restrict__ cache8, int64_t cap8, const int32_t* __restrict__ table8, int mb8,
    const int32_t* __restrict__ kv_len, int B, uint8_t* __restrict__ cache, int64_t cap, const int32_t* __restrict__ table,
    int mb16, int32_t* dev_status) {
    __shared__ int64_t first[2];  // [total tiles, tiles before the first sequence of this CTA]
    __shared__ int first_b;
    const int tid = threadIdx.x, lane = tid & 31;
    if (tid < 32) {
        int32_t bad = 0;
        int64_t total = 0;
        for (int b = lane; b < B; b += 32) total += read_tiles(kv_len, b, mb8, mb16, &bad);
        if (bad && blockIdx.x == 0) report(dev_status, bad);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        const int64_t lo = total * kReadUnitsPerTile * blockIdx.x / gridDim.x / kReadUnitsPerTile;
        int64_t run = 0, before = total;
        int b0 = B;
        for (int base = 0; base < B; base += 32) {
            const int b = base + lane;
            const int nt = b < B ? read_tiles(kv_len, b, mb8, mb16, &bad) : 0;
            int64_t inc = nt;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += v;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, b < B && run + inc > lo);
            if (hit) {
                const int f = __ffs(hit) - 1;
                b0 = base + f;
                before = run + __shfl_sync(0xffffffffu, inc - nt, f);
                break;
            }
            run += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (lane == 0) {
            first[0] = total;
            first[1] = before;
            first_b = b0;
        }
    }
    __syncthreads();
    // this thread's units: one place of the rows rr, rr + 8, .. of a work unit (the swizzles repeat every eight rows), in
    // latent chunk tid / 64 or, the last warp, in the RoPE part
    const bool lat = tid < 256;
    const int place = lat ? tid & 7 : tid & 3, rr = lat ? (tid >> 3) & 7 : lane >> 2;
    const int v = lat ? 8 * (tid >> 6) + (place ^ rr) : 32 + (place ^ ((rr >> 1) & 3));  // columns 16 v .. 16 v + 15
    const int src_row = lat ? 128 : 64;
    const int src_off = (lat ? (tid >> 6) * kBlock8Chunk : kBlock8Rope) + rr * src_row + (place << 4);
    const int dst_off = (v >> 2) * kBlockChunk + rr * 128;
    const int at0 = (((2 * v) & 7) ^ rr) << 4, at1 = at0 ^ 16;
    const int64_t units = first[0] * kReadUnitsPerTile;
    const int64_t lo = units * blockIdx.x / gridDim.x, hi = units * (blockIdx.x + 1) / gridDim.x;
    int64_t tb = first[1] * kReadUnitsPerTile;
    int32_t bad = 0;
    for (int b = first_b; b < B && tb < hi; ++b) {
        const int nt = read_tiles(kv_len, b, mb8, mb16, &bad);
        const int64_t te = tb + static_cast<int64_t>(nt) * kReadUnitsPerTile;
        const int L = kv_len[b];
        for (int64_t u = lo > tb ? lo : tb; u < (hi < te ? hi : te); ++u) {
            const int t = static_cast<int>((u - tb) / kReadUnitsPerTile);
            const int row0 = static_cast<int>((u - tb) % kReadUnitsPerTile) * kReadRows;
            const int32_t e8 = table8[static_cast<int64_t>(b) * mb8 + t], e16 = table[static_cast<int64_t>(b) * mb16 + t];
            if (e8 < 0 || e8 >= cap8 || e16 < 0 || e16 >= cap) {
                if (tid == 0) report(dev_status, MLA_DEVERR_ROW_RANGE);
                continue;
            }
            const uint8_t* src = cache8 + static_cast<int64_t>(e8) * kBlock8Bytes;
            const float* sc = reinterpret_cast<const float*>(src + kBlock8Scales) + row0 + rr;
            src += src_off + row0 * src_row;
            uint8_t* dst = cache + static_cast<int64_t>(e16) * kBlockBytes + dst_off + row0 * 128;
            const int rows = min(kReadRows, L - t * kBlockTokens - row0) - rr;  // row 8 k of this thread's: < rows
            uint4 x[4];
            float f[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                x[k] = make_uint4(0, 0, 0, 0);
                f[k] = 0.f;
                if (8 * k < rows) {
                    x[k] = *reinterpret_cast<const uint4*>(src + 8 * k * src_row);
                    f[k] = sc[8 * k];
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (8 * k >= rows) continue;
                uint8_t* d = dst + 8 * k * 128;
                *reinterpret_cast<uint4*>(d + at0) =
                    make_uint4(two_back(x[k].x, f[k]), two_back(x[k].x >> 16, f[k]), two_back(x[k].y, f[k]),
                               two_back(x[k].y >> 16, f[k]));
                *reinterpret_cast<uint4*>(d + at1) =
                    make_uint4(two_back(x[k].z, f[k]), two_back(x[k].z >> 16, f[k]), two_back(x[k].w, f[k]),
                               two_back(x[k].w >> 16, f[k]));
            }
        }
        tb = te;
    }
}

}  // namespace

cudaError_t launch_append_cache8(uint8_t* cache, int64_t cap_blocks, const int32_t* block_table, int num_seqs,
                                 int max_blocks, const int32_t* seq_idx, const int32_t* pos, const uint16_t* c_kv,
                                 const uint16_t* k_rope, const float* rope_table, int64_t rope_len, int T,
                                 int32_t* dev_status, cudaStream_t stream) {
    const int threads = 256;
    const int64_t blocks = (static_cast<int64_t>(T) * 32 + threads - 1) / threads;
    append_cache8_kernel<<<static_cast<unsigned>(blocks), threads, 0, stream>>>(
        cache, cap_blocks, block_table, num_seqs, max_blocks, seq_idx, pos, c_kv, k_rope, rope_table, rope_len, T,
        dev_status);
    return cudaGetLastError();
}

cudaError_t launch_read_cache8(const uint8_t* cache8, int64_t cap8, const int32_t* table8, int mb8,
                               const int32_t* kv_len, int B, uint8_t* cache, int64_t cap, const int32_t* table, int mb16,
                               int32_t* dev_status, cudaStream_t stream) {
    const int64_t most = static_cast<int64_t>(B) * (mb8 < mb16 ? mb8 : mb16) * kReadUnitsPerTile;
    const int64_t want = most < 148 * 7 ? most : 148 * 7;
    read_cache8_kernel<<<static_cast<unsigned>(want), kReadThreads, 0, stream>>>(cache8, cap8, table8, mb8, kv_len, B,
                                                                                 cache, cap, table, mb16, dev_status);
    return cudaGetLastError();
}

}  // namespace mla
