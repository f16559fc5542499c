// End of mla_decode8: the merge of the attend kernel's pieces and the up-projection by W^UV, in one kernel.
//
//   o[t, h] = sum_p 2^(R_p - M) O_p / sum_p 2^(R_p - M) t_p    over the pieces p of t's sequence, M = max_p R_p
//   lse     = (M + log2 sum_p 2^(R_p - M) l_p) ln 2            (R_p integers: exact factors)
// with l_p the sum of the probabilities and t_p the sum as O_p has them, rounded to 8 significant bits each: a token that
// carries its row alone then comes out exactly (4 x 128K, error against 64 bits 0.0026 -> 0.0018, for 2 to 3 % of the time).
//   out[t, h, :] = W^UV_h o[t, h]                              (128 = 128 x 512)
//
// One CTA per (block of query rows, head): its 16 warps merge the rows, each a row at a time (or, with fewer rows than
// warps, several warps a row, each over a part of the pieces), into shared memory as the B operand of 32 MMAs
// (M = 128 output columns, N = 2 rows, K = 512: o as bf16 and what that leaves as a second bf16 row, whose results are added;
// o rounded once was the call's largest error, 0.0017 of 0.0027 in the 2-norm) whose A operand, W^UV_h, is under way by TMA before the attend kernel ends.
// It has to move the pieces (2 KB a row and piece, from L2) and W^UV_h (128 KB a CTA, from HBM once), 4 us at B 32, H 128;
// what it takes, 8 to 13 us after the attend kernel, is latency: lengths, pieces, sums, MMAs, result, one after the other.
// A warp therefore keeps four pieces' loads in flight, of whichever rows, and what depends on the lengths alone is done
// before the wait.  A piece row comes in 128-byte runs: in 32-byte runs a merge of 32 rows took 20000 cycles instead of
// 8000 (an L1 request a run).  With a merge kernel, o_lat in memory and a projection kernel of 256 rows a CTA instead,
// the whole call took 104 us instead of 82 (B 2, H 20, 101 queries each), 51 instead of 35 (B 37, H 11, 3 queries each),
// 57 instead of 51 (B 64, H 16, 4K), and the same at B 32, H 128, 8K.
#include <cuda.h>
#include <math_constants.h>

#include <algorithm>

#include "decode8_common.cuh"

namespace mla {

namespace proj {
bool weight_map(CUtensorMap* map, const uint16_t* W, int H);  // proj_tc.cu
}

namespace fin8 {

using namespace d8;

constexpr int kWarps = 16, kThreads = 32 * kWarps;
constexpr int kMaxRows = 32;
constexpr int kSms = 148;
constexpr int kBatch = 4;  // pieces whose loads are in flight together (64 bytes a lane each)
constexpr int kWBytes = kDh * kDc * 2, kWChunk = kDh * 128;
constexpr int kOffPart = kWBytes;                        // [16 warps][4][32 lanes] float4: a warp's share of a row; then out
constexpr int kOffMz = kOffPart + kWarps * 2048;         // [16 warps] M and the sums
constexpr int kOffTab = kOffMz + kWarps * 16;             // [32] the block's rows: Row
constexpr int kOffSeq = kOffTab + kMaxRows * 16;         // [32] tiles of the block's sequences; pieces (first, how many)
constexpr int kOffBar = kOffSeq + kMaxRows * 8;          // W there, MMAs done
constexpr int kOffRed = kOffBar + 16;                    // [2][16] tile counts; TMEM address
constexpr int kOffO = ((kOffRed + 2 * kWarps * 4 + 16 + 1023) / 1024) * 1024;  // o: 8 chunks of [N rows x 64 columns] bf16, swizzled; rows, then their second terms
static_assert(kOffO + 2 * kMaxRows * 1024 <= 232448 && kMaxRows * kDh * 2 <= kOffMz - kOffPart, "shared memory");
static_assert(kOffTab % 16 == 0 && kOffBar % 8 == 0, "alignment");

struct Row {
    int first, pieces;  // of the row's sequence (see below)
    int seg, r;         // slot of unit 0's piece, row in its group of 128
};

struct FinParams {
    const float* o_part;
    const float4* ml_part;
    const int32_t* kv_len;
    uint16_t* out;
    float* lse;
    int32_t* dev_status;
    int max_blocks, B, n_q, H, P_g, slots, rs, rows;  // rows: query rows a block (8, 16 or 32)
};

__device__ __forceinline__ void ld_global8(const float* p, float* v) {
    asm volatile("ld.global.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "l"(p));
}

__global__ void __launch_bounds__(kThreads, 1) finish8_kernel(const __grid_constant__ CUtensorMap wmap, const FinParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBar);
    int* red = reinterpret_cast<int*>(smem + kOffRed);
    Row* tab = reinterpret_cast<Row*>(smem + kOffTab);
    int2* seq = reinterpret_cast<int2*>(smem + kOffSeq);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffRed + 2 * kWarps * 4);
    const int h = blockIdx.y;
    const int T = p.B * p.n_q;
    const int N = 2 * p.rows;  // B operand rows (those past n are not written, nor their results read)
    volatile int never = 0;
    if ((sbase & 1023u) != 0) {
        if (tid == 0) report(p.dev_status, MLA_DEVERR_TIMEOUT);
        return;
    }
    if (tid == 0) {
        mbar_init(&bars[0], 1);
        mbar_init(&bars[1], 1);
        fence_mbar_init();
        // W^UV is an input of the call: no kernel of it writes it
        mbar_arrive_expect_tx(&bars[0], kWBytes);
        for (int c = 0; c < 8; ++c) tma_load_3d(sbase + c * kWChunk, &wmap, 0, h * kDh, c, &bars[0]);
    }
    if (warp == 0) tmem_alloc(tmem_slot, 64);
    // tiles of all sequences, and of those before the first block's first (the lengths are inputs too)
    int b_at = blockIdx.x * p.rows / p.n_q, s_all = 0, s_pre = 0;
    for (int i = tid; i < p.B; i += kThreads) {
        const int tiles = valid_seq_tiles(p.kv_len[i], p.n_q, p.max_blocks);
        s_all += tiles;
        if (i < b_at) s_pre += tiles;
    }
    s_all = __reduce_add_sync(0xffffffffu, s_all);
    s_pre = __reduce_add_sync(0xffffffffu, s_pre);
    if (lane == 0) {
        red[warp] = s_all;
        red[kWarps + warp] = s_pre;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    int Nt = 0, pre = 0;  // pre: tiles of the sequences before b_at
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        Nt += red[w];
        pre += red[kWarps + w];
    }
    bool ok = true;
    for (uint32_t it = 0, t0 = blockIdx.x * p.rows; ok && t0 < T; ++it, t0 += gridDim.x * p.rows) {
        const int n = min(p.rows, T - t0);
        if (warp == 0) {
            // the block's sequences b0 .. b0 + nb - 1 and rows
            const int b0 = t0 / p.n_q, nb = (t0 + n - 1) / p.n_q - b0 + 1;
            int more = 0;
            for (int i = b_at + lane; i < b0; i += 32) more += valid_seq_tiles(p.kv_len[i], p.n_q, p.max_blocks);
            pre += __reduce_add_sync(0xffffffffu, more);
            b_at = b0;
            const int nt = lane < nb ? valid_seq_tiles(p.kv_len[b0 + lane], p.n_q, p.max_blocks) : 0;
            int inc = nt;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += v;
            }
            // a sequence's pieces: the work units whose tile range meets its own, [ts, ts + tiles).  With at least as many
            // tiles as units they follow one another: (the first, how many); otherwise a unit has one tile or none, and
            // each tile is a piece: (its first tile, how many)
            const int64_t ts = pre + inc - nt, P = p.P_g;
            int2 e = make_int2(static_cast<int>(ts), nt);
            if (Nt >= p.P_g && nt > 0) {
                e.x = static_cast<int>(((ts + 1) * P - 1) / Nt);
                e.y = static_cast<int>(((ts + nt) * P - 1) / Nt) - e.x + 1;
            }
            seq[lane] = e;
            __syncwarp();
            if (lane < n) {
                const int b = (t0 + lane) / p.n_q, rr = (t0 + lane - b * p.n_q) * p.H + h;
                tab[lane] = {seq[b - b0].x, seq[b - b0].y, (rr >> 7) * p.slots + b, rr & 127};
            }
        }
        __syncthreads();
        if (it == 0) grid_dependency_wait();  // the pieces come from the attend kernel

        // S warps a row: warp k of them takes every S-th piece.  A batch's loads go out together, whichever rows they are of
        int S = 1;
        while (2 * S * n <= kWarps) S *= 2;
        const int k = warp % S;
        float2 acc[8];
        float M = kNoRef, z = 0.f, zt = 0.f;
#pragma unroll
        for (int q = 0; q < 8; ++q) acc[q] = make_float2(0.f, 0.f);
        auto write_row = [&](int i) {  // row i's o into the B operand, its lse out
            const float inv = zt > 0.f ? 1.f / zt : (zt != zt ? CUDART_NAN_F : 0.f);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int j = lane + 32 * q;  // columns 8 j .. 8 j + 7
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const float a = acc[4 * q + w].x * inv, b = acc[4 * q + w].y * inv;
                    hi[w] = pack_bf16x2(a, b);
                    lo[w] = pack_bf16x2(a - __uint_as_float(hi[w] << 16), b - __uint_as_float(hi[w] & 0xFFFF0000u));
                }
                uint8_t* at = smem + kOffO + (j >> 3) * N * 128 + i * 128 + (((j & 7) ^ (i & 7)) << 4);
                *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4*>(at + p.rows * 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
            if (lane == 0 && p.lse)  // nothing visible: -inf; a NaN shows
                p.lse[static_cast<int64_t>(t0 + i) * p.H + h] =
                    (z > 0.f || z != z) ? (M + log2f(z)) * 0.69314718055994530942f : -CUDART_INF_F;
        };
        int i = warp / S, e = k;
        while (i < n) {
            float2 v[kBatch][8];
            float4 ml[kBatch];
            int row[kBatch];  // the row that item ends, or -1
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                ml[u] = make_float4(kNoRef, 0.f, 0.f, 0.f);
                row[u] = -1;
                if (i < n) {
                    const Row w = tab[i];
                    if (e < w.pieces) {
                        const int unit = Nt >= p.P_g ? w.first + e : ((w.first + e + 1) * p.P_g - 1) / Nt;
                        const int64_t at = w.seg + unit;
                        const float* src = p.o_part + ((at * 16 + (lane >> 2)) * p.rs + w.r) * 32 + 8 * (lane & 3);
                        ld_global8(src, &v[u][0].x);
                        ld_global8(src + 8 * 32 * p.rs, &v[u][4].x);
                        ml[u] = p.ml_part[at * p.rs + w.r];
                    }
                    e += S;
                    if (e >= w.pieces) {
                        row[u] = i;
                        i += kWarps / S;
                        e = k;
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                if (ml[u].x != kNoRef) {
                    if (ml[u].x > M) {
                        const float sc = ref_step(M, ml[u].x);
                        M = ml[u].x;
                        z *= sc;
                        zt *= sc;
#pragma unroll
                        for (int q = 0; q < 8; ++q) acc[q] = mul2(acc[q], make_float2(sc, sc));
                    }
                    const float w = ref_step(ml[u].x, M);
                    z = fmaf(ml[u].y, w, z);
                    zt = fmaf(ml[u].z, w, zt);
#pragma unroll
                    for (int q = 0; q < 8; ++q) acc[q] = fma2(make_float2(w, w), v[u][q], acc[q]);
                }
                if (S == 1 && row[u] >= 0) {
                    write_row(row[u]);
                    M = kNoRef;
                    z = zt = 0.f;
#pragma unroll
                    for (int q = 0; q < 8; ++q) acc[q] = make_float2(0.f, 0.f);
                }
            }
        }
        if (S > 1) {  // (a warp had one row at most)
            float4* part = reinterpret_cast<float4*>(smem + kOffPart) + lane;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                part[128 * warp + 32 * q] = make_float4(acc[2 * q].x, acc[2 * q].y, acc[2 * q + 1].x, acc[2 * q + 1].y);
            if (lane == 0) reinterpret_cast<float4*>(smem + kOffMz)[warp] = make_float4(M, z, zt, 0.f);
            __syncthreads();
            if (k == 0 && warp / S < n) {
                const float4* mz = reinterpret_cast<const float4*>(smem + kOffMz) + warp;
                float top = M;
                for (int u = 1; u < S; ++u) top = fmaxf(top, mz[u].x);
                float sc = ref_step(M, top);
                M = top;
                z *= sc;
                zt *= sc;
#pragma unroll
                for (int q = 0; q < 8; ++q) acc[q] = mul2(acc[q], make_float2(sc, sc));
                for (int u = 1; u < S; ++u) {
                    sc = ref_step(mz[u].x, top);  // (a warp without a piece: zeros)
                    z = fmaf(mz[u].y, sc, z);
                    zt = fmaf(mz[u].z, sc, zt);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float4 x = part[128 * (warp + u) + 32 * q];
                        acc[2 * q] = fma2(make_float2(x.x, x.y), make_float2(sc, sc), acc[2 * q]);
                        acc[2 * q + 1] = fma2(make_float2(x.z, x.w), make_float2(sc, sc), acc[2 * q + 1]);
                    }
                }
                write_row(warp / S);
            }
        }
        fence_proxy_async_cta();
        __syncthreads();

        if (warp == 0) {
            ok = mbar_wait(&bars[0], 0, &never, kLimitNs);
            ok = __all_sync(0xffffffffu, ok);
            if (elect_one()) {
                if (ok) {
                    // D[d, row] = sum_c W^UV_h[d, c] o[row, c]
                    tc_fence_after();
                    const uint32_t idesc = idesc_bf16_f32(kDh, N, false, false);
                    const uint64_t a = sdesc_sw128(sbase, 16, 1024), o = sdesc_sw128(sbase + kOffO, 16, 1024);
                    for (int c = 0; c < 8; ++c)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_ss(tmem, a + ((c * kWChunk + kk * 32) >> 4), o + static_cast<uint64_t>((c * N * 128 + kk * 32) >> 4),
                                   idesc, (c | kk) ? 1u : 0u);
                } else {
                    report(p.dev_status, MLA_DEVERR_TIMEOUT);
                }
                mma_commit(smem_u32(&bars[1]));  // also after a failure: TMEM is freed only once it fires
            }
            __syncwarp();
        }
        const bool done = mbar_wait(&bars[1], it & 1u, &never, kLimitNs);
        if (!done && lane == 0) report(p.dev_status, MLA_DEVERR_TIMEOUT);
        ok = __syncthreads_and(ok && done);
        tc_fence_after();
        if (ok) {
            // lane = output column; row j's 128 are staged as 256 bytes
            const int d = 32 * (warp & 3) + lane;
            const int j0 = 8 * (warp >> 2);
            if (j0 < n) {
                uint32_t v[8], w[8];
                const uint32_t at = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + j0;
                tmem_ld8(at, v);
                tmem_ld8(at + p.rows, w);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    *reinterpret_cast<uint16_t*>(smem + kOffPart + (j0 + j) * (kDh * 2) + 2 * d) =
                        f32_to_bf16_rne(__uint_as_float(v[j]) + __uint_as_float(w[j]));
            }
        }
        tc_fence_before();
        __syncthreads();
        if (ok)
            for (int i = tid; i < n * 16; i += kThreads)
                reinterpret_cast<uint4*>(p.out + (static_cast<int64_t>(t0 + (i >> 4)) * p.H + h) * kDh)[i & 15] =
                    *reinterpret_cast<const uint4*>(smem + kOffPart + 16 * i);
    }
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 64);
    }
}

}  // namespace fin8

cudaError_t launch_finish8(const float* o_part, const float4* ml_part, const int32_t* kv_len, int max_blocks, int B, int n_q,
                           int H, int P_g, int slots, int rs, const uint16_t* W_UV, uint16_t* out, float* lse_out,
                           int32_t* dev_status, cudaStream_t stream) {
    CUtensorMap map;
    if (!proj::weight_map(&map, W_UV, H)) return cudaErrorNotSupported;
    const int T = B * n_q;
    // rows a block: the fewest with which all blocks run at once, one to an SM; beyond that a CTA takes several blocks of
    // its head, W^UV_h and the set-up serving them all
    int rows = 8;
    while (rows < fin8::kMaxRows && static_cast<int64_t>(H) * ((T + rows - 1) / rows) > fin8::kSms) rows *= 2;
    const int blocks = (T + rows - 1) / rows;
    const fin8::FinParams prm = {o_part, ml_part, kv_len, out, lse_out, dev_status, max_blocks, B, n_q, H, P_g, slots, rs, rows};
    const int smem = fin8::kOffO + 2 * rows * 1024;
    cudaError_t e = cudaFuncSetAttribute(fin8::finish8_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         fin8::kOffO + 2 * fin8::kMaxRows * 1024);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(std::min(blocks, fin8::kSms / H), H);
    cfg.blockDim = dim3(fin8::kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fin8::finish8_kernel, map, prm);
}

}  // namespace mla
