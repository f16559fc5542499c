// Absorbed MLA decode over the 8-bit cache on the tensor cores (tcgen05 + TMEM), more than 32 query rows.
//
// The step is mla_decode's (decode_tc.cu): a cluster of two CTAs owns 128 query rows, the "S" CTA forms the scores and
// the softmax, the "O" CTA keeps O[128 x 512] in its whole tensor memory and accumulates P V; the (sequence, tile)
// space is cut into equal ranges, one per cluster, and a range's pieces of sequences go to the workspace for the merge.
// What differs is that a cached row is c_t = s_t code_t with e4m3 codes:
//   - the codes are the operands of both contractions as they lie in the block (kind::f8f6f4, K = 32): no
//     dequantisation, half the bytes from HBM and through shared memory.  Q and P are written as hi + lo of two e4m3
//     terms (decode8_common.cuh), so Q is exact and P keeps 8 significant bits; two K = 32 MMAs at twice the bf16 rate
//     cost what the bf16 MMA of the same elements costs;
//   - scores: x = S * (2^a scale log2 e) * s_t with the query row's power of two 2^a; P' = 2^(x + log2 s_t - R) carries
//     s_t, because the rows of V are codes, and the row's sum takes P' / s_t.  R is RowRef's reference exponent;
//   - a tile (72 KB of codes) comes as copies of 32 and 40 KB into a ring that holds two tiles, so a tile's copies are
//     under way while the one before it is multiplied.
// S CTA: the query's latent part in TMEM (hi 128 columns, lo 128 columns), its RoPE part in shared memory, two score
// buffers of 128 columns; 36 MMAs (M = 128, N = 128) a tile.  O CTA: 16 MMAs (M = 128, N = 256) a tile.
//
// Every wait is bounded: on expiry the kernel records MLA_DEVERR_TIMEOUT, both CTAs of the pair abandon their loops,
// let in-flight copies and MMAs land, free TMEM and return.
#include <cuda.h>
#include <math_constants.h>

#include <mutex>

#include "decode8_common.cuh"

namespace mla {

namespace tc8 {

using namespace d8;

constexpr int kRows = 128;                        // query rows per CTA pair
constexpr int kChunk = kBlock8Chunk;              // [128 tokens x 128 columns] of codes: 16 KB
constexpr int kVStageBytes = 2 * kChunk;          // O CTA: a V stage = two chunks = one N = 256 column block
constexpr int kVStages = 4;                       // two tiles
constexpr int kPBytes = 2 * kRows * kTile;        // hi and lo chunks of [128 rows x 128 tokens]
constexpr int kMsgBytes = kPBytes + kRows;        // P | per-row rescale exponents (int8): one bulk copy
constexpr int kMsgStride = 33792;                 // 1024-aligned message slots
constexpr int kPSlots = 3;
constexpr int kSoftWarps = 8;
constexpr int kSoftThreads = kSoftWarps * 32;
constexpr int kWarpProducer = 8, kWarpMma = 9, kWarpSender = 10;
constexpr int kThreads = 352;
constexpr int kSyncThreads = kSoftThreads + 32;   // softmax warps + the sender warp
constexpr uint32_t kNbQFree = 5, kNbFail = 6, kNbStaged = 7, kNbStageFree = 8;  // named barriers (1..4: quadrant pairs)

// TMEM columns (512 allocated in each CTA)
constexpr uint32_t kColQ = 0;     // S CTA: latent Q codes, four to a column: hi 0..127, lo 128..255
constexpr uint32_t kColS0 = 256;  // S CTA: two 128-column score buffers
__device__ __forceinline__ uint32_t col_s(uint32_t sb) { return kColS0 + 128u * sb; }

// shared memory, S CTA.  Staging buffer 1 shares its space with the Q transpose tiles; barriers, the token scales and
// one block of the exchange sit in the gap behind staging buffer 0.
constexpr int kSOffRing = 0;                           // two tiles
constexpr int kSOffQR = 2 * kTileBytes;                // RoPE part of Q: [128 rows x (hi 64 | lo 64)] swizzled, 16 KB
constexpr int kSOffStage0 = kSOffQR + kRows * 128;
constexpr int kSOffScale = kSOffStage0 + kMsgBytes;    // the tile's 128 token scales s
constexpr int kSOffX7 = kSOffScale + kTile * 4;        // exchange block 7
constexpr int kSOffBar = kSOffX7 + 128;
constexpr int kSOffQT = kSOffStage0 + kMsgStride;      // 8 warps x [32 rows x 128 B] transpose tiles
constexpr int kSOffStage1 = kSOffQT;
constexpr int kSOffExp = kSOffStage1 + kMsgBytes;      // log2 s
constexpr int kSOffInv = kSOffExp + kTile * 4;         // 1 / s
constexpr int kSOffXchg = kSOffInv + kTile * 4;        // exchange blocks 0..6: a warp's 32 half-row maxima or sums
constexpr int kSEnd = kSOffXchg + 7 * 128;
constexpr int kSBarFull = 0, kSBarEmpty = 4, kSBarSFull = 8, kSBarSEmpty = 10, kSBarPEmpty = 12,
              kSBarQReady = kSBarPEmpty + kPSlots, kSBarFin = kSBarQReady + 1, kSNumBars = kSBarFin + 1;
constexpr int kSOffTail = kSOffBar + kSNumBars * 8;
// shared memory, O CTA
constexpr int kOOffV = 0;
constexpr int kOOffMsg = kVStages * kVStageBytes;
constexpr int kOOffBar = kOOffMsg + (kPSlots - 1) * kMsgStride + kMsgBytes;
constexpr int kOBarVFull = 0, kOBarVEmpty = kVStages, kOBarPFull = 2 * kVStages, kOBarOFull = kOBarPFull + kPSlots,
              kOBarOFree = kOBarOFull + 1, kOBarRescReq = kOBarOFree + 1, kOBarRescDone = kOBarRescReq + 1,
              kOBarODrain = kOBarRescDone + 1, kOBarFin = kOBarODrain + 1, kONumBars = kOBarFin + 1;
constexpr int kOOffTail = kOOffBar + kONumBars * 8;
constexpr int kTailBytes = 32;  // tmem base, abort flag, resc slot, [tile total, first sequence, its first tile]
constexpr int kSmemBytes = kSEnd > kOOffTail + kTailBytes ? kSEnd : kOOffTail + kTailBytes;
static_assert(kSmemBytes <= 232448, "shared memory budget");
static_assert(kSOffTail + kTailBytes <= kSOffQT, "barriers and tail fit the gap behind staging buffer 0");
static_assert(kSOffQR % 1024 == 0 && kSOffStage0 % 1024 == 0 && kSOffStage1 % 1024 == 0 && kOOffMsg % 1024 == 0 &&
                  kMsgStride % 1024 == 0 && kTileBytes % 1024 == 0,
              "swizzle atoms 1024-aligned");
static_assert(kOOffBar % 8 == 0 && kSOffBar % 8 == 0 && kSOffScale % 16 == 0 && kSOffExp % 16 == 0, "alignment");
static_assert(kMsgBytes % 16 == 0 && kSoftWarps * 32 * 128 <= kPBytes, "bulk copy size; transpose tiles");

__device__ __forceinline__ void raise_abort(volatile int* abort_flag, uint32_t peer_abort, int32_t* dev_status) {
    *abort_flag = 1;
    st_cluster_u32(peer_abort, 1u);
    if (dev_status) atomicOr(dev_status, MLA_DEVERR_TIMEOUT);
}

__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }
__device__ __forceinline__ float fmax64(const float (&v)[64]) {
    float a = v[0], b = v[1], c = v[2], d = v[3];
#pragma unroll
    for (int k = 4; k < 60; k += 8) {
        a = max3(a, v[k], v[k + 1]);
        b = max3(b, v[k + 2], v[k + 3]);
        c = max3(c, v[k + 4], v[k + 5]);
        d = max3(d, v[k + 6], v[k + 7]);
    }
    return max3(max3(a, b, c), max3(d, v[60], v[61]), fmaxf(v[62], v[63]));
}

__global__ void __launch_bounds__(kThreads, 1) decode8_tc_kernel(const Params p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_ctarank();  // 0: S CTA, 1: O CTA
    const uint32_t peer = rank ^ 1u;
    const int tail = rank == 0 ? kSOffTail : kOOffTail;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + (rank == 0 ? kSOffBar : kOOffBar));
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + tail);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + tail + 4);
    volatile int* resc_pb = reinterpret_cast<volatile int*>(smem + tail + 8);
    int* first = reinterpret_cast<int*>(smem + tail + 12);
    volatile int never = 0;  // abort flag for teardown waits (never raised)

    if ((sbase & 1023u) != 0) {  // identical in both CTAs: both leave here
        if (tid == 0 && p.dev_status) atomicOr(p.dev_status, MLA_DEVERR_TIMEOUT);
        return;
    }
    if (tid == 0) {
        if (rank == 0) {
            for (int i = 0; i < 4; ++i) {
                mbar_init(&bars[kSBarFull + i], 1);
                mbar_init(&bars[kSBarEmpty + i], 1);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(&bars[kSBarSFull + i], 1);
                mbar_init(&bars[kSBarSEmpty + i], kSoftThreads);
            }
            for (int i = 0; i < kPSlots; ++i) mbar_init(&bars[kSBarPEmpty + i], 1);
            mbar_init(&bars[kSBarQReady], kSoftThreads);
            mbar_init(&bars[kSBarFin], 1);
        } else {
            for (int i = 0; i < kVStages; ++i) {
                mbar_init(&bars[kOBarVFull + i], 1);
                mbar_init(&bars[kOBarVEmpty + i], 1);
            }
            for (int i = 0; i < kPSlots; ++i) mbar_init(&bars[kOBarPFull + i], 1);
            mbar_init(&bars[kOBarOFull], 1);
            mbar_init(&bars[kOBarOFree], kRows);
            mbar_init(&bars[kOBarRescReq], 1);
            mbar_init(&bars[kOBarRescDone], kRows);
            mbar_init(&bars[kOBarODrain], 1);
            mbar_init(&bars[kOBarFin], 1);
        }
        *abort_flag = 0;
        *resc_pb = 0;
        fence_mbar_init();
    }
    if (warp == kWarpProducer) tmem_alloc(tmem_slot, 512);
    // everything above touches only this CTA's own resources; the call's inputs are read after this wait
    grid_dependency_wait();
    const int cid = static_cast<int>(blockIdx.x >> 1);
    const int g = cid / p.P_g, pidx = cid % p.P_g;
    if (warp == 0) find_first(p, pidx, lane, first);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    cluster_sync();  // peer barriers initialised before any remote arrive
    const uint32_t tmem = *tmem_slot;
    const int Nt = first[0];
    const bool active = g < p.G;
    SegWalk walk;
    walk.b = first[1];
    walk.tb = first[2];
    walk.lo = static_cast<int>((static_cast<int64_t>(pidx) * Nt) / p.P_g);
    walk.hi = static_cast<int>((static_cast<int64_t>(pidx + 1) * Nt) / p.P_g);
    walk.pidx = pidx;
    const uint32_t peer_abort = mapa(sbase + (rank == 0 ? kOOffTail : kSOffTail) + 4, peer);
    const int64_t out_row_base = (static_cast<int64_t>(g) * p.slots) * kRows;

    if (active && rank == 0) {
        // =============================================================== S CTA
        if (warp == kWarpProducer) {
            // ---- copy producer: marked to stay in L2 for the O CTA's read of the latent part
            if (lane == 0) {
                SegWalk w = walk;
                Seg s;
                uint32_t n = 0;  // tiles
                bool ok = true;
                const uint64_t keep = l2_policy_evict_last();
                while (ok && w.next(p, s)) {
                    for (int t = s.t0; ok && t < s.t1; ++t, ++n) {
                        const uint8_t* src = block_of(p, s.tab[t], true);
                        const uint32_t u = n >> 1, base = (n & 1u) * kTileBytes, bi = 2 * (n & 1u);
                        ok = mbar_wait(&bars[kSBarEmpty + bi], (u & 1u) ^ 1u, abort_flag, kLimitNs);
                        if (!ok) break;
                        mbar_arrive_expect_tx(&bars[kSBarFull + bi], kCopyA);
                        bulk_load_hint(sbase + kSOffRing + base, src, kCopyA, &bars[kSBarFull + bi], keep);
                        ok = mbar_wait(&bars[kSBarEmpty + bi + 1], (u & 1u) ^ 1u, abort_flag, kLimitNs);
                        if (!ok) {
                            mbar_wait(&bars[kSBarFull + bi], u & 1u, &never, kLimitNs);
                            break;
                        }
                        mbar_arrive_expect_tx(&bars[kSBarFull + bi + 1], kCopyB);
                        bulk_load_hint(sbase + kSOffRing + base + kCopyA, src + kCopyA, kCopyB,
                                       &bars[kSBarFull + bi + 1], keep);
                    }
                }
                if (!ok) raise_abort(abort_flag, peer_abort, p.dev_status);
                // let every issued copy land before the CTA can exit
                for (uint32_t i = (n > 2 ? n - 2 : 0); i < n; ++i)
                    for (int k = 0; k < 2; ++k)
                        mbar_wait(&bars[kSBarFull + 2 * (i & 1u) + k], (i >> 1) & 1u, &never, kLimitNs);
            }
        } else if (warp == kWarpMma) {
            // ---- MMA issuer (one thread): S[sb] = (Q_hi + Q_lo) K^T
            if (elect_one()) {
                constexpr uint32_t idesc = idesc_f8_f32(kRows, kTile, false, false);
                const uint64_t ring_desc = sdesc_sw128(sbase + kSOffRing, 16, 1024);
                const uint64_t rope_desc = sdesc_sw64(sbase + kSOffRing + kBlock8Rope, 16, 512);
                const uint64_t qr_desc = sdesc_sw128(sbase + kSOffQR, 16, 1024);
                SegWalk w = walk;
                Seg s;
                uint32_t n = 0, kseg = 0;
                bool ok = true;
                while (ok && w.next(p, s)) {
                    ok = mbar_wait(&bars[kSBarQReady], kseg & 1u, abort_flag, kLimitNs);
                    ++kseg;
                    for (int t = s.t0; ok && t < s.t1; ++t, ++n) {
                        const uint32_t sb = n & 1u, us = n >> 1;
                        ok = mbar_wait(&bars[kSBarSEmpty + sb], (us & 1u) ^ 1u, abort_flag, kLimitNs);
                        const uint32_t d = tmem + col_s(sb);
                        const uint64_t tile_off = static_cast<uint64_t>(sb * kTileBytes) >> 4;
#pragma unroll 1
                        for (int k = 0; ok && k < 2; ++k) {
                            ok = mbar_wait(&bars[kSBarFull + 2 * sb + k], us & 1u, abort_flag, kLimitNs);
                            if (!ok) break;
                            tc_fence_after();
                            // rolled: code that fits the instruction cache beside the softmax warps' (fully unrolled, the
                            // issue of a tile's 36 MMAs took longer than their 2304 cycles)
#pragma unroll 1
                            for (int j = 0; j < 2; ++j) {
                                const int c = 2 * k + j;
                                const uint64_t cd = ring_desc + tile_off + (static_cast<uint64_t>(c * kChunk) >> 4);
                                const uint32_t qa = tmem + kColQ + 32 * c;
#pragma unroll
                                for (int kk = 0; kk < 4; ++kk) {
                                    mma8_ts(d, qa + 8 * kk, cd + 2 * kk, idesc, (c | kk) ? 1u : 0u);
                                    mma8_ts(d, qa + 128 + 8 * kk, cd + 2 * kk, idesc, 1u);
                                }
                            }
                            if (k == 1) {
                                const uint64_t rd = rope_desc + tile_off;
#pragma unroll
                                for (int kk = 0; kk < 2; ++kk) {
                                    mma8_ss(d, qr_desc + 2 * kk, rd + 2 * kk, idesc, 1u);
                                    mma8_ss(d, qr_desc + 4 + 2 * kk, rd + 2 * kk, idesc, 1u);
                                }
                            }
                            mma_commit(smem_u32(&bars[kSBarEmpty + 2 * sb + k]));
                        }
                        if (ok) mma_commit(smem_u32(&bars[kSBarSFull + sb]));
                    }
                }
                if (!ok) raise_abort(abort_flag, peer_abort, p.dev_status);
                mma_commit(smem_u32(&bars[kSBarFin]));
                mbar_wait(&bars[kSBarFin], 0, &never, kLimitNs);
            }
            __syncwarp();
        } else if (warp < kSoftWarps) {
            // ---- softmax: warp (qd, hf) owns TMEM lanes 32 qd.. (query rows) and score columns 64 hf .. 64 hf + 63
            const int qd = warp & 3, hf = warp >> 2;
            const int r = 32 * qd + lane;
            const uint32_t t_lane = tmem + (static_cast<uint32_t>(32 * qd) << 16);
            // exchange with the warp of the same rows' other half: block 4 hf + qd (the last one apart)
            auto xblock = [&](int h) {
                const int i = 4 * h + qd;
                return reinterpret_cast<float*>(smem + (i < 7 ? kSOffXchg + 128 * i : kSOffX7)) + lane;
            };
            volatile float* xmine = xblock(hf);
            volatile float* xother = xblock(hf ^ 1);
            const int rr = g * kRows + r;
            const bool row_ok = rr < p.R;
            const int j = row_ok ? rr / p.H : 0;
            SegWalk w = walk, wn;
            Seg s, sn;
            uint32_t n = 0;
            bool failed = false;
            bool have = w.next(p, s);
            while (!failed && have) {
                wn = w;
                const bool have_next = wn.next(p, sn);
                const int64_t qrow0 = static_cast<int64_t>(s.b) * p.R + g * kRows + 32 * qd;
                const int t_pf = max(s.t0, s.t1 - 2);
                const char* nq = (have_next && row_ok) ? reinterpret_cast<const char*>(
                                                              p.q + (static_cast<int64_t>(sn.b) * p.R + rr) * kRow)
                                                        : nullptr;
                // token r's scale in the tiles to come (the warps of hf = 0): that of tile t + 1 and the table entry of
                // tile t + 2 are under way while tile t is worked on
                auto entry = [&](int t) { return (hf == 0 && t < s.t1) ? s.tab[t] : 0; };
                auto scale_bits = [&](int32_t e, int t) {
                    return (hf == 0 && t < s.t1 && t * kTile + r < s.L)
                               ? reinterpret_cast<const uint32_t*>(block_of(p, e, false) + kBlock8Scales)[r]
                               : 0x3F800000u;
                };
                auto put_scale = [&](uint32_t bits) {  // s = 2^k, k, 2^-k
                    reinterpret_cast<uint32_t*>(smem + kSOffScale)[r] = bits;
                    reinterpret_cast<float*>(smem + kSOffExp)[r] = static_cast<float>(static_cast<int>(bits >> 23) - 127);
                    reinterpret_cast<uint32_t*>(smem + kSOffInv)[r] = 0x7F000000u - bits;
                };
                const int32_t e0 = entry(s.t0), e1 = entry(s.t0 + 1);
                int32_t e2 = entry(s.t0 + 2);
                // this segment's query rows, two e4m3 terms each: latent part -> TMEM (warps of hf = 0: columns 0..255
                // of a row, hf = 1: 256..511), RoPE part -> shared memory.  The warp loads its 32 rows coalesced (a
                // lane per 16-byte unit) and transposes each 64-column chunk through a swizzled 4 KB tile into the
                // lane-per-row order of tcgen05.st.  The bf16 rows wait in the score buffers (free between segments)
                // until the row's largest magnitude is known.
                float rowf;
                {
                    uint8_t* qt = smem + kSOffQT + warp * (32 * 128);
                    const int lu = lane & 7, lr = lane >> 3;  // unit and row-in-quad of this lane's loads
                    const uint32_t raw = t_lane + kColS0 + 128 * hf;
                    uint32_t m2 = 0;
                    uint4 y[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int ri = 8 * i + (lane >> 2);
                        y[i] = make_uint4(0, 0, 0, 0);
                        if (g * kRows + 32 * qd + ri < p.R)
                            y[i] = reinterpret_cast<const uint4*>(p.q + (qrow0 + ri) * kRow)[64 + 4 * hf + (lane & 3)];
                    }
#pragma unroll 1
                    for (int c = 0; c < 4; c += 2) {
                        uint4 x[2][8];
#pragma unroll
                        for (int jj = 0; jj < 2; ++jj)
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const int ri = 4 * i + lr;
                                x[jj][i] = make_uint4(0, 0, 0, 0);
                                if (g * kRows + 32 * qd + ri < p.R)
                                    x[jj][i] = reinterpret_cast<const uint4*>(
                                        p.q + (qrow0 + ri) * kRow)[8 * (4 * hf + c + jj) + lu];
                            }
                        if (c == 0) {
                            if (hf == 0) put_scale(scale_bits(e0, s.t0));
                            // the transpose tiles double as staging buffer 1: before the first write to them, wait
                            // until the sender has seen every copy of earlier messages read out
                            bar_sync(kNbQFree, kSyncThreads);
                        }
#pragma unroll
                        for (int jj = 0; jj < 2; ++jj) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const int ri = 4 * i + lr;
                                *reinterpret_cast<uint4*>(qt + ri * 128 + ((lu ^ (ri & 7)) << 4)) = x[jj][i];
                            }
                            __syncwarp();
                            uint32_t v[32];
#pragma unroll
                            for (int u = 0; u < 8; ++u) {
                                const uint4 z = *reinterpret_cast<const uint4*>(qt + lane * 128 + ((u ^ (lane & 7)) << 4));
                                v[4 * u] = z.x; v[4 * u + 1] = z.y; v[4 * u + 2] = z.z; v[4 * u + 3] = z.w;
                                m2 = max_abs2(max_abs2(max_abs2(max_abs2(m2, z.x), z.y), z.z), z.w);
                            }
                            __syncwarp();
                            tmem_st32(raw + 32 * (c + jj), v);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int ri = 8 * i + (lane >> 2);
                        *reinterpret_cast<uint4*>(qt + ri * 128 + (((lane & 3) ^ (ri & 7)) << 4)) = y[i];
                    }
                    __syncwarp();
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        y[u] = *reinterpret_cast<const uint4*>(qt + lane * 128 + ((u ^ (lane & 7)) << 4));
                        m2 = max_abs2(max_abs2(max_abs2(max_abs2(m2, y[u].x), y[u].y), y[u].z), y[u].w);
                    }
                    // the row's largest magnitude, over both halves of its columns
                    const uint32_t mine = max(m2 & 0xFFFFu, m2 >> 16);
                    *xmine = __uint_as_float(mine);
                    bar_sync(1 + qd, 64);
                    const uint32_t top = max(mine, __float_as_uint(*xother));
                    const int a = top < 0x7F80u ? row_exp(top) : 0;
                    const float inv = exp2_int(-a);
                    // an infinity or NaN in the query: every score of the row is NaN
                    rowf = top < 0x7F80u ? exp2_int(a) * p.scale_log2 : CUDART_NAN_F;
                    uint8_t* qr = smem + kSOffQR + r * 128;
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        uint4 hi, lo;
                        split4_q(y[2 * u].x, y[2 * u].y, inv, hi.x, lo.x);
                        split4_q(y[2 * u].z, y[2 * u].w, inv, hi.y, lo.y);
                        split4_q(y[2 * u + 1].x, y[2 * u + 1].y, inv, hi.z, lo.z);
                        split4_q(y[2 * u + 1].z, y[2 * u + 1].w, inv, hi.w, lo.w);
                        *reinterpret_cast<uint4*>(qr + (((2 * hf + u) ^ (r & 7)) << 4)) = hi;
                        *reinterpret_cast<uint4*>(qr + (((4 + 2 * hf + u) ^ (r & 7)) << 4)) = lo;
                    }
                    tmem_wait_st();
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t v[32], hi[32], lo[32];
                        tmem_ld32(raw + 32 * c, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int u = 0; u < 16; ++u) split4_q(v[2 * u], v[2 * u + 1], inv, hi[u], lo[u]);
                        tmem_st16(t_lane + kColQ + 16 * (4 * hf + c), hi);
                        tmem_st16(t_lane + kColQ + 128 + 16 * (4 * hf + c), lo);
                    }
                }
                fence_proxy_async_cta();
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&bars[kSBarQReady]);
                uint32_t sc1 = scale_bits(e1, s.t0 + 1);
                const int lim = row_ok ? (s.L - p.n_q + j + 1) : 0;  // keys 0 .. lim-1 are visible
                RowRef ref;
                ref.reset();
                float l = 0.f;
                for (int t = s.t0; t < s.t1; ++t, ++n) {
                    const uint32_t sb = n & 1u, us = n >> 1;
                    if (t == t_pf && have_next && row_ok)
                        for (int c = hf; c < 9; c += 2) prefetch_l2(nq + 128 * c);
                    bool ok = mbar_wait(&bars[kSBarSFull + sb], us & 1u, abort_flag, kLimitNs);
                    __syncwarp();
                    tc_fence_after();
                    float y[64];
                    {
                        uint32_t a[32], b[32];
                        tmem_ld32(t_lane + col_s(sb) + 64 * hf, a);
                        tmem_ld32(t_lane + col_s(sb) + 64 * hf + 32, b);
                        tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            y[k] = __uint_as_float(a[k]);
                            y[32 + k] = __uint_as_float(b[k]);
                        }
                    }
                    tc_fence_before();
                    mbar_arrive(&bars[kSBarSEmpty + sb]);
                    // y = log2(p s_t), before the reference: S s_t (2^a scale log2 e) + log2 s_t
                    const float4* sc4 = reinterpret_cast<const float4*>(smem + kSOffScale) + 16 * hf;
                    const float4* ex4 = reinterpret_cast<const float4*>(smem + kSOffExp) + 16 * hf;
                    const float4* in4 = reinterpret_cast<const float4*>(smem + kSOffInv) + 16 * hf;
                    const float2 rowf2 = make_float2(rowf, rowf);
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const float4 sv = sc4[k], ev = ex4[k];
                        const float2 y0 = fma2(mul2(make_float2(y[4 * k], y[4 * k + 1]), make_float2(sv.x, sv.y)), rowf2,
                                               make_float2(ev.x, ev.y));
                        const float2 y1 = fma2(mul2(make_float2(y[4 * k + 2], y[4 * k + 3]), make_float2(sv.z, sv.w)),
                                               rowf2, make_float2(ev.z, ev.w));
                        y[4 * k] = y0.x;
                        y[4 * k + 1] = y0.y;
                        y[4 * k + 2] = y1.x;
                        y[4 * k + 3] = y1.y;
                    }
                    const int nvalid = lim - t * kTile - 64 * hf;  // columns < nvalid are visible
                    if (nvalid < 64) {
#pragma unroll
                        for (int k = 0; k < 64; ++k) y[k] = k < nvalid ? y[k] : -CUDART_INF_F;
                    }
                    const float half_top = fmax64(y);
                    *xmine = half_top;
                    bar_sync(1 + qd, 64);
                    const int d = ref.move(fmaxf(half_top, *xother));
                    const float2 mneg = make_float2(ref.minus(), ref.minus());
                    float2 ls0 = make_float2(0.f, 0.f), ls1 = ls0;
                    uint32_t hi[16], lo[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const float4 iv = in4[k];
                        float2 p0 = add2(make_float2(y[4 * k], y[4 * k + 1]), mneg);
                        float2 p1 = add2(make_float2(y[4 * k + 2], y[4 * k + 3]), mneg);
                        p0 = make_float2(ex2_approx(p0.x), ex2_approx(p0.y));
                        p1 = make_float2(ex2_approx(p1.x), ex2_approx(p1.y));
                        ls0 = fma2(p0, make_float2(iv.x, iv.y), ls0);
                        ls1 = fma2(p1, make_float2(iv.z, iv.w), ls1);
                        split4_p(p0.x, p0.y, p1.x, p1.y, dither_pair(2 * k), dither_pair(2 * k + 1), hi[k], lo[k]);
                    }
                    const float lsum = (ls0.x + ls0.y) + (ls1.x + ls1.y);
                    l = fmaf(l, RowRef::factor(d), lsum);
                    if (bar_red_or(kNbFail, kSyncThreads, !ok || *abort_flag != 0)) {
                        failed = true;
                        break;
                    }
                    // every reader of this tile's scales is past them
                    if (hf == 0) put_scale(sc1);
                    sc1 = scale_bits(e2, t + 2);
                    e2 = entry(t + 3);
                    // the sender has seen the copy that last used this staging buffer (tile n - 2) read it
                    bar_sync(kNbStageFree, kSyncThreads);
                    uint8_t* stage = smem + ((n & 1u) ? kSOffStage1 : kSOffStage0);
                    // row r, columns 64 hf ..: 16-byte units 4 hf + u at ((4 hf + u) ^ (r % 8)) of the hi and lo chunks
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        uint8_t* at = stage + r * 128 + (((4 * hf + u) ^ (r & 7)) << 4);
                        *reinterpret_cast<uint4*>(at) = make_uint4(hi[4 * u], hi[4 * u + 1], hi[4 * u + 2], hi[4 * u + 3]);
                        *reinterpret_cast<uint4*>(at + kRows * kTile) =
                            make_uint4(lo[4 * u], lo[4 * u + 1], lo[4 * u + 2], lo[4 * u + 3]);
                    }
                    if (hf == 0) reinterpret_cast<int8_t*>(stage + kPBytes)[r] = static_cast<int8_t>(d);
                    fence_proxy_async_cta();
                    bar_arrive(kNbStaged, kSyncThreads);
                }
                if (failed) break;
                // segment result: (R, l) with l summed over both column halves; a NaN sum keeps its piece
                if (hf == 1) *xmine = l;
                bar_sync(1 + qd, 64);
                if (hf == 0 && row_ok) {
                    const float lt = l + *xother;
                    p.ml_part[out_row_base + static_cast<int64_t>(s.slot) * kRows + r] =
                        make_float2(lt != lt ? 0.f : ref.R, lt);
                }
                bar_sync(1 + qd, 64);
                w = wn;
                s = sn;
                have = have_next;
            }
            if (failed && tid == 0) raise_abort(abort_flag, peer_abort, p.dev_status);
        } else if (warp == kWarpSender) {
            // ---- sender: ships each staged P tile (one bulk copy, completing on the O CTA's barrier) once the O CTA
            //      has released that message slot.  Takes the same per-tile barrier steps as the softmax warps.
            const uint32_t peer_msg = mapa(sbase + kOOffMsg, peer);
            const uint32_t peer_pfull = mapa(sbase + kOOffBar + kOBarPFull * 8, peer);
            SegWalk w = walk;
            Seg s;
            uint32_t n = 0;
            bool failed = false;
            while (!failed && w.next(p, s)) {
                // every staged message read out before the Q reload reuses staging buffer 1
                if (lane == 0) bulk_wait_group_read<0>();
                __syncwarp();
                bar_arrive(kNbQFree, kSyncThreads);
                for (int t = s.t0; t < s.t1; ++t, ++n) {
                    const uint32_t pb = n % kPSlots, up = n / kPSlots;
                    if (bar_red_or(kNbFail, kSyncThreads, *abort_flag != 0)) {
                        failed = true;
                        break;
                    }
                    if (lane == 0) bulk_wait_group_read<1>();
                    __syncwarp();
                    bar_arrive(kNbStageFree, kSyncThreads);
                    bar_sync(kNbStaged, kSyncThreads);
                    if (lane == 0) {
                        if (mbar_wait<true>(&bars[kSBarPEmpty + pb], (up & 1u) ^ 1u, abort_flag, kLimitNs)) {
                            mbar_arrive_expect_tx_remote(peer_pfull + 8 * pb, kMsgBytes);
                            bulk_copy_to_peer(peer_msg + pb * kMsgStride,
                                              sbase + ((n & 1u) ? kSOffStage1 : kSOffStage0), kMsgBytes,
                                              peer_pfull + 8 * pb);
                            bulk_commit_group();
                        } else {
                            raise_abort(abort_flag, peer_abort, p.dev_status);
                        }
                    }
                    __syncwarp();
                }
            }
            if (lane == 0) {
                bulk_wait_group_read<0>();
                // the O CTA's last releases of its message slots arrive here: they have to land before this CTA ends
                for (uint32_t i = (n > kPSlots ? n - kPSlots : 0); !failed && i < n; ++i)
                    mbar_wait<true>(&bars[kSBarPEmpty + i % kPSlots], (i / kPSlots) & 1u, abort_flag, kLimitNs);
            }
            __syncwarp();
        }
    } else if (active && rank == 1) {
        // =============================================================== O CTA
        if (warp == kWarpProducer) {
            // ---- copy producer: the four latent chunks of each block as two copies of two, into the ring of V stages
            if (lane == 0) {
                SegWalk w = walk;
                Seg s;
                uint32_t nv = 0;  // stage loads issued
                bool ok = true;
                const uint64_t last_use = l2_policy_evict_first();
                while (ok && w.next(p, s)) {
                    for (int t = s.t0; ok && t < s.t1; ++t) {
                        const uint8_t* src = block_of(p, s.tab[t], true);
                        for (int k = 0; k < 2; ++k, ++nv) {
                            const uint32_t st = nv % kVStages, u = nv / kVStages;
                            ok = mbar_wait(&bars[kOBarVEmpty + st], (u & 1u) ^ 1u, abort_flag, kLimitNs);
                            if (!ok) break;
                            mbar_arrive_expect_tx(&bars[kOBarVFull + st], kVStageBytes);
                            bulk_load_hint(sbase + kOOffV + st * kVStageBytes, src + k * kVStageBytes, kVStageBytes,
                                           &bars[kOBarVFull + st], last_use);
                        }
                    }
                }
                if (!ok) raise_abort(abort_flag, peer_abort, p.dev_status);
                for (uint32_t i = (nv > kVStages ? nv - kVStages : 0); i < nv; ++i)
                    mbar_wait(&bars[kOBarVFull + i % kVStages], (i / kVStages) & 1u, &never, kLimitNs);
            }
        } else if (warp == kWarpMma) {
            // ---- MMA issuer: O += (P_hi + P_lo) V (A = P, K-major SW128; B = V, MN-major SW128, 16 KB between atoms of
            //      128 columns)
            constexpr uint32_t idesc_hi = idesc_f8_f32(kRows, 256, false, true);
            constexpr uint32_t idesc_lo = idesc_f8_f32(kRows, 256, false, true, true);
            const uint32_t peer_pempty = mapa(sbase + kSOffBar + kSBarPEmpty * 8, peer);
            const uint64_t p_desc = sdesc_sw128(sbase + kOOffMsg, 16, 1024);
            const uint64_t v_desc = sdesc_sw128(sbase + kOOffV, kChunk, 1024);
            const bool leader = elect_one();
            SegWalk w = walk;
            Seg s;
            uint32_t n = 0, nv = 0, kseg = 0, nresc = 0;
            bool ok = true;
            while (ok && w.next(p, s)) {
                for (int t = s.t0; ok && t < s.t1; ++t, ++n) {
                    const uint32_t pb = n % kPSlots, up = n / kPSlots;
                    const bool fresh = (t == s.t0);
                    if (leader) {
                        ok = mbar_wait<true>(&bars[kOBarPFull + pb], up & 1u, abort_flag, kLimitNs);
                        if (ok && fresh) ok = mbar_wait(&bars[kOBarOFree], (kseg & 1u) ^ 1u, abort_flag, kLimitNs);
                    }
                    ok = __any_sync(0xffffffffu, ok && leader);
                    if (!ok) break;
                    const uint8_t* msg = smem + kOOffMsg + pb * kMsgStride;
                    const bool resc = __any_sync(0xffffffffu, reinterpret_cast<const uint32_t*>(msg + kPBytes)[lane] != 0);
                    if (!fresh && resc) {
                        // some row's reference moved: have the epilogue rescale O once all earlier MMAs are done
                        if (leader) {
                            *resc_pb = static_cast<int>(pb);
                            mma_commit(smem_u32(&bars[kOBarODrain]));
                            mbar_arrive(&bars[kOBarRescReq]);
                            ok = mbar_wait(&bars[kOBarRescDone], nresc & 1u, abort_flag, kLimitNs);
                        }
                        ++nresc;
                        ok = __any_sync(0xffffffffu, ok && leader);
                        if (!ok) break;
                    }
                    const int nvalid = min(kTile, s.L - t * kTile);
#pragma unroll 1
                    for (int k = 0; k < 2; ++k, ++nv) {
                        const uint32_t st = nv % kVStages, u = nv / kVStages;
                        if (leader) ok = mbar_wait(&bars[kOBarVFull + st], u & 1u, abort_flag, kLimitNs);
                        ok = __any_sync(0xffffffffu, ok && leader);
                        if (!ok) break;
                        uint8_t* vst = smem + kOOffV + st * kVStageBytes;
                        if (nvalid < kTile) {
                            // rows past the sequence end: P is 0 there, make V 0 too (no 0 * NaN)
                            const int nz = (kTile - nvalid) * 8;  // 16-byte units per chunk
                            for (int i = lane; i < 2 * nz; i += 32) {
                                const int c = i / nz, q = i % nz;
                                *reinterpret_cast<uint4*>(vst + c * kChunk + nvalid * 128 + q * 16) =
                                    make_uint4(0, 0, 0, 0);
                            }
                            fence_proxy_async_cta();
                        }
                        __syncwarp();
                        if (leader) {
                            tc_fence_after();
                            const uint64_t vd = v_desc + (static_cast<uint64_t>(st * kVStageBytes) >> 4);
                            const uint64_t pd = p_desc + (static_cast<uint64_t>(pb * kMsgStride) >> 4);
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk) {
                                mma8_ss(tmem + 256 * k, pd + 2 * kk, vd + ((kk * 4096) >> 4), idesc_hi,
                                        (fresh && kk == 0) ? 0u : 1u);
                                mma8_ss(tmem + 256 * k, pd + ((kRows * kTile) >> 4) + 2 * kk, vd + ((kk * 4096) >> 4),
                                        idesc_lo, 1u);
                            }
                            mma_commit(smem_u32(&bars[kOBarVEmpty + st]));
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                    if (leader) mma_commit(peer_pempty + 8 * pb);
                    __syncwarp();
                }
                if (!ok) break;
                if (leader) mma_commit(smem_u32(&bars[kOBarOFull]));
                __syncwarp();
                ++kseg;
            }
            if (!ok && leader) raise_abort(abort_flag, peer_abort, p.dev_status);
            if (leader) {
                mma_commit(smem_u32(&bars[kOBarFin]));
                mbar_wait(&bars[kOBarFin], 0, &never, kLimitNs);
            }
            __syncwarp();
        } else if (warp < 4) {
            // ---- epilogue: warps 0..3, one thread per query row
            const int r = tid;
            const uint32_t t_lane = tmem + (static_cast<uint32_t>(warp * 32) << 16);
            SegWalk w = walk;
            Seg s;
            uint32_t kseg = 0, nresc = 0;
            bool ok = true;
            while (ok && w.next(p, s)) {
                // serve rescale requests until this segment's O is complete.  Lane 0 polls; the warp then waits
                // together so tcgen05.ld/st stay converged.
                const uint64_t t0 = globaltimer_ns();
                uint32_t it = 0;
                for (;;) {
                    int ev = 0;  // 1: O complete, 2: rescale request, 3: give up
                    if (lane == 0) {
                        if (mbar_test(smem_u32(&bars[kOBarOFull]), kseg & 1u)) ev = 1;
                        else if (mbar_test(smem_u32(&bars[kOBarRescReq]), nresc & 1u)) ev = 2;
                        else if (*abort_flag) ev = 3;
                        else if ((++it & 255u) == 0 && globaltimer_ns() - t0 > kLimitNs) ev = 3;
                    }
                    ev = __shfl_sync(0xffffffffu, ev, 0);
                    if (ev == 1) {
                        ok = mbar_wait(&bars[kOBarOFull], kseg & 1u, abort_flag, kLimitNs);
                        break;
                    }
                    if (ev == 3) {
                        ok = false;
                        break;
                    }
                    if (ev == 2) {
                        ok = mbar_wait(&bars[kOBarRescReq], nresc & 1u, abort_flag, kLimitNs) &&
                             mbar_wait(&bars[kOBarODrain], nresc & 1u, abort_flag, kLimitNs);
                        __syncwarp();
                        tc_fence_after();
                        const int d =
                            reinterpret_cast<const int8_t*>(smem + kOOffMsg + *resc_pb * kMsgStride + kPBytes)[r];
                        if (__any_sync(0xffffffffu, d != 0)) {
                            const float a = RowRef::factor(d);
#pragma unroll 1
                            for (int c = 0; c < 16; ++c) {
                                uint32_t v[32];
                                tmem_ld32(t_lane + 32 * c, v);
                                tmem_wait_ld();
#pragma unroll
                                for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * a);
                                tmem_st32(t_lane + 32 * c, v);
                            }
                            tmem_wait_st();
                        }
                        tc_fence_before();
                        mbar_arrive(&bars[kOBarRescDone]);
                        ++nresc;
                        if (!__all_sync(0xffffffffu, ok)) {
                            ok = false;
                            break;
                        }
                        continue;
                    }
                    __nanosleep(256);
                }
                ok = __all_sync(0xffffffffu, ok);
                __syncwarp();
                if (!ok) break;
                tc_fence_after();
                // column group j (4 latent columns) of all 128 rows is contiguous: 512 consecutive bytes a warp store
                float4* oseg = reinterpret_cast<float4*>(p.o_part) +
                               (out_row_base + static_cast<int64_t>(s.slot) * kRows) * (kDc / 4);
#pragma unroll 1
                for (int c = 0; c < 16; ++c) {
                    uint32_t v[32];
                    tmem_ld32(t_lane + 32 * c, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        oseg[(8 * c + k) * kRows + r] =
                            make_float4(__uint_as_float(v[4 * k]), __uint_as_float(v[4 * k + 1]),
                                        __uint_as_float(v[4 * k + 2]), __uint_as_float(v[4 * k + 3]));
                }
                tc_fence_before();
                mbar_arrive(&bars[kOBarOFree]);
                ++kseg;
            }
            if (!ok && lane == 0) raise_abort(abort_flag, peer_abort, p.dev_status);
        }
    }

    // ------------------------------------------------------------------ teardown
    grid_dependents_launch();  // the merge kernel may be scheduled; it waits for this grid to finish
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // the peer no longer touches this CTA's shared memory
    if (warp == kWarpProducer) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace tc8

cudaError_t launch_decode8_tc(const uint16_t* q, const uint8_t* cache, int64_t cap_blocks, const int32_t* block_table,
                              int max_blocks, const int32_t* kv_len, int B, int n_q, int H, float scale, int P_g,
                              float* o_part, float2* ml_part, int slots, int32_t* dev_status, cudaStream_t stream) {
    const int R = n_q * H;
    d8::Params prm = {q, cache, block_table, kv_len, o_part, ml_part, dev_status, cap_blocks, max_blocks, B, n_q, H, R,
                      (R + tc8::kRows - 1) / tc8::kRows, P_g, slots, tc8::kRows, scale * 1.44269504088896340736f};
    if (P_g < 1 || B + P_g > slots) return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(tc8::decode8_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         tc8::kSmemBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * prm.G * P_g);
    cfg.blockDim = dim3(tc8::kThreads);
    cfg.dynamicSmemBytes = tc8::kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, tc8::decode8_tc_kernel, prm);
}

}  // namespace mla
