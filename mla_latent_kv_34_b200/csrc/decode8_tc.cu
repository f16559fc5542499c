// Absorbed MLA decode over the 8-bit cache on the tensor cores (tcgen05 + TMEM), more than 48 query rows.
//
// The step is mla_decode's (decode_tc.cu): a cluster of two CTAs owns 128 query rows, the "S" CTA forms the scores and
// the softmax, the "O" CTA keeps O[128 x 512] in its whole tensor memory and accumulates P V; the (sequence, tile)
// space is cut into equal ranges, one per cluster, and a range's pieces of sequences go to the workspace for the merge
// (finish8.cu).  What differs is that a cached row is c_t = s_t code_t with e4m3 codes:
//   - the codes are the operands of both contractions as they lie in the block (kind::f8f6f4, K = 32): no
//     dequantisation, half the bytes from HBM and through shared memory.  Q and P are written as hi + lo terms
//     (decode8_common.cuh), so Q is exact and P keeps 8 significant bits; two K = 32 MMAs at twice the bf16 rate
//     cost what the bf16 MMA of the same elements costs;
//   - scores: y = S s_t (2^a scale log2 e) + log2 s_t with the query row's power of two 2^a; P' = 2^(y - R) carries
//     s_t, because the rows of V are codes, and the row's sums take P' / s_t.  R is RowRef's reference exponent;
//   - a tile (72 KB of codes) comes as copies of 32 and 40 KB into a ring that holds two tiles, so a tile's copies are
//     under way while the one before it is multiplied.
// S CTA: the query's latent part in TMEM (hi 128 columns, lo 128 columns), its RoPE part in shared memory, two score
// buffers of 128 columns; 36 MMAs (M = 128, N = 128) a tile.  O CTA: 16 MMAs (M = 128, N = 256) a tile, P from shared memory.
//
// Softmax: sixteen warps, (quadrant of 32 rows) x (quarter tile of 32 tokens); a thread has two rows and 16 tokens, so the
// tokens' scales are unpacked once for two rows.  The four units of a row in a tile follow one another only in R, which a
// warp hands to the next as soon as its maximum is known; nothing else holds the warps in step.  P goes out in messages of
// two units: staged in shared memory, one bulk copy to the O CTA's slot, whose barrier the O CTA arms itself.
//
// What bounds it: a tile takes 2.2 us (4 sequences over 8 to 40 tiles a pair), for 2304 cycles of score MMAs, 2880 of the S CTA's
// shared memory (MMA operands, copies in and out, P, scales) and 2800 of a softmax warp's instructions, in loops that fill the
// instruction cache: code that is seldom run is kept short or called.  At B 32, H 128, 8K the attend phase takes 97 to 101 us
// (45 at the bf16 rate), of which 12 are the
// start (queries to codes, first tile) and as many a second sequence's start; 4 x 128K 161 (89), ragged 128 x 2 tokens of
// 1 to 32K 1.2 ms a call, 1.25 to 1.31 one after another (736 us).  A move of some row's reference costs the tile a pass over O, 1 us:
// scores with a standard deviation of 3 at B 32, H 128, 8K take 210 us a call instead of 112.  A first form on CUDA cores took
// 7.3, 14.6 and 89 ms; without the scan of the tiles (TileAsks) and with a reference that only rises it took 1.95 to 2.05 us a
// tile, 1.18 ms a ragged call, and lost tails.  Looked at and left: bringing later tiles to L2 ahead of the ring (slower: 90.9 -> 93.9 us),
// all of a query's loads before the first is used (more registers and code: 91 -> 96 us), scanning from global memory (its
// requests share the path of shared memory: 108 -> 122 us a call).
//
// Every wait is bounded: on expiry the kernel records MLA_DEVERR_TIMEOUT, both CTAs of the pair abandon their loops,
// let in-flight copies and MMAs land, free TMEM and return.
#include <math_constants.h>

#include "decode8_common.cuh"

namespace mla {

namespace tc8 {

using namespace d8;

constexpr int kRows = 128;                        // query rows per CTA pair
constexpr int kChunk = kBlock8Chunk;              // [128 tokens x 128 columns] of codes: 16 KB
constexpr int kVBytes = 4 * kChunk;               // O CTA: a V stage = the four latent chunks of a tile (two copies)
constexpr int kVStages = 2;
constexpr int kUnit = kTile / 4;                  // tokens of a unit: a quarter tile
constexpr int kPBytes = kRows * 128;              // a P message: two units, [128 rows x (hi 64 tokens | lo 64 tokens)]
constexpr int kMsgBytes = kPBytes + 2 * kRows + 16;  // P | per unit and row the rescale exponent (int8) | the tile is lifted
constexpr int kMsgStride = 17408;                 // 1024-aligned
constexpr int kPSlots = 5;                        // O CTA: message slots
constexpr int kStages = 3;                        // S CTA: staging buffers
constexpr int kSoftWarps = 16;
constexpr int kSoftThreads = kSoftWarps * 32;
constexpr int kWarpProducer = 16, kWarpMma = 17, kWarpSender = 18, kWarpScale = 19;
constexpr int kThreads = 640;

// TMEM columns (512 allocated in each CTA)
constexpr uint32_t kColQ = 0;     // S CTA: latent Q codes, four to a column: hi 0..127, lo 128..255
constexpr uint32_t kColS0 = 256;  // S CTA: two 128-column score buffers
__device__ __forceinline__ uint32_t col_s(uint32_t sb) { return kColS0 + 128u * sb; }

// shared memory, S CTA.  The staging buffers also hold the Q transpose tiles, while a segment's queries are loaded.
constexpr int kSOffRing = 0;                           // two tiles
constexpr int kSOffQR = 2 * kTileBytes;                // RoPE part of Q: [128 rows x (hi 64 | lo 64)] swizzled, 16 KB
constexpr int kSOffStage = kSOffQR + kRows * 128;      // kStages staging buffers, kMsgStride apart
constexpr int kScaleBufs = 4;
constexpr int kScaleInv = 2 * kTile * 2, kScaleF = 3 * kTile * 2, kScaleFlags = kScaleF + kTile;  // within a buffer
constexpr int kScaleBytes = kScaleFlags + 16;          // a tile's token scales s, log2 s and 1 / s as bf16 (all exact), lifts; TileAsks
constexpr int kSOffScale = kSOffStage + kStages * kMsgStride;
constexpr int kSOffRef = kSOffScale + kScaleBufs * kScaleBytes;  // [4][128] reference exponents handed on
constexpr int kSOffLx = kSOffRef + 4 * kRows * 4;      // [3][3][128] a segment's two sums and R of the first three quarters
constexpr int kSOffPeak = kSOffLx + 9 * kRows * 4;     // [128] RowPeak
constexpr int kSOffLow = kSOffPeak + kRows * 8;        // [16 warps][32] LowUnit
constexpr int kNextBytes = 56;
constexpr int kSOffNext = kSOffLow + kSoftWarps * 32 * 8;  // [2] NextSeg: a segment's, the one's before
constexpr int kSOffBar = kSOffNext + 2 * kNextBytes;
constexpr int kSBarFull = 0, kSBarEmpty = 4, kSBarSFull = 8, kSBarSEmpty = 10, kSBarPEmpty = 12,
              kSBarFree = kSBarPEmpty + kPSlots, kSBarStaged = kSBarFree + kStages, kSBarRef = kSBarStaged + kStages,
              kSBarQx = kSBarRef + 16, kSBarLx = kSBarQx + 4, kSBarQFree = kSBarLx + 4, kSBarQReady = kSBarQFree + 1,
              kSBarFin = kSBarQReady + 1, kSNumBars = kSBarFin + 1;
constexpr int kSOffTail = kSOffBar + kSNumBars * 8;
// shared memory, O CTA
constexpr int kOOffV = 0;
constexpr int kOOffMsg = kVStages * kVBytes;
constexpr int kOOffBar = kOOffMsg + kPSlots * kMsgStride;
constexpr int kOBarVFull = 0, kOBarVEmpty = kVStages, kOBarPFull = 2 * kVStages, kOBarOFull = kOBarPFull + kPSlots,
              kOBarOFree = kOBarOFull + 1, kOBarRescReq = kOBarOFree + 1, kOBarRescDone = kOBarRescReq + 1,
              kOBarODrain = kOBarRescDone + 1, kOBarFin = kOBarODrain + 1, kOBarReady = kOBarFin + 1,
              kONumBars = kOBarReady + kVStages;
constexpr int kOOffTail = kOOffBar + kONumBars * 8;
constexpr int kTailBytes = 32;  // tmem base, abort flag, resc slot, [tile total, first sequence, its first tile]
constexpr int kSmemBytes = (kSOffTail > kOOffTail ? kSOffTail : kOOffTail) + kTailBytes;
static_assert(kSmemBytes <= 232448, "shared memory budget");
static_assert(kSOffQR % 1024 == 0 && kSOffStage % 1024 == 0 && kOOffMsg % 1024 == 0 && kMsgStride % 1024 == 0 &&
                  kTileBytes % 1024 == 0,
              "swizzle atoms 1024-aligned");
static_assert(kOOffBar % 8 == 0 && kSOffBar % 8 == 0 && kSOffScale % 16 == 0, "alignment");
static_assert(kMsgBytes % 16 == 0 && kSoftWarps * 32 * 64 <= kStages * kMsgStride, "bulk copy size; transpose tiles");

__device__ __forceinline__ void raise_abort(volatile int* abort_flag, uint32_t peer_abort, int32_t* dev_status) {
    *abort_flag = 1;
    st_cluster_u32(peer_abort, 1u);
    if (dev_status) atomicOr(dev_status, MLA_DEVERR_TIMEOUT);
}

// A unit is 32 tokens of a row.  The first one's largest P' goes into (1, 2]: a flat row then has 7 powers of two to rise
// before R moves (B 32, H 128, 8K: 124 us with 5 and 161 with 3, instead of 108).
using Ref = RowRef<1, 6, 6>;

// The softmax warps' next segment, looked up while they wait for the first scores and kept out of their registers.  (Each writes
// the same; a warp that has begun a segment meets others still in the one before at most.)
struct NextSeg {
    Seg s;
    SegWalk w;
};
static_assert(sizeof(NextSeg) == kNextBytes && kSOffNext % 8 == 0, "");

__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }
__device__ __forceinline__ float fmax16(const float (&v)[16]) {
    const float a = max3(v[0], v[1], v[2]), b = max3(v[3], v[4], v[5]), c = max3(v[6], v[7], v[8]);
    const float d = max3(v[9], v[10], v[11]), e = max3(v[12], v[13], v[14]);
    return fmaxf(max3(a, b, c), max3(d, e, v[15]));
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
                mbar_init(&bars[kSBarEmpty + i], 2);  // the scores' MMAs and the scan of its rows
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(&bars[kSBarSFull + i], 2);  // the scores' MMAs and the scales
                mbar_init(&bars[kSBarSEmpty + i], kSoftThreads);
            }
            for (int i = 0; i < kPSlots; ++i) mbar_init(&bars[kSBarPEmpty + i], 1);
            for (int i = 0; i < kStages; ++i) {
                mbar_init(&bars[kSBarFree + i], 1);
                mbar_init(&bars[kSBarStaged + i], kSoftThreads / 2);  // the eight warps of two units
            }
            for (int i = 0; i < 16; ++i) mbar_init(&bars[kSBarRef + i], 32);
            for (int i = 0; i < 4; ++i) {
                mbar_init(&bars[kSBarQx + i], 128);
                mbar_init(&bars[kSBarLx + i], 96);
            }
            mbar_init(&bars[kSBarQFree], 1);
            mbar_init(&bars[kSBarQReady], kSoftThreads);
            mbar_init(&bars[kSBarFin], 1);
        } else {
            for (int i = 0; i < kVStages; ++i) {
                mbar_init(&bars[kOBarVFull + i], 1);
                mbar_init(&bars[kOBarVEmpty + i], 2);  // the aggregation's MMAs and the look at its rows
                mbar_init(&bars[kOBarReady + i], 1);
            }
            // a message slot's barrier is armed here, not by the sender: a remote arrive (a release at cluster scope)
            // held the sender up for about 2000 cycles a message
            for (int i = 0; i < kPSlots; ++i) {
                mbar_init(&bars[kOBarPFull + i], 1);
                mbar_arrive_expect_tx(&bars[kOBarPFull + i], kMsgBytes);
            }
            mbar_init(&bars[kOBarOFull], 1);
            mbar_init(&bars[kOBarOFree], kSoftThreads);
            mbar_init(&bars[kOBarRescReq], 1);
            mbar_init(&bars[kOBarRescDone], kSoftThreads);
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
                    bool ready = false;  // the tile and its score buffer were seen to be there while the last one's MMAs went out
                    for (int t = s.t0; ok && t < s.t1; ++t, ++n) {
                        const uint32_t sb = n & 1u, us = n >> 1;
                        if (!ready)
                            ok = mbar_wait(&bars[kSBarSEmpty + sb], (us & 1u) ^ 1u, abort_flag, kLimitNs) &&
                                 mbar_wait(&bars[kSBarFull + 2 * sb], us & 1u, abort_flag, kLimitNs);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t d = tmem + col_s(sb);
                        const uint64_t tile_off = static_cast<uint64_t>(sb * kTileBytes) >> 4;
                        bool next = false;
                        // rolled: code that fits the instruction cache beside the softmax warps' (fully unrolled, the issue of
                        // a tile's 36 MMAs took longer than their 2304 cycles)
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            if (c == 2 && !ready) {
                                ok = mbar_wait(&bars[kSBarFull + 2 * sb + 1], us & 1u, abort_flag, kLimitNs);
                                if (!ok) break;
                                tc_fence_after();
                            }
                            // asked for while MMAs are still queued, so that the next tile's follow at once
                            if (c == 3 && t + 1 < s.t1) {
                                const uint32_t un = (n + 1) >> 1;
                                next = mbar_poll(smem_u32(&bars[kSBarSEmpty + (sb ^ 1u)]), (un & 1u) ^ 1u) &&
                                       mbar_poll(smem_u32(&bars[kSBarFull + 2 * (sb ^ 1u)]), un & 1u) &&
                                       mbar_poll(smem_u32(&bars[kSBarFull + 2 * (sb ^ 1u) + 1]), un & 1u);
                            }
                            const uint64_t cd = ring_desc + tile_off + (static_cast<uint64_t>(c * kChunk) >> 4);
                            const uint32_t qa = tmem + kColQ + 32 * c;
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk) {
                                mma8_ts(d, qa + 8 * kk, cd + 2 * kk, idesc, (c | kk) ? 1u : 0u);
                                mma8_ts(d, qa + 128 + 8 * kk, cd + 2 * kk, idesc, 1u);
                            }
                            if (c == 1) mma_commit(smem_u32(&bars[kSBarEmpty + 2 * sb]));
                        }
                        if (!ok) break;
                        const uint64_t rd = rope_desc + tile_off;
#pragma unroll
                        for (int kk = 0; kk < 2; ++kk) {
                            mma8_ss(d, qr_desc + 2 * kk, rd + 2 * kk, idesc, 1u);
                            mma8_ss(d, qr_desc + 4 + 2 * kk, rd + 2 * kk, idesc, 1u);
                        }
                        mma_commit(smem_u32(&bars[kSBarSFull + sb]));
                        mma_commit(smem_u32(&bars[kSBarEmpty + 2 * sb + 1]));
                        ready = next;
                    }
                }
                if (!ok) raise_abort(abort_flag, peer_abort, p.dev_status);
                mma_commit(smem_u32(&bars[kSBarFin]));
                mbar_wait(&bars[kSBarFin], 0, &never, kLimitNs);
            }
            __syncwarp();
        } else if (warp < kSoftWarps) {
            // ---- softmax: warp (qd, cq) owns TMEM lanes 32 qd.. (query rows) and the tokens 32 cq .. 32 cq + 31 of every
            //      tile: a unit.  The units of a row follow one another only in the reference exponent, which a warp hands
            //      on as soon as it knows its maximum; its exponentials and its part of the P message then overlap the
            //      other warps', so nothing holds the sixteen warps in step (a barrier a tile left them waiting on one
            //      another and on latencies half the time).
            const int qd = warp & 3, cq = warp >> 2;
            const int r = 32 * qd + lane;
            const uint32_t t_lane = tmem + (static_cast<uint32_t>(32 * qd) << 16);
            const int rr = g * kRows + r;
            const bool row_ok = rr < p.R;
            const int gA = g * kRows + 32 * qd + (lane & 15), gB = gA + 16;
            const int cb = 32 * cq + 16 * (lane >> 4);  // this thread's first score column
            volatile float* ref_in = reinterpret_cast<volatile float*>(smem + kSOffRef) + ((cq + 3) & 3) * kRows + 32 * qd;
            volatile float* ref_out = reinterpret_cast<volatile float*>(smem + kSOffRef) + cq * kRows + 32 * qd;
            volatile float* lx = reinterpret_cast<volatile float*>(smem + kSOffLx) + 32 * qd + lane;
            uint64_t* bar_in = &bars[kSBarRef + 4 * ((cq + 3) & 3) + qd];
            uint64_t* bar_out = &bars[kSBarRef + 4 * cq + qd];
            SegWalk w = walk;
            Seg s;
            uint32_t n = 0, kseg = 0, nref = 0;  // tiles, segments, references received
            // a row's state where its reference moves; both in shared memory, since moves are rare and registers are not
            LowUnit& low = reinterpret_cast<LowUnit*>(smem + kSOffLow)[32 * warp + lane];
            RowPeak& peak = reinterpret_cast<RowPeak*>(smem + kSOffPeak)[r];
            low.at = kNoTile;
            uint32_t stg = cq >> 1, stg_phase = 1;  // the staging buffer of message 2 n + cq / 2, and the phase it is free in
            bool ok = true;
            bool have = w.next(p, s);
            while (ok && have) {
                // this segment's query rows, two e4m3 terms each: latent columns 128 cq .. -> TMEM, RoPE columns 16 cq ..
                // -> shared memory.  The warp loads its 32 rows coalesced (a lane per 16-byte unit) and transposes each
                // 32-column chunk through a swizzled 2 KB tile into the lane-per-row order of tcgen05.st.  The bf16 rows
                // wait in the score buffers (free between segments) until the row's largest magnitude is known.
                float rowf;
                {
                    const uint16_t* qb = p.q + (static_cast<int64_t>(s.b) * p.R + g * kRows + 32 * qd) * kRow;
                    const int rows_here = p.R - g * kRows - 32 * qd;  // rows of this quadrant (may be <= 0)
                    uint8_t* qt = smem + kSOffStage + warp * (32 * 64);
                    const int lu = lane & 3, lr = lane >> 2;  // unit and row-in-eight of this lane's loads
                    const uint32_t raw = t_lane + kColS0 + 64 * cq;
                    uint32_t m2 = 0;
                    uint4 y[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int ri = 16 * i + (lane >> 1);
                        y[i] = make_uint4(0, 0, 0, 0);
                        if (ri < rows_here) y[i] = reinterpret_cast<const uint4*>(qb + ri * kRow)[64 + 2 * cq + (lane & 1)];
                    }
#pragma unroll 1
                    for (int c = 0; c < 4; c += 2) {
                        uint4 x[2][4];
#pragma unroll
                        for (int jj = 0; jj < 2; ++jj)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int ri = 8 * i + lr;
                                x[jj][i] = make_uint4(0, 0, 0, 0);
                                if (ri < rows_here)
                                    x[jj][i] = reinterpret_cast<const uint4*>(qb + ri * kRow)[16 * cq + 4 * (c + jj) + lu];
                            }
                        // the transpose tiles are the staging buffers: before the first write to them, wait until the
                        // sender has seen every copy of earlier messages read out (and, with it, the other warps)
                        if (c == 0 && kseg > 0) ok = mbar_wait(&bars[kSBarQFree], (kseg - 1) & 1u, abort_flag, kLimitNs);
#pragma unroll
                        for (int jj = 0; jj < 2; ++jj) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int ri = 8 * i + lr;
                                *reinterpret_cast<uint4*>(qt + ri * 64 + ((lu ^ ((ri >> 1) & 3)) << 4)) = x[jj][i];
                            }
                            __syncwarp();
                            uint32_t v[32];
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                const uint4 z = *reinterpret_cast<const uint4*>(qt + lane * 64 + ((u ^ ((lane >> 1) & 3)) << 4));
                                v[4 * u] = z.x; v[4 * u + 1] = z.y; v[4 * u + 2] = z.z; v[4 * u + 3] = z.w;
                                m2 = max_abs2(max_abs2(max_abs2(max_abs2(m2, z.x), z.y), z.z), z.w);
                            }
                            __syncwarp();
                            tmem_st16(raw + 16 * (c + jj), v);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int ri = 16 * i + (lane >> 1);
                        *reinterpret_cast<uint4*>(qt + ri * 64 + (((lane & 1) ^ ((ri >> 1) & 3)) << 4)) = y[i];
                    }
                    __syncwarp();
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        y[u] = *reinterpret_cast<const uint4*>(qt + lane * 64 + ((u ^ ((lane >> 1) & 3)) << 4));
                        m2 = max_abs2(max_abs2(max_abs2(max_abs2(m2, y[u].x), y[u].y), y[u].z), y[u].w);
                    }
                    // the row's largest magnitude, over the four quarters of its columns
                    ref_out[lane] = __uint_as_float(max(m2 & 0xFFFFu, m2 >> 16));
                    mbar_arrive(&bars[kSBarQx + qd]);
                    ok = mbar_wait(&bars[kSBarQx + qd], kseg & 1u, abort_flag, kLimitNs) && ok;
                    uint32_t top = 0;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        top = max(top, reinterpret_cast<volatile uint32_t*>(smem + kSOffRef)[k * kRows + r]);
                    const int a = top < 0x7F80u ? row_exp(top) : 0;
                    const float inv = exp2_int(-a);
                    // an infinity or NaN in the query: every score of the row is NaN
                    rowf = top < 0x7F80u ? exp2_int(a) * p.scale_log2 : CUDART_NAN_F;
                    uint8_t* qr = smem + kSOffQR + r * 128;
                    {
                        uint4 hi, lo;
                        split4_q(y[0].x, y[0].y, inv, hi.x, lo.x);
                        split4_q(y[0].z, y[0].w, inv, hi.y, lo.y);
                        split4_q(y[1].x, y[1].y, inv, hi.z, lo.z);
                        split4_q(y[1].z, y[1].w, inv, hi.w, lo.w);
                        *reinterpret_cast<uint4*>(qr + ((cq ^ (r & 7)) << 4)) = hi;
                        *reinterpret_cast<uint4*>(qr + (((4 + cq) ^ (r & 7)) << 4)) = lo;
                    }
                    __syncwarp();
                    tmem_wait_st();
#pragma unroll 1
                    for (int c = 0; c < 2; ++c) {
                        uint32_t v[32], hi[32], lo[32];
                        tmem_ld32(raw + 32 * c, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int u = 0; u < 16; ++u) split4_q(v[2 * u], v[2 * u + 1], inv, hi[u], lo[u]);
                        tmem_st16(t_lane + kColQ + 32 * cq + 16 * c, hi);
                        tmem_st16(t_lane + kColQ + 128 + 32 * cq + 16 * c, lo);
                    }
                }
                fence_proxy_async_cta();
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&bars[kSBarQReady]);
                // the next segment, whose queries are prefetched near the end of this one
                {
                    NextSeg next{s, w};
                    have = next.w.next(p, next.s);
                    __syncwarp();
                    if (lane == 0) *reinterpret_cast<NextSeg*>(smem + kSOffNext + (kseg & 1u) * kNextBytes) = next;
                    __syncwarp();
                }
                const NextSeg* nx = reinterpret_cast<const NextSeg*>(smem + kSOffNext + (kseg & 1u) * kNextBytes);
                const int t_pf = have && row_ok ? max(s.t0, s.t1 - 2) : -1;
                // from here on a thread has rows rA = 32 qd + lane % 16 and rB = rA + 16, and 16 of the warp's columns: the
                // tokens' scales are then read and unpacked once for two rows
                const float rowfA = __shfl_sync(0xffffffffu, rowf, lane & 15), rowfB = __shfl_sync(0xffffffffu, rowf, 16 + (lane & 15));
                const float2 fA = make_float2(rowfA, rowfA), fB = make_float2(rowfB, rowfB);
                float RA = kNoRef, RB = kNoRef, R = kNoRef;  // the references of rows rA, rB and 32 qd + lane
                float lA = 0.f, lB = 0.f, tA = 0.f, tB = 0.f;
                const int limA = gA < p.R ? s.L - p.n_q + gA / p.H + 1 : s.L;  // keys 0 .. lim-1 are visible
                const int limB = gB < p.R ? s.L - p.n_q + gB / p.H + 1 : s.L;  // (rows of no query: zeros, not stored)
                for (int t = s.t0; t < s.t1; ++t, ++n) {
                    const uint32_t sb = n & 1u, us = n >> 1;
                    if (t == t_pf)
                        for (int c = cq; c < 9; c += 4)
                            prefetch_l2(reinterpret_cast<const char*>(p.q + (static_cast<int64_t>(nx->s.b) * p.R + rr) * kRow) + 128 * c);
                    const uint4* sw4 = reinterpret_cast<const uint4*>(smem + kSOffScale + (n % kScaleBufs) * kScaleBytes) + cb / 8;
                    ok = mbar_wait(&bars[kSBarSFull + sb], us & 1u, abort_flag, kLimitNs) && ok;
                    __syncwarp();
                    tc_fence_after();
                    const TileAsks* ask =
                        reinterpret_cast<const TileAsks*>(smem + kSOffScale + (n % kScaleBufs) * kScaleBytes + kScaleFlags);
                    int d = 0;  // the exponent of the row's rescale
                    uint32_t hiA[4], loA[4], hiB[4], loB[4];
                    float yA[16], yB[16];
                    {
                        uint32_t a[16], b[16];
                        tmem_ld16_halves(t_lane + col_s(sb) + 32 * cq, a);
                        tmem_ld16_halves(t_lane + (16u << 16) + col_s(sb) + 32 * cq, b);
                        tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            yA[k] = __uint_as_float(a[k]);
                            yB[k] = __uint_as_float(b[k]);
                        }
                    }
                    tc_fence_before();
                    mbar_arrive(&bars[kSBarSEmpty + sb]);
                    // y = log2(p s_t), before the reference: S s_t (2^a scale log2 e) + log2 s_t
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint4 sw = sw4[k], ew = sw4[k + kTile / 8];
                        const uint32_t ss[4] = {sw.x, sw.y, sw.z, sw.w}, ee[4] = {ew.x, ew.y, ew.z, ew.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int c = 8 * k + 2 * i;
                            const float2 s2 = bf16x2_f32(ss[i]), e2f = bf16x2_f32(ee[i]);
                            const float2 a2 = fma2(mul2(make_float2(yA[c], yA[c + 1]), s2), fA, e2f);
                            const float2 b2 = fma2(mul2(make_float2(yB[c], yB[c + 1]), s2), fB, e2f);
                            yA[c] = a2.x;
                            yA[c + 1] = a2.y;
                            yB[c] = b2.x;
                            yB[c + 1] = b2.y;
                        }
                    }
                    const int vA = limA - t * kTile - cb, vB = limB - t * kTile - cb;  // columns < v are visible
                    if (vA < 16 || vB < 16) {
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            yA[k] = k < vA ? yA[k] : -CUDART_INF_F;
                            yB[k] = k < vB ? yB[k] : -CUDART_INF_F;
                        }
                    }
                    float mA = fmax16(yA), mB = fmax16(yB);
                    mA = fmaxf(mA, __shfl_xor_sync(0xffffffffu, mA, 16));
                    mB = fmaxf(mB, __shfl_xor_sync(0xffffffffu, mB, 16));
                    // the reference: the previous unit's (another warp's), moved if this unit needs it, handed on
                    if (cq > 0 || t > s.t0) {
                        ok = mbar_wait(bar_in, nref & 1u, abort_flag, kLimitNs) && ok;
                        ++nref;
                        RA = ref_in[lane & 15];
                        RB = ref_in[16 + (lane & 15)];
                    }
                    const float top = lane < 16 ? mA : mB;
                    float last = R;  // this warp's last unit's: the sums are relative to it
                    R = lane < 16 ? RA : RB;
                    if (t == s.t0) {  // (nothing in the sums yet)
                        if (cq == 0) {
                            R = Ref::first(top, peak);
                            RA = __shfl_sync(0xffffffffu, R, lane & 15);
                            RB = __shfl_sync(0xffffffffu, R, 16 + (lane & 15));
                        }
                        last = R;
                    }
                    if (!__all_sync(0xffffffffu, Ref::stays(top, R))) {
                        const float was = R;
                        R = Ref::moved(top, R, R == last, n, ask->eager != 0, low, peak);
                        d = ref_exp(was, R);
                        RA = __shfl_sync(0xffffffffu, R, lane & 15);
                        RB = __shfl_sync(0xffffffffu, R, 16 + (lane & 15));
                    }
                    if (cq < 3 || t + 1 < s.t1) {
                        ref_out[lane] = R;
                        mbar_arrive(bar_out);
                    }
                    const float2 nA = make_float2(-RA, -RA), nB = make_float2(-RB, -RB);
                    const uint32_t dm = dither_mask(cb >> 4, t);
                    float2 sA = make_float2(0.f, 0.f), sB = sA, rA = sA, rB = sA;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        // 1 / s, as bf16 (of lifted tokens, 2^m / s)
                        const uint4 sw = sw4[k + kScaleInv / 16];
                        const uint32_t sb4[4] = {sw.x, sw.y, sw.z, sw.w};
#pragma unroll
                        for (int i = 0; i < 4; i += 2) {
                            const int c = 8 * k + 2 * i, o = c / 4;
                            const float2 i0 = bf16x2_f32(sb4[i]), i1 = bf16x2_f32(sb4[i + 1]);
                            float2 a0 = add2(make_float2(yA[c], yA[c + 1]), nA), a1 = add2(make_float2(yA[c + 2], yA[c + 3]), nA);
                            a0 = make_float2(ex2_approx(a0.x), ex2_approx(a0.y));
                            a1 = make_float2(ex2_approx(a1.x), ex2_approx(a1.y));
                            sA = fma2(a0, i0, sA);
                            sA = fma2(a1, i1, sA);
                            // as the MMAs will have it (8 significant bits): O is divided by the sum of what it sums
                            a0 = bf16x2_f32(cvt_bf16x2(a0.x, a0.y));
                            a1 = bf16x2_f32(cvt_bf16x2(a1.x, a1.y));
                            rA = fma2(a0, i0, rA);
                            rA = fma2(a1, i1, rA);
                            split4_p(a0.x, a0.y, a1.x, a1.y, dither_pair(c / 2) + dm, dither_pair(c / 2 + 1) + dm, hiA[o], loA[o]);
                            float2 b0 = add2(make_float2(yB[c], yB[c + 1]), nB), b1 = add2(make_float2(yB[c + 2], yB[c + 3]), nB);
                            b0 = make_float2(ex2_approx(b0.x), ex2_approx(b0.y));
                            b1 = make_float2(ex2_approx(b1.x), ex2_approx(b1.y));
                            sB = fma2(b0, i0, sB);
                            sB = fma2(b1, i1, sB);
                            b0 = bf16x2_f32(cvt_bf16x2(b0.x, b0.y));
                            b1 = bf16x2_f32(cvt_bf16x2(b1.x, b1.y));
                            rB = fma2(b0, i0, rB);
                            rB = fma2(b1, i1, rB);
                            split4_p(b0.x, b0.y, b1.x, b1.y, dither_pair(c / 2) + dm, dither_pair(c / 2 + 1) + dm, hiB[o], loB[o]);
                        }
                    }
                    if (__any_sync(0xffffffffu, R != last)) {
                        const float step = ref_step(last, R);
                        const float a = __shfl_sync(0xffffffffu, step, lane & 15);
                        const float b = __shfl_sync(0xffffffffu, step, 16 + (lane & 15));
                        lA *= a;
                        tA *= a;
                        lB *= b;
                        tB *= b;
                    }
                    lA += sA.x + sA.y;
                    lB += sB.x + sB.y;
                    tA += rA.x + rA.y;
                    tB += rB.x + rB.y;
                    ok = mbar_wait(&bars[kSBarFree + stg], stg_phase, abort_flag, kLimitNs) && ok;
                    // a row's 16 columns: the 16-byte unit (cb / 16) % 4 of its hi part and of its lo part
                    uint8_t* stage = smem + kSOffStage + stg * kMsgStride;
                    uint8_t* at = stage + (32 * qd + (lane & 15)) * 128;
                    uint8_t* ah = at + ((((cb >> 4) & 3) ^ (lane & 7)) << 4);
                    uint8_t* al = at + (((4 + ((cb >> 4) & 3)) ^ (lane & 7)) << 4);
                    *reinterpret_cast<uint4*>(ah) = make_uint4(hiA[0], hiA[1], hiA[2], hiA[3]);
                    *reinterpret_cast<uint4*>(ah + 2048) = make_uint4(hiB[0], hiB[1], hiB[2], hiB[3]);
                    *reinterpret_cast<uint4*>(al) = make_uint4(loA[0], loA[1], loA[2], loA[3]);
                    *reinterpret_cast<uint4*>(al + 2048) = make_uint4(loB[0], loB[1], loB[2], loB[3]);
                    reinterpret_cast<int8_t*>(stage + kPBytes)[(cq & 1) * kRows + r] = static_cast<int8_t>(d);
                    if ((warp & 7) == 0 && lane == 0) *reinterpret_cast<uint32_t*>(stage + kPBytes + 2 * kRows) = ask->lift;
                    fence_proxy_async_cta();
                    mbar_arrive(&bars[kSBarStaged + stg]);
                    stg += 2;
                    if (stg >= kStages) {
                        stg -= kStages;
                        stg_phase ^= 1u;
                    }
                    if (!__all_sync(0xffffffffu, ok)) {
                        ok = false;
                        break;
                    }
                }
                if (!ok) break;
                // segment result: R and the two sums over the row's eight column parts; a NaN sum keeps its piece
                lA += __shfl_xor_sync(0xffffffffu, lA, 16);
                lB += __shfl_xor_sync(0xffffffffu, lB, 16);
                tA += __shfl_xor_sync(0xffffffffu, tA, 16);
                tB += __shfl_xor_sync(0xffffffffu, tB, 16);
                float lt = lane < 16 ? lA : lB;
                float tt = lane < 16 ? tA : tB;
                const float rmine = R;
                if (cq < 3) {
                    lx[3 * cq * kRows] = lt;
                    lx[(3 * cq + 1) * kRows] = tt;
                    lx[(3 * cq + 2) * kRows] = rmine;
                    mbar_arrive(&bars[kSBarLx + qd]);
                } else {
                    ok = mbar_wait(&bars[kSBarLx + qd], kseg & 1u, abort_flag, kLimitNs);
                    ok = __all_sync(0xffffffffu, ok);
#pragma unroll
                    for (int k = 0; k < 3; ++k) {
                        const float f = ref_step(lx[(3 * k + 2) * kRows], rmine);
                        lt = fmaf(lx[3 * k * kRows], f, lt);
                        tt = fmaf(lx[(3 * k + 1) * kRows], f, tt);
                    }
                    if (row_ok && ok)
                        p.ml_part[out_row_base + static_cast<int64_t>(s.slot) * kRows + r] =
                            make_float4(lt != lt ? 0.f : rmine, lt, tt, 0.f);
                }
                ++kseg;
                w = nx->w;
                s = nx->s;
            }
            if (!ok) raise_abort(abort_flag, peer_abort, p.dev_status);
        } else if (warp == kWarpScale) {
            // ---- scales: the 128 tokens' s = 2^k and k of each tile, ahead of the softmax, and what the tile asks of the
            //      references (TileAsks).  The buffer of tile n was tile n - 4's; a softmax warp that has read the scores of
            //      tile n - 2 is past tile n - 3.
            SegWalk w = walk;
            Seg s;
            uint32_t n = 0;
            bool ok = true;
            TileScan scan;
            uint32_t next[4];
            while (ok && w.next(p, s)) {
                auto entry = [&](int t) { return t < s.t1 ? s.tab[t] : 0; };
                auto load = [&](int t, int32_t e) {  // (a block's scales are there, whether of tokens or not)
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (t < s.t1) x = reinterpret_cast<const uint4*>(block_of(p, e, false) + kBlock8Scales)[lane];
                    next[0] = x.x; next[1] = x.y; next[2] = x.z; next[3] = x.w;
                };
                // the scales are asked for a tile ahead, the table entry two
                load(s.t0, entry(s.t0));
                int32_t e1 = entry(s.t0 + 1);
                scan.reset();
                for (int t = s.t0; ok && t < s.t1; ++t, ++n) {
                    uint32_t bits[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) bits[i] = next[i];
                    if (s.L - t * kTile < kTile) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) bits[i] = t * kTile + 4 * lane + i < s.L ? bits[i] : kNoScale;
                    }
                    load(t + 1, e1);
                    e1 = entry(t + 2);
                    const uint32_t sb = n & 1u, us = n >> 1;
                    ok = mbar_wait(&bars[kSBarFull + 2 * sb], us & 1u, abort_flag, kLimitNs) &&
                         mbar_wait(&bars[kSBarFull + 2 * sb + 1], us & 1u, abort_flag, kLimitNs);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    // (the buffer of lifts is free already: SEmpty of the tile before this one has been seen)
                    uint8_t* buf = smem + kSOffScale + (n % kScaleBufs) * kScaleBytes;
                    const TileAsks ask = scan.tile(smem + kSOffRing + sb * kTileBytes, min(kTile, s.L - t * kTile), bits, lane,
                                                    buf + kScaleF);
                    if (lane < 2) mbar_arrive(&bars[kSBarEmpty + 2 * sb + lane]);
                    ok = mbar_wait(&bars[kSBarSEmpty + sb], (us & 1u) ^ 1u, abort_flag, kLimitNs);
                    uint32_t e[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) e[i] = __float_as_uint(static_cast<float>(static_cast<int>(bits[i] >> 23) - 127));
                    uint8_t* to = buf + 8 * lane;
                    const uint2 sc = make_uint2(__byte_perm(bits[0], bits[1], 0x7632), __byte_perm(bits[2], bits[3], 0x7632));
                    uint2 is = make_uint2(0x7F007F00u - sc.x, 0x7F007F00u - sc.y);
                    if (ask.lift) {
                        const uint32_t f = *reinterpret_cast<const uint32_t*>(buf + kScaleF + 4 * lane);
                        uint32_t up[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t m = f >> (8 * i) & 0xFFu;
                            e[i] = __float_as_uint(__uint_as_float(e[i]) - static_cast<float>(m));
                            up[i] = m << 7;
                        }
                        is.x += up[0] | (up[1] << 16);
                        is.y += up[2] | (up[3] << 16);
                    }
                    *reinterpret_cast<uint2*>(to) = sc;
                    *reinterpret_cast<uint2*>(to + 2 * kTile) =
                        make_uint2(__byte_perm(e[0], e[1], 0x7632), __byte_perm(e[2], e[3], 0x7632));
                    *reinterpret_cast<uint2*>(to + kScaleInv) = is;
                    if (lane == 0) *reinterpret_cast<TileAsks*>(to + kScaleFlags) = ask;
                    ok = __all_sync(0xffffffffu, ok);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars[kSBarSFull + sb]);
                }
            }
            if (!ok && lane == 0) raise_abort(abort_flag, peer_abort, p.dev_status);
        } else if (warp == kWarpSender) {
            // ---- sender: ships each staged P message (one bulk copy, completing on the O CTA's barrier) once the O CTA
            //      has released that message slot
            const uint32_t peer_msg = mapa(sbase + kOOffMsg, peer);
            const uint32_t peer_pfull = mapa(sbase + kOOffBar + kOBarPFull * 8, peer);
            if (lane == 0) {
                SegWalk w = walk;
                Seg s;
                uint32_t u = 0;  // units
                bool ok = true;
                while (ok && w.next(p, s)) {
                    const uint32_t first_u = u;
                    for (int t = 2 * s.t0; t < 2 * s.t1; ++t, ++u) {
                        const uint32_t stg = u % kStages, pb = u % kPSlots;
                        ok = mbar_wait(&bars[kSBarStaged + stg], (u / kStages) & 1u, abort_flag, kLimitNs) &&
                             mbar_wait<true>(&bars[kSBarPEmpty + pb], ((u / kPSlots) & 1u) ^ 1u, abort_flag, kLimitNs);
                        if (!ok) break;
                        bulk_copy_to_peer(peer_msg + pb * kMsgStride, sbase + kSOffStage + stg * kMsgStride, kMsgBytes,
                                          peer_pfull + 8 * pb);
                        bulk_commit_group();
                        if (u > first_u) {
                            bulk_wait_group_read<1>();  // the copy before this one has read its source
                            mbar_arrive(&bars[kSBarFree + (u - 1) % kStages]);
                        }
                    }
                    // every staged message read out before the Q reload reuses the staging buffers
                    bulk_wait_group_read<0>();
                    if (ok) {
                        mbar_arrive(&bars[kSBarFree + (u - 1) % kStages]);
                        mbar_arrive(&bars[kSBarQFree]);
                    }
                }
                if (!ok) raise_abort(abort_flag, peer_abort, p.dev_status);
                // the O CTA's last releases of its message slots arrive here: they have to land before this CTA ends
                for (uint32_t i = (u > kPSlots ? u - kPSlots : 0); ok && i < u; ++i)
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
                uint32_t n = 0;  // tiles
                bool ok = true;
                const uint64_t last_use = l2_policy_evict_first();
                while (ok && w.next(p, s)) {
                    for (int t = s.t0; ok && t < s.t1; ++t, ++n) {
                        const uint8_t* src = block_of(p, s.tab[t], true);
                        const uint32_t st = n % kVStages, u = n / kVStages;
                        ok = mbar_wait(&bars[kOBarVEmpty + st], (u & 1u) ^ 1u, abort_flag, kLimitNs);
                        if (!ok) break;
                        mbar_arrive_expect_tx(&bars[kOBarVFull + st], kVBytes);
                        for (int k = 0; k < 2; ++k)
                            bulk_load_hint(sbase + kOOffV + st * kVBytes + k * (kVBytes / 2), src + k * (kVBytes / 2),
                                           kVBytes / 2, &bars[kOBarVFull + st], last_use);
                    }
                }
                if (!ok) raise_abort(abort_flag, peer_abort, p.dev_status);
                for (uint32_t i = (n > kVStages ? n - kVStages : 0); i < n; ++i)
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
            uint32_t n = 0, kseg = 0, nresc = 0, nready = 0;  // (nready: bit st, the phase of kOBarReady + st)
            bool ok = true;
            while (ok && w.next(p, s)) {
                for (int t = s.t0; ok && t < s.t1; ++t, ++n) {
                    const uint32_t st = n % kVStages;
                    const int nvalid = min(kTile, s.L - t * kTile);
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t u = 2 * n + h, pb = u % kPSlots;
                        if (leader) {
                            ok = mbar_wait<true>(&bars[kOBarPFull + pb], (u / kPSlots) & 1u, abort_flag, kLimitNs);
                            if (ok) mbar_arrive_expect_tx(&bars[kOBarPFull + pb], kMsgBytes);  // for its next message
                            if (ok && t == s.t0 && h == 0)
                                ok = mbar_wait(&bars[kOBarOFree], (kseg & 1u) ^ 1u, abort_flag, kLimitNs);
                            if (ok && h == 0) {
                                ok = mbar_wait(&bars[kOBarVFull + st], (n / kVStages) & 1u, abort_flag, kLimitNs);
                                // tokens are lifted (the S CTA's scan has found them in the same codes), or not seen by every query
                                if (*reinterpret_cast<const uint32_t*>(smem + kOOffMsg + pb * kMsgStride + kPBytes + 2 * kRows) != 0 ||
                                    s.L - p.n_q + 1 - t * kTile < nvalid) {
                                    ok = ok && mbar_wait(&bars[kOBarReady + st], nready >> st & 1u, abort_flag, kLimitNs);
                                    nready ^= 1u << st;
                                }
                            }
                        }
                        ok = __any_sync(0xffffffffu, ok && leader);
                        if (!ok) break;
                        // (read by every lane: which of the two units move some row's reference)
                        const uint32_t* moved = reinterpret_cast<const uint32_t*>(smem + kOOffMsg + pb * kMsgStride + kPBytes);
                        const uint32_t moved0 = moved[lane], moved1 = moved[32 + lane];
                        const bool resc0 = __any_sync(0xffffffffu, moved0 != 0);
                        const bool resc1 = __any_sync(0xffffffffu, moved1 != 0);
                        if (h == 0 && nvalid < kTile) {
                            // rows past the sequence end: P is 0 there, make V 0 too (no 0 * NaN)
                            const int nz = (kTile - nvalid) * 8;  // 16-byte units per chunk
                            for (int i = lane; i < 4 * nz; i += 32) {
                                const int c = i / nz, q = i % nz;
                                *reinterpret_cast<uint4*>(smem + kOOffV + st * kVBytes + c * kChunk + nvalid * 128 + q * 16) =
                                    make_uint4(0, 0, 0, 0);
                            }
                            fence_proxy_async_cta();
                        }
#pragma unroll 1
                        for (int kk = 0; kk < 2; ++kk) {
                            const bool fresh = (t == s.t0 && h == 0 && kk == 0);
                            if (!fresh && (kk ? resc1 : resc0)) {
                                // have the epilogue rescale O once all earlier MMAs are done
                                if (leader) {
                                    *resc_pb = static_cast<int>(pb * kMsgStride + kk * kRows);
                                    mma_commit(smem_u32(&bars[kOBarODrain]));
                                    mbar_arrive(&bars[kOBarRescReq]);
                                    ok = mbar_wait(&bars[kOBarRescDone], nresc & 1u, abort_flag, kLimitNs);
                                }
                                ++nresc;
                                ok = __any_sync(0xffffffffu, ok && leader);
                                if (!ok) break;
                            }
                            if (elect_one()) {
                                tc_fence_after();
                                const uint64_t v = v_desc + (static_cast<uint64_t>(st * kVBytes + (2 * h + kk) * (kUnit * 128)) >> 4);
                                const uint64_t pd = p_desc + (static_cast<uint64_t>(pb * kMsgStride + kk * 32) >> 4);
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    mma8_ss(tmem + 256 * k, pd, v + ((k * 2 * kChunk) >> 4), idesc_hi, fresh ? 0u : 1u);
                                    mma8_ss(tmem + 256 * k, pd + 4, v + ((k * 2 * kChunk) >> 4), idesc_lo, 1u);
                                }
                            }
                            __syncwarp();
                        }
                        if (!ok) break;
                        if (leader) {
                            mma_commit(peer_pempty + 8 * pb);
                            if (h == 1) mma_commit(smem_u32(&bars[kOBarVEmpty + st]));
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
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
        } else if (warp == kWarpScale) {
            // ---- what V's rows need before they are multiplied: small tokens lifted, NaN in rows that not every query sees made
            //      0 (P = 0 times NaN).  The MMA warp waits for it where there is such a row; a stage stays until it has been
            //      looked at.
            SegWalk w = walk;
            Seg s;
            uint32_t n = 0;
            bool ok = true;
            while (ok && w.next(p, s)) {
                for (int t = s.t0; ok && t < s.t1; ++t, ++n) {
                    const uint32_t st = n % kVStages;
                    ok = mbar_wait(&bars[kOBarVFull + st], (n / kVStages) & 1u, abort_flag, kLimitNs);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    uint8_t* v = smem + kOOffV + st * kVBytes;
                    const int nvalid = min(kTile, s.L - t * kTile), some = max(0, s.L - p.n_q + 1 - t * kTile);
                    const uint32_t small = small_tokens(v, nvalid, lane);
                    bool touched = false;
                    if (__any_sync(0xffffffffu, small != 0)) touched = lift_tile(v, nvalid, small, lane);
                    if (some < nvalid) {
                        nan_to_zero_rows(v, some, nvalid, lane);
                        touched = true;
                    }
                    if (touched) fence_proxy_async_cta();
                    __syncwarp();
                    if (lane == 0) {
                        if (touched) mbar_arrive(&bars[kOBarReady + st]);
                        mbar_arrive(&bars[kOBarVEmpty + st]);
                    }
                }
            }
            if (!ok && lane == 0) raise_abort(abort_flag, peer_abort, p.dev_status);
        } else if (warp < kSoftWarps) {
            // ---- epilogue: warp (qd, cq), one thread per query row and 128 columns
            const int r = 32 * (warp & 3) + lane, cq = warp >> 2;
            const uint32_t t_lane = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + 128 * cq;
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
                            reinterpret_cast<const int8_t*>(smem + kOOffMsg + kPBytes + *resc_pb)[r];
                        if (__any_sync(0xffffffffu, d != 0)) {
                            const float a = ref_factor(d);
#pragma unroll 1
                            for (int c = 0; c < 4; ++c) {
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
                // the workspace holds [column / 32][row] x 32 fp32.  A thread has its row's 32 columns; four lanes exchange 8
                // by 8 of them, so that they store a row's 128 bytes together
                float* oseg = p.o_part + (out_row_base + static_cast<int64_t>(s.slot) * kRows) * kDc + (r & ~3) * 32 + 8 * (lane & 3);
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    uint32_t v[32];
                    tmem_ld32(t_lane + 32 * c, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int bit = 1; bit <= 2; bit *= 2)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (!(k & bit))
#pragma unroll
                                for (int e = 0; e < 8; ++e) {
                                    uint32_t &x = v[8 * k + e], &y = v[8 * (k | bit) + e];
                                    const uint32_t got = __shfl_xor_sync(0xffffffffu, (lane & bit) ? x : y, bit);
                                    if (lane & bit) x = got;
                                    else y = got;
                                }
                    // now v[8 k ..] is row (r & ~3) + k's, columns 8 (lane & 3) .. of the 32
#pragma unroll
                    for (int k = 0; k < 4; ++k) st_global8(oseg + ((4 * cq + c) * kRows + k) * 32, v + 8 * k);
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
                              float* o_part, float4* ml_part, int slots, int32_t* dev_status, cudaStream_t stream) {
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
