// Absorbed MLA decode over the 8-bit cache for few query rows (few heads): one SM per work unit.
//
// The attend phase of mla_decode8, with both contractions transposed, the 128 tokens of a block as the M side:
//   S^T[token, row] = K . [Q_hi | Q_lo]^T   M = 128 tokens (A: the block's codes as they lie), N = 2 NR: 18 MMAs
//   O^T[latent, row] += V^T . [P_hi | P_lo]^T   M = 128 latent columns per block of four (A: the same codes, MN-major),
//                                           K = 128 tokens in steps of 32: 16 MMAs of N = 2 NR (hi and lo * 2^4 in
//                                           columns of their own, added at the end), or, where those do not fit, 32 of
//                                           N = NR (lo as e5m2)
// (NR: the rows rounded up to 16, 32 or 48).  Scores and O^T fit one SM's tensor memory, so a block is read once, by one
// SM, and nothing crosses SMs.  The bound is HBM: 580 bytes a token.  B 64, H 16, 4K: 45 us for the attend phase, 24 at a
// copy's rate; once under way a tile takes 2.0 us an SM (5.5 TB/s), the rest is the start (5500 cycles to the first
// copy, then all SMs' first tiles at once) and the end (scores, softmax, aggregation and output of the last tile, 7000).
// A ring of 2.75 tiles instead of two changed that by 2 %.  Waiting for the next tile's copies before the aggregation at hand
// is issued, and a lo term with MMAs of its own, took 62 us.  The form of 48 rows keeps 52 bytes a thread in local memory.
//
// Softmax: a thread per token (tensor-memory lane) and half the rows; a set of four warps has a tile's 128 tokens.  A row's
// maximum over a warp's tokens is a warp reduction, then the set's warps exchange them at one barrier and each decides on
// the reference exponent (RowRef in decode8_common.cuh) by itself; the token's scale is one register.
//
// Warps: 0..7 softmax (set = warp / 4), 8 copies, 9 MMAs, 10 what a tile's rows ask of the references (TileAsks), 12..15
// rescaling of O^T and a segment's output.  Scheduling and output are the pair kernel's (decode8_tc.cu).  Every wait is bounded.
#include <math_constants.h>

#include "decode8_common.cuh"

namespace mla {

namespace sm8 {

using namespace d8;

constexpr int kChunk = kBlock8Chunk;
constexpr int kSoftWarps = 8, kSoftThreads = 256;
constexpr int kWarpProducer = 8, kWarpMma = 9, kWarpScan = 10, kWarpEpi = 12;
constexpr int kThreads = 512;

constexpr uint32_t kNbSet = 1;  // named barriers 1, 2: the four softmax warps of a set

constexpr int kBFull = 0, kBEmpty = 4, kBSFull = 8, kBSEmpty = 10, kBPReady = 12, kBPFree = 14, kBQReady = 16, kBOFull = 17,
              kBOFree = 18, kBRescReq = 19, kBRescDone = 20, kBODrain = 21, kBLReady = 22, kBFin = 23, kNumBars = 24;

template <int NR>
struct Lay {
    static constexpr bool kStack = 12 * NR <= 512;           // hi and lo of P in accumulator columns of their own
    static constexpr int kN = 2 * NR;                        // columns of a score buffer
    static constexpr int kOC = kStack ? 2 * NR : NR;         // accumulator columns of a latent block
    static constexpr int kRN = NR / 2;                       // rows of a softmax thread
    static constexpr uint32_t kTmemCols = 2 * kN + 4 * kOC <= 256 ? 256 : 512;
    static constexpr int kOffRing = 0;                       // two tiles
    static constexpr int kQChunk = kN * 128;                 // [hi rows | lo rows] x 128 columns, swizzled
    static constexpr int kOffQ = 2 * kTileBytes;             // four chunks, then the RoPE columns (64 bytes a row)
    static constexpr int kOffP = kOffQ + 4 * kQChunk + kN * 64;
    static constexpr int kPBytes = kN * 128;                 // [hi rows | lo rows] x 128 tokens, swizzled
    static constexpr int kOffD = kOffP + 2 * kPBytes;        // [2 buffers][NR] int8 rescale exponents
    static constexpr int kOffRowF = kOffD + 2 * NR;          // [NR] fp32: 2^a scale log2 e
    static constexpr int kOffMax = kOffRowF + 4 * NR;        // [2 tiles][8 warps][kRN] row maxima
    static constexpr int kOffRef = kOffMax + 16 * kRN * 4;   // [8 warps][kRN] reference exponents, as the warp broadcasts them
    static constexpr int kOffL = kOffRef + 8 * kRN * 4;      // [8 warps][kRN] a segment's sums
    static constexpr int kOffT = kOffL + 8 * kRN * 4;        // [8 warps][kRN] the second sums (not kStack)
    static constexpr int kOffLR = kOffT + (kStack ? 0 : 8 * kRN * 4);  // [2 sets][kRN] its references
    static constexpr int kOffF = kOffLR + 2 * kRN * 4;       // [4 tiles][128] lifts of the tokens
    static constexpr int kOffAsk = kOffF + 4 * kTile;        // [4 tiles] TileAsks
    static constexpr int kOffBar = kOffAsk + 4 * 8;
    static constexpr int kOffTail = kOffBar + kNumBars * 8;  // tmem base, abort flag, rescale place, [total, sequence, tile]
    static constexpr int kSmemBytes = kOffTail + 32;
    static_assert(2 * kN + 4 * kOC <= 512, "tensor memory");
    static_assert(kOffQ % 1024 == 0 && kQChunk % 1024 == 0 && kOffP % 1024 == 0 && kPBytes % 1024 == 0, "swizzle atoms");
    static_assert(kOffD % 16 == 0 && kOffRowF % 16 == 0 && kOffRef % 16 == 0 && kOffL % 16 == 0 && kOffBar % 8 == 0, "");
    static_assert(kSmemBytes <= 232448, "shared memory budget");
    __device__ static constexpr uint32_t col_s(uint32_t sb) { return sb * kN; }
    __device__ static constexpr uint32_t col_o(uint32_t c) { return 2 * kN + c * kOC; }
};

__device__ __forceinline__ void raise_abort(volatile int* abort_flag, int32_t* dev_status) {
    *abort_flag = 1;
    if (dev_status) atomicOr(dev_status, MLA_DEVERR_TIMEOUT);
}

// A unit is a tile of a row.  The largest P' of the first 128 tokens goes into (8, 16]: few rows rise 2^5 above that, a move is
// cheaper here (at most 48 rows), and the stacked lo term's steps (2^-13) are then 2^-16 of the largest.
using Ref = RowRef<4, 6, 3>;

// Maximum over the warp's 32 lanes (NaN only if all are).
__device__ __forceinline__ float warp_max_f32(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

template <int NR>
__global__ void __launch_bounds__(kThreads, 1) decode8_sm_kernel(const Params p) {
    using L = Lay<NR>;
    constexpr int RN = L::kRN;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffTail);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kOffTail + 4);
    volatile int* resc_at = reinterpret_cast<volatile int*>(smem + L::kOffTail + 8);
    int* first = reinterpret_cast<int*>(smem + L::kOffTail + 12);
    volatile int never = 0;

    if ((sbase & 1023u) != 0) {
        if (tid == 0 && p.dev_status) atomicOr(p.dev_status, MLA_DEVERR_TIMEOUT);
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < 4; ++i) {
            mbar_init(&bars[kBFull + i], 1);
            mbar_init(&bars[kBEmpty + i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars[kBSFull + i], 2);  // the scores' MMAs and the scan of its rows
            mbar_init(&bars[kBSEmpty + i], kSoftThreads);
            mbar_init(&bars[kBPReady + i], kSoftThreads);
            mbar_init(&bars[kBPFree + i], 1);
        }
        mbar_init(&bars[kBQReady], kSoftThreads);
        mbar_init(&bars[kBOFull], 1);
        mbar_init(&bars[kBOFree], 128);
        mbar_init(&bars[kBRescReq], 1);
        mbar_init(&bars[kBRescDone], 128);
        mbar_init(&bars[kBODrain], 1);
        mbar_init(&bars[kBLReady], kSoftWarps);
        mbar_init(&bars[kBFin], 1);
        *abort_flag = 0;
        *resc_at = 0;
        fence_mbar_init();
    }
    if (warp == kWarpProducer) tmem_alloc(tmem_slot, L::kTmemCols);
    // everything above touches only this CTA's own resources; the call's inputs are read after this wait
    grid_dependency_wait();
    const int pidx = static_cast<int>(blockIdx.x);
    if (warp == 0) find_first(p, pidx, lane, first);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int Nt = first[0];
    SegWalk walk;
    walk.b = first[1];
    walk.tb = first[2];
    walk.lo = static_cast<int>((static_cast<int64_t>(pidx) * Nt) / p.P_g);
    walk.hi = static_cast<int>((static_cast<int64_t>(pidx + 1) * Nt) / p.P_g);
    walk.pidx = pidx;

    if (warp == kWarpProducer) {
        // ---- copies: a tile's codes as 32 and 40 KB, read by this SM only, once
        if (lane == 0) {
            SegWalk w = walk;
            Seg s;
            uint32_t n = 0;
            bool ok = true;
            const uint64_t once = l2_policy_evict_first();
            while (ok && w.next(p, s)) {
                for (int t = s.t0; ok && t < s.t1; ++t, ++n) {
                    const uint8_t* src = block_of(p, s.tab[t], true);
                    const uint32_t u = n >> 1, base = (n & 1u) * kTileBytes, bi = 2 * (n & 1u);
                    ok = mbar_wait(&bars[kBEmpty + bi], (u & 1u) ^ 1u, abort_flag, kLimitNs);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&bars[kBFull + bi], kCopyA);
                    bulk_load_hint(sbase + L::kOffRing + base, src, kCopyA, &bars[kBFull + bi], once);
                    // (both halves of a slot are released together)
                    ok = mbar_wait(&bars[kBEmpty + bi + 1], (u & 1u) ^ 1u, abort_flag, kLimitNs);
                    if (!ok) {
                        mbar_wait(&bars[kBFull + bi], u & 1u, &never, kLimitNs);
                        break;
                    }
                    mbar_arrive_expect_tx(&bars[kBFull + bi + 1], kCopyB);
                    bulk_load_hint(sbase + L::kOffRing + base + kCopyA, src + kCopyA, kCopyB, &bars[kBFull + bi + 1], once);
                }
            }
            if (!ok) raise_abort(abort_flag, p.dev_status);
            // let every issued copy land before the CTA can exit
            for (uint32_t i = (n > 2 ? n - 2 : 0); i < n; ++i)
                for (int k = 0; k < 2; ++k)
                    mbar_wait(&bars[kBFull + 2 * (i & 1u) + k], (i >> 1) & 1u, &never, kLimitNs);
        }
        __syncwarp();
    } else if (warp == kWarpMma) {
        // ---- MMA issuer: the scores of a tile go out as soon as it is there, its aggregation as soon as P is: whichever of
        //      the next two is ready first (waiting for a copy with a P at hand would hold that tile's slot, and the copy
        //      that wants it)
        const bool leader = elect_one();
        const uint32_t tm = uniform(tmem);
        constexpr uint32_t idesc_s = idesc_f8_f32(128, L::kN, false, false);
        constexpr uint32_t idesc_hi = idesc_f8_f32(128, L::kStack ? L::kN : NR, true, false);
        constexpr uint32_t idesc_lo = idesc_f8_f32(128, NR, true, false, false, true);
        const uint64_t k_desc = sdesc_sw128(sbase + L::kOffRing, 16, 1024);            // K-major chunks
        const uint64_t kr_desc = sdesc_sw64(sbase + L::kOffRing + kBlock8Rope, 16, 512);
        const uint64_t v_desc = sdesc_sw128(sbase + L::kOffRing, kChunk, 1024);        // the same chunks MN-major
        const uint64_t q_desc = sdesc_sw128(sbase + L::kOffQ, 16, 1024);
        const uint64_t qr_desc = sdesc_sw64(sbase + L::kOffQ + 4 * L::kQChunk, 16, 512);
        const uint64_t p_desc = sdesc_sw128(sbase + L::kOffP, 16, 1024);
        SegWalk w = walk;
        Seg s;
        uint32_t n0 = 0, kseg = 0, nresc = 0;  // tiles of the segments before
        bool ok = true;
        while (ok && w.next(p, s)) {
            if (leader) ok = mbar_wait(&bars[kBQReady], kseg & 1u, abort_flag, kLimitNs);
            ok = __any_sync(0xffffffffu, ok && leader);
            const uint32_t tiles = static_cast<uint32_t>(s.t1 - s.t0);
            uint32_t is = 0, ip = 0;  // tiles whose scores are issued, tiles aggregated
            while (ok && ip < tiles) {
                const uint32_t n = n0 + is, sb = n & 1u, us = n >> 1;
                const uint32_t m = n0 + ip, pb = m & 1u, um = m >> 1;
                int what = 0;  // 1: scores of tile is, 2: aggregation of tile ip, 3: give up
                if (leader) {
                    uint64_t since = 0;
                    uint32_t it = 0;
                    while (what == 0) {
                        if (ip < is && mbar_poll(smem_u32(&bars[kBPReady + pb]), um & 1u)) what = 2;
                        else if (is < tiles && is < ip + 2 && mbar_poll(smem_u32(&bars[kBSEmpty + sb]), (us & 1u) ^ 1u) &&
                                 mbar_poll(smem_u32(&bars[kBFull + 2 * sb]), us & 1u) &&
                                 mbar_poll(smem_u32(&bars[kBFull + 2 * sb + 1]), us & 1u))
                            what = 1;
                        else if ((++it & 255u) == 0) {
                            const uint64_t now = globaltimer_ns();
                            if (since == 0) since = now;
                            if (*abort_flag || now - since > kLimitNs) what = 3;
                        }
                    }
                    if (what == 2 && ip == 0 && !mbar_wait(&bars[kBOFree], (kseg & 1u) ^ 1u, abort_flag, kLimitNs)) what = 3;
                }
                what = __reduce_max_sync(0xffffffffu, leader ? what : 0);
                if (what == 3) {
                    ok = false;
                    break;
                }
                if (what == 1) {
                    const int nvalid = min(kTile, s.L - (s.t0 + static_cast<int>(is)) * kTile);
                    if (nvalid < kTile) {
                        // rows past the sequence end: P is 0 there, make V 0 too (no 0 * NaN); their scores are masked
                        const int nz = (kTile - nvalid) * 8;  // 16-byte units per chunk
                        for (int i = lane; i < 4 * nz; i += 32) {
                            const int c = i / nz, u = i % nz;
                            *reinterpret_cast<uint4*>(smem + L::kOffRing + sb * kTileBytes + c * kChunk + nvalid * 128 + u * 16) =
                                make_uint4(0, 0, 0, 0);
                        }
                        fence_proxy_async_cta();
                    }
                    __syncwarp();
                    const uint32_t sbu = uniform(sb);
                    if (elect_one()) {
                        tc_fence_after();
                        const uint64_t off = static_cast<uint64_t>(sbu * kTileBytes) >> 4;
                        const uint32_t d = tm + L::col_s(sbu);
#pragma unroll 1
                        for (int c = 0; c < 4; ++c)
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                mma8_ss(d, k_desc + off + ((c * kChunk + kk * 32) >> 4), q_desc + ((c * L::kQChunk + kk * 32) >> 4),
                                        idesc_s, (c | kk) ? 1u : 0u);
                        mma8_ss(d, kr_desc + off, qr_desc, idesc_s, 1u);
                        mma8_ss(d, kr_desc + off + 2, qr_desc + 2, idesc_s, 1u);
                        mma_commit(smem_u32(&bars[kBSFull + sbu]));
                    }
                    __syncwarp();
                    ++is;
                    continue;
                }
                if (ip > 0 && __any_sync(0xffffffffu, 4 * lane < NR && reinterpret_cast<const uint32_t*>(
                                                                           smem + L::kOffD + pb * NR)[lane] != 0)) {
                    // some row's reference moved: have O^T rescaled once all earlier MMAs are done
                    if (leader) {
                        *resc_at = static_cast<int>(pb * NR);
                        mma_commit(smem_u32(&bars[kBODrain]));
                        mbar_arrive(&bars[kBRescReq]);
                        ok = mbar_wait(&bars[kBRescDone], nresc & 1u, abort_flag, kLimitNs);
                    }
                    ++nresc;
                    ok = __any_sync(0xffffffffu, ok && leader);
                    if (!ok) break;
                }
                const uint32_t pbu = uniform(pb), accum = uniform(ip > 0 ? 1u : 0u);
                if (elect_one()) {
                    tc_fence_after();
                    const uint64_t v = v_desc + (static_cast<uint64_t>(pbu * kTileBytes) >> 4);
                    const uint64_t pd = p_desc + (static_cast<uint64_t>(pbu * L::kPBytes) >> 4);
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        const uint32_t o = tm + L::col_o(c);
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const uint64_t vc = v + ((c * kChunk + u * 4096) >> 4);
                            mma8_ss(o, vc, pd + 2 * u, idesc_hi, u ? 1u : accum);
                            if (!L::kStack) mma8_ss(o, vc, pd + 2 * u + ((NR * 128) >> 4), idesc_lo, 1u);
                        }
                        if (c & 1) mma_commit(smem_u32(&bars[kBEmpty + 2 * pbu + (c >> 1)]));
                    }
                    mma_commit(smem_u32(&bars[kBPFree + pbu]));
                    if (ip + 1 == tiles) mma_commit(smem_u32(&bars[kBOFull]));
                }
                __syncwarp();
                ++ip;
            }
            n0 += tiles;
            ++kseg;
        }
        if (!ok && leader) raise_abort(abort_flag, p.dev_status);
        if (leader) {
            mma_commit(smem_u32(&bars[kBFin]));
            mbar_wait(&bars[kBFin], 0, &never, kLimitNs);
        }
        __syncwarp();
    } else if (warp < kSoftWarps) {
        // ---- softmax: set k has rows k RN .. k RN + RN - 1; thread = token 32 qd + lane of a tile
        const int qd = warp & 3, set = warp >> 2, row0 = set * RN;
        const int tk = 32 * qd + lane;
        const uint32_t t_lane = tmem + (static_cast<uint32_t>(32 * qd) << 16);
        float* refs = reinterpret_cast<float*>(smem + L::kOffRef) + warp * RN;
        const float* rowf_all = reinterpret_cast<const float*>(smem + L::kOffRowF);
        // the token's dither, for both halves of a pair of rows, but for what depends on the tile
        const uint32_t dither0 = (rev4(tk & 15) << 4) * 0x00010001u;
        SegWalk w = walk;
        Seg s;
        uint32_t n = 0, kseg = 0;
        bool ok = true;
        while (ok && w.next(p, s)) {
            // the token's scale in the tiles to come, a tile ahead (the table entry two ahead)
            auto entry = [&](int t) { return t < s.t1 ? s.tab[t] : 0; };
            auto scale_bits = [&](int32_t e, int t) {
                return (t < s.t1 && t * kTile + tk < s.L)
                           ? reinterpret_cast<const uint32_t*>(block_of(p, e, false) + kBlock8Scales)[tk]
                           : 0x3F800000u;
            };
            const int32_t e0 = entry(s.t0);
            int32_t e1 = entry(s.t0 + 1);
            // the segment's query rows as hi and lo codes.  The previous segment's score MMAs are done (this warp has read
            // its last scores), but other warps may still want the rows' factors: they are read before the last tile's
            // P is announced.
            {
                constexpr int kRW = NR / kSoftWarps;  // rows a warp: warp, warp + 8, ..
                uint4 x[kRW][3];
#pragma unroll
                for (int i = 0; i < kRW; ++i) {
                    const int r = warp + kSoftWarps * i;
                    const uint4* src = reinterpret_cast<const uint4*>(p.q + (static_cast<int64_t>(s.b) * p.R + r) * kRow);
#pragma unroll
                    for (int k = 0; k < 3; ++k) {
                        x[i][k] = make_uint4(0, 0, 0, 0);
                        if (r < p.R && lane + 32 * k < 72) x[i][k] = src[lane + 32 * k];
                    }
                }
                if (kseg > 0)  // every warp past the last tile
                    ok = mbar_wait(&bars[kBLReady], (kseg - 1) & 1u, abort_flag, kLimitNs);
#pragma unroll
                for (int i = 0; i < kRW; ++i) {
                    const int r = warp + kSoftWarps * i;
                    uint32_t m2 = 0;
#pragma unroll
                    for (int k = 0; k < 3; ++k)
                        m2 = max_abs2(max_abs2(max_abs2(max_abs2(m2, x[i][k].x), x[i][k].y), x[i][k].z), x[i][k].w);
                    const uint32_t top = __reduce_max_sync(0xffffffffu, max(m2 & 0xFFFFu, m2 >> 16));
                    const int a = top < 0x7F80u ? row_exp(top) : 0;
                    const float inv = exp2_int(-a);
                    // an infinity or NaN in the query: every score of the row is NaN
                    if (lane == 0)
                        reinterpret_cast<float*>(smem + L::kOffRowF)[r] = top < 0x7F80u ? exp2_int(a) * p.scale_log2 : CUDART_NAN_F;
#pragma unroll
                    for (int k = 0; k < 3; ++k) {
                        const int u = lane + 32 * k;  // columns 8 u .. 8 u + 7
                        if (u >= 72) continue;
                        uint2 hi, lo;
                        split4_q(x[i][k].x, x[i][k].y, inv, hi.x, lo.x);
                        split4_q(x[i][k].z, x[i][k].w, inv, hi.y, lo.y);
                        const int rl = NR + r;
                        uint8_t *ah, *al;
                        if (u < 64) {
                            uint8_t* c = smem + L::kOffQ + (u >> 4) * L::kQChunk + (u & 1) * 8;
                            ah = c + r * 128 + ((((u >> 1) & 7) ^ (r & 7)) << 4);
                            al = c + rl * 128 + ((((u >> 1) & 7) ^ (rl & 7)) << 4);
                        } else {
                            uint8_t* c = smem + L::kOffQ + 4 * L::kQChunk + (u & 1) * 8;
                            ah = c + r * 64 + ((((u >> 1) & 3) ^ ((r >> 1) & 3)) << 4);
                            al = c + rl * 64 + ((((u >> 1) & 3) ^ ((rl >> 1) & 3)) << 4);
                        }
                        *reinterpret_cast<uint2*>(ah) = hi;
                        *reinterpret_cast<uint2*>(al) = lo;
                    }
                }
            }
            fence_proxy_async_cta();
            tc_fence_before();
            mbar_arrive(&bars[kBQReady]);
            ok = mbar_wait(&bars[kBQReady], kseg & 1u, abort_flag, kLimitNs) && ok;  // every row's factor is there
            // sums of P' / s, and (where lo has 3 bits) of P' as the MMAs have it
            float rowf[RN], lp[RN], tp[L::kStack ? 1 : RN];
#pragma unroll
            for (int i = 0; i < RN; ++i) {
                rowf[i] = rowf_all[row0 + i];
                lp[i] = 0.f;
                if (!L::kStack) tp[i] = 0.f;
            }
            // lane i < RN: row row0 + i's reference (rows of no query: one that makes P 0, and stays)
            float R = lane < RN && row0 + lane < p.R ? kNoRef : -kNoRef;
            uint32_t sc = scale_bits(e0, s.t0);
            RowPeak peak = {R, R};
            LowUnit low = {0.f, kNoTile};
            const int lim0 = s.L - p.n_q + 1;  // keys below this are visible to every query of the step
            for (int t = s.t0; t < s.t1; ++t, ++n) {
                const uint32_t sb = n & 1u, us = n >> 1;
                const float st = __uint_as_float(sc);
                float inv_s = __uint_as_float(0x7F000000u - sc);
                float et = static_cast<float>(static_cast<int>(sc >> 23) - 127);
                sc = scale_bits(e1, t + 1);
                e1 = entry(t + 2);
                ok = mbar_wait(&bars[kBSFull + sb], us & 1u, abort_flag, kLimitNs) && ok;
                __syncwarp();
                tc_fence_after();
                float y[RN];
                {
                    uint32_t h[RN], l[RN];
#pragma unroll
                    for (int i = 0; i < RN; i += 8) {
                        tmem_ld8(t_lane + L::col_s(sb) + row0 + i, h + i);
                        tmem_ld8(t_lane + L::col_s(sb) + NR + row0 + i, l + i);
                    }
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < RN; ++i) y[i] = __uint_as_float(h[i]) + __uint_as_float(l[i]);
                }
                tc_fence_before();
                mbar_arrive(&bars[kBSEmpty + sb]);
                const int tok = t * kTile + tk;
                const TileAsks& ask = reinterpret_cast<const TileAsks*>(smem + L::kOffAsk)[n & 3u];
                if (ask.lift) {
                    const int m = smem[L::kOffF + (n & 3u) * kTile + tk];
                    if (m > 0 && tok < s.L) {
                        et -= static_cast<float>(m);
                        inv_s *= exp2_int(m);
                        if (set == 0) {  // (the scores are formed)
                            ok = mbar_wait(&bars[kBFull + 2 * sb], us & 1u, abort_flag, kLimitNs) &&
                                 mbar_wait(&bars[kBFull + 2 * sb + 1], us & 1u, abort_flag, kLimitNs) && ok;
                            lift_row(smem + L::kOffRing + sb * kTileBytes + tk * 128, m);
                        }
                    }
                    __syncwarp();
                }
                // y = log2(p s_t), before the reference
#pragma unroll
                for (int i = 0; i < RN; ++i) y[i] = fmaf(y[i] * st, rowf[i], et);
                if (tok >= lim0) {
                    bool bad = false;  // a token that not every query sees: NaN made 0 in V (its scores are NaN, and formed)
#pragma unroll
                    for (int i = 0; i < RN; ++i) bad = bad || y[i] != y[i];
                    if (bad && set == 0 && tok < s.L) {
                        ok = mbar_wait(&bars[kBFull + 2 * sb], us & 1u, abort_flag, kLimitNs) &&
                             mbar_wait(&bars[kBFull + 2 * sb + 1], us & 1u, abort_flag, kLimitNs) && ok;
                        nan_to_zero_row(smem + L::kOffRing + sb * kTileBytes + tk * 128);
                    }
#pragma unroll
                    for (int i = 0; i < RN; ++i)
                        if (tok >= lim0 + (row0 + i) / p.H) y[i] = -CUDART_INF_F;
                }
                // the tile's row maxima: lane i gets row row0 + i's over the warp's tokens, then over the set's
                float top = -CUDART_INF_F;
#pragma unroll
                for (int i = 0; i < RN; ++i) {
                    const float v = warp_max_f32(y[i]);
                    if (lane == i) top = v;
                }
                float* mx = reinterpret_cast<float*>(smem + L::kOffMax) + (8 * sb + 4 * set) * RN;
                if (lane < RN) mx[qd * RN + lane] = top;
                if (bar_red_or(kNbSet + set, 128, !ok || *abort_flag != 0)) {
                    ok = false;
                    break;
                }
                if (lane < RN && row0 + lane < p.R)
                    top = fmaxf(fmaxf(mx[lane], mx[RN + lane]), fmaxf(mx[2 * RN + lane], mx[3 * RN + lane]));
                else top = R;
                const uint32_t dither = dither0 + dither_mask(tk >> 4, t);
                if (t == s.t0 && R == kNoRef) R = Ref::first(top, peak);
                int d = 0;
                if (!__all_sync(0xffffffffu, Ref::stays(top, R))) {
                    const float was = R;
                    R = Ref::moved(top, R, t > s.t0, n, ask.eager != 0, low, peak);
                    d = ref_exp(was, R);
                }
                if (__any_sync(0xffffffffu, d != 0)) {
#pragma unroll
                    for (int i = 0; i < RN; ++i) {
                        const float f = ref_factor(__shfl_sync(0xffffffffu, d, i));
                        lp[i] *= f;
                        if (!L::kStack) tp[i] *= f;
                    }
                }
                if (lane < RN) refs[lane] = R;
                __syncwarp();
                uint32_t hi[RN / 4], lo[RN / 4];
#pragma unroll
                for (int i = 0; i < RN; i += 4) {
                    const float4 R4 = *reinterpret_cast<const float4*>(refs + i);
                    const float Rs[4] = {R4.x, R4.y, R4.z, R4.w};
                    float v[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        v[k] = ex2_approx(y[i + k] - Rs[k]);  // (without any visible token yet: y = -inf, P = 0)
                        lp[i + k] = fmaf(v[k], inv_s, lp[i + k]);
                    }
                    if (L::kStack) {
                        split4_p16(v[0], v[1], v[2], v[3], (dither >> 1) & 0x007F007Fu, hi[i / 4], lo[i / 4]);
                    } else {
                        const float2 a = bf16x2_f32(cvt_bf16x2(v[0], v[1])), b = bf16x2_f32(cvt_bf16x2(v[2], v[3]));
                        tp[i] = fmaf(a.x, inv_s, tp[i]);
                        tp[i + 1] = fmaf(a.y, inv_s, tp[i + 1]);
                        tp[i + 2] = fmaf(b.x, inv_s, tp[i + 2]);
                        tp[i + 3] = fmaf(b.y, inv_s, tp[i + 3]);
                        split4_p(a.x, a.y, b.x, b.y, dither, dither, hi[i / 4], lo[i / 4]);
                    }
                }
                ok = mbar_wait(&bars[kBPFree + sb], (us & 1u) ^ 1u, abort_flag, kLimitNs) && ok;
                // row r, token tk: byte tk % 16 of the 16-byte unit tk / 16, at (unit ^ (row % 8)) of its 128-byte row
                uint8_t* pb = smem + L::kOffP + sb * L::kPBytes + (tk & 15);
#pragma unroll
                for (int i = 0; i < RN; ++i) {
                    const int r = row0 + i;
                    uint8_t* at = pb + r * 128 + (((tk >> 4) ^ (r & 7)) << 4);
                    at[0] = static_cast<uint8_t>(hi[i / 4] >> (8 * (i & 3)));
                    at[NR * 128] = static_cast<uint8_t>(lo[i / 4] >> (8 * (i & 3)));  // (NR is a multiple of 8: the same place)
                }
                if (qd == 0 && lane < RN) reinterpret_cast<int8_t*>(smem + L::kOffD)[sb * NR + row0 + lane] = static_cast<int8_t>(d);
                fence_proxy_async_cta();
                mbar_arrive(&bars[kBPReady + sb]);
            }
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            // the rows' sums over this warp's tokens, with the references they are relative to, once the previous segment's
            // have been read
            if (kseg > 0) ok = __all_sync(0xffffffffu, mbar_wait(&bars[kBOFree], (kseg - 1) & 1u, abort_flag, kLimitNs));
            if (!ok) break;
            float sum = 0.f, tsum = 0.f;
#pragma unroll
            for (int i = 0; i < RN; ++i) {
                float v = lp[i], t = L::kStack ? 0.f : tp[i];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    v += __shfl_xor_sync(0xffffffffu, v, o);
                    if (!L::kStack) t += __shfl_xor_sync(0xffffffffu, t, o);
                }
                if (lane == i) {
                    sum = v;
                    tsum = t;
                }
            }
            if (lane < RN) {
                reinterpret_cast<float*>(smem + L::kOffL)[warp * RN + lane] = sum;
                if (!L::kStack) reinterpret_cast<float*>(smem + L::kOffT)[warp * RN + lane] = tsum;
                if (qd == 0) reinterpret_cast<float*>(smem + L::kOffLR)[row0 + lane] = R;  // (the set's warps have the same)
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[kBLReady]);
            ++kseg;
        }
        if (!ok) raise_abort(abort_flag, p.dev_status);
    } else if (warp == kWarpScan) {
        // ---- what each tile asks of the references (TileAsks), ahead of the softmax, which is past tile n - 3 where it has read
        //      the scores of tile n - 2.  A tile's codes stay until its aggregation, after the softmax.
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
                ok = mbar_wait(&bars[kBFull + 2 * sb], us & 1u, abort_flag, kLimitNs) &&
                     mbar_wait(&bars[kBFull + 2 * sb + 1], us & 1u, abort_flag, kLimitNs);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                // (the buffer of lifts is free already: SEmpty of the tile before this one has been seen)
                const TileAsks ask = scan.tile(smem + sb * kTileBytes, min(kTile, s.L - t * kTile), bits, lane,
                                                smem + L::kOffF + (n & 3u) * kTile);
                ok = __all_sync(0xffffffffu, mbar_wait(&bars[kBSEmpty + sb], (us & 1u) ^ 1u, abort_flag, kLimitNs));
                if (lane == 0) reinterpret_cast<TileAsks*>(smem + L::kOffAsk)[n & 3u] = ask;
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[kBSFull + sb]);
            }
        }
        if (!ok && lane == 0) raise_abort(abort_flag, p.dev_status);
    } else if (warp >= kWarpEpi) {
        // ---- rescaling and output: warps 12..15, lane = latent column 128 c + 32 qd + lane of block c
        const int qd = warp & 3;
        const uint32_t t_lane = tmem + (static_cast<uint32_t>(32 * qd) << 16);
        SegWalk w = walk;
        Seg s;
        uint32_t kseg = 0, nresc = 0;
        bool ok = true;
        while (ok && w.next(p, s)) {
            const uint64_t t0 = globaltimer_ns();
            uint32_t it = 0;
            for (;;) {
                int ev = 0;  // 1: O^T complete, 2: rescale request, 3: give up
                if (lane == 0) {
                    if (mbar_test(smem_u32(&bars[kBOFull]), kseg & 1u)) ev = 1;
                    else if (mbar_test(smem_u32(&bars[kBRescReq]), nresc & 1u)) ev = 2;
                    else if (*abort_flag) ev = 3;
                    else if ((++it & 255u) == 0 && globaltimer_ns() - t0 > kLimitNs) ev = 3;
                }
                ev = __shfl_sync(0xffffffffu, ev, 0);
                if (ev == 1) {
                    ok = mbar_wait(&bars[kBOFull], kseg & 1u, abort_flag, kLimitNs) &&
                         mbar_wait(&bars[kBLReady], kseg & 1u, abort_flag, kLimitNs);
                    break;
                }
                if (ev == 3) {
                    ok = false;
                    break;
                }
                if (ev == 2) {
                    ok = mbar_wait(&bars[kBRescReq], nresc & 1u, abort_flag, kLimitNs) &&
                         mbar_wait(&bars[kBODrain], nresc & 1u, abort_flag, kLimitNs);
                    __syncwarp();
                    tc_fence_after();
                    const int8_t* dd = reinterpret_cast<const int8_t*>(smem + L::kOffD + *resc_at);
#pragma unroll 1
                    for (int r = 0; r < NR; r += 8) {
                        float f[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) f[k] = ref_factor(dd[r + k]);
#pragma unroll
                        for (int part = 0; part < L::kOC / NR; ++part) {  // hi columns, lo columns
                            uint32_t v[4][8];
#pragma unroll
                            for (int c = 0; c < 4; ++c) tmem_ld8(t_lane + L::col_o(c) + part * NR + r, v[c]);
                            tmem_wait_ld();
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
#pragma unroll
                                for (int k = 0; k < 8; ++k) v[c][k] = __float_as_uint(__uint_as_float(v[c][k]) * f[k]);
                                tmem_st8(t_lane + L::col_o(c) + part * NR + r, v[c]);
                            }
                        }
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    mbar_arrive(&bars[kBRescDone]);
                    ++nresc;
                    if (!__all_sync(0xffffffffu, ok)) {
                        ok = false;
                        break;
                    }
                    continue;
                }
                __nanosleep(64);
            }
            ok = __all_sync(0xffffffffu, ok);
            __syncwarp();
            if (!ok) break;
            tc_fence_after();
            // R and the sums per row: the set's four warps ended with the same reference
            for (int r = 32 * qd + lane; r < p.R; r += 128) {
                const int at = (r / RN) * 4 * RN + r % RN;
                const float* part = reinterpret_cast<const float*>(smem + L::kOffL) + at;
                const float l = (part[0] + part[RN]) + (part[2 * RN] + part[3 * RN]);
                const float ref = reinterpret_cast<const float*>(smem + L::kOffLR)[r];
                float t = l;  // (the stacked lo term holds a bit more: one sum serves for both)
                if (!L::kStack) {
                    const float* tp = reinterpret_cast<const float*>(smem + L::kOffT) + at;
                    t = (tp[0] + tp[RN]) + (tp[2 * RN] + tp[3 * RN]);
                }
                p.ml_part[static_cast<int64_t>(s.slot) * p.rs + r] = make_float4(l != l ? 0.f : ref, l, t, 0.f);
            }
            // the workspace holds [column / 32][row] x 32 fp32, rs rows per slot
            float* oseg = p.o_part + static_cast<int64_t>(s.slot) * p.rs * kDc;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                float* to = oseg + ((4 * c + qd) * p.rs) * 32 + lane;
#pragma unroll 1
                for (int r = 0; r < NR; r += 8) {
                    uint32_t v[8], u[8];
                    tmem_ld8(t_lane + L::col_o(c) + r, v);
                    if (L::kStack) tmem_ld8(t_lane + L::col_o(c) + NR + r, u);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (r + k < p.R)
                            to[32 * (r + k)] = L::kStack ? fmaf(__uint_as_float(u[k]), 0x1p-4f, __uint_as_float(v[k])) : __uint_as_float(v[k]);
                }
            }
            tc_fence_before();
            mbar_arrive(&bars[kBOFree]);
            ++kseg;
        }
        if (!ok && lane == 0) raise_abort(abort_flag, p.dev_status);
    }

    // ------------------------------------------------------------------ teardown
    grid_dependents_launch();  // the merge kernel may be scheduled; it waits for this grid to finish
    tc_fence_before();
    __syncthreads();
    if (warp == kWarpProducer) {
        tc_fence_after();
        tmem_dealloc(tmem, L::kTmemCols);
    }
}

template <int NR>
cudaError_t launch(const Params& prm, cudaStream_t stream) {
    using L = Lay<NR>;
    cudaError_t e = cudaFuncSetAttribute(decode8_sm_kernel<NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmemBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(prm.P_g);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = L::kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, decode8_sm_kernel<NR>, prm);
}

}  // namespace sm8

cudaError_t launch_decode8_sm(const uint16_t* q, const uint8_t* cache, int64_t cap_blocks, const int32_t* block_table,
                              int max_blocks, const int32_t* kv_len, int B, int n_q, int H, float scale, int ctas,
                              float* o_part, float4* ml_part, int slots, int rs, int32_t* dev_status,
                              cudaStream_t stream) {
    const int R = n_q * H;
    if (R < 1 || R > kMaxSm8Rows || R > rs || ctas < 1 || B + ctas > slots) return cudaErrorInvalidValue;
    const d8::Params prm = {q, cache, block_table, kv_len, o_part, ml_part, dev_status, cap_blocks, max_blocks, B, n_q, H, R,
                            1, ctas, slots, rs, scale * 1.44269504088896340736f};
    if (R <= 16) return sm8::launch<16>(prm, stream);
    return R <= 32 ? sm8::launch<32>(prm, stream) : sm8::launch<48>(prm, stream);
}

}  // namespace mla
