// Latent attention over a 4-bit cache on tcgen05 / TMEM: the mathematics, the
// CTA pair and the scheduling of sm100_attend.cuh, with rows unpacked on the
// SM.  For query token (b, i) and all 128 heads:
//   S = scale * Q-hat . row^T,  P = softmax(S) (online),  o_lat = P . latents,  lse = ln sum exp S
//
// What bounds it: 416 bytes and 278,528 flop a row and query token are 669
// flop per byte, far above the 255 of the measured peaks, so the tensor cores
// bound it, and the cache's bandwidth does not (a 128-key tile takes an SM
// 1.2 us of HBM time against 1.4 us of score products at the measured rate).
//
// Split.  As the latent accumulator of 128 heads fills an SM's TMEM, a pair of
// CTAs shares a query token: the scorer (cluster rank 0) computes S and P, the
// accumulator (rank 1) sums P . latents.  Each of them fetches the packed rows
// and unpacks what it multiplies, because the unpacked rows (1024 bytes a row
// one way) would be three times the traffic of P between the two.
//   * Tiles of 128 keys: scores of 128 x 128 run the tensor cores at their full
//     rate (64 keys a tile at 0.77 of it).  Q-hat's latent part (256 columns)
//     and two score buffers (2 x 128) fill the scorer's TMEM; Q-hat's RoPE
//     part is the shared-memory A operand of the last four products.
//   * Unpacked latents stream through a ring of four chunks of 128 keys x 64
//     latents (bf16: the scores' A operand is bf16 and both operands have one
//     type); two sets of four warps unpack alternate chunks, a lane a row.
//   * P goes to the accumulator in units of 64 keys as fp16, scaled by 2^7, and
//     the accumulator unpacks the latents to fp16: every value is exact in
//     either type, and P keeps 11 bits where bf16 keeps 8.  P is at most 2^15
//     (the accumulated maximum may lag the true one by 2^8), and what fp16
//     drops is below 2^-32 of the row's sum a key.
//   * A row's latents are finite whatever its bytes are, so rows past the
//     sequence's end need no clearing: their scores are replaced by -infinity
//     (a NaN key only reaches its own score), and 0 times a finite number is 0.
//
// Measured (B200, 128 heads; bursts of twenty calls, and in brackets calls in a
// row for seconds): 1 x 4096 rows 28 us, most of it the latency of one tile and
// of the merge; 64 x 4096 rows 104 us; 8 x 131072 rows 311 (350) us, 940 (830)
// TFLOP/s; 128 x 2048..16384 rows with two queries 688 (776) us, 980 (870).  What holds the
// long ones up is power: at 993 W the clock falls to 1.75 GHz, and fewer
// instructions a value gained 5 % where deeper rings, other bank layouts and
// earlier hand-offs, which only hide latency, gained nothing.  Code counts too:
// inline waits whose spin loops did not fit the instruction cache, and an
// issuing branch that the compiler did not know to be uniform (lane == 0), cost
// a fifth each.
//
// Roles (640 threads; warp w reaches TMEM lanes 32*(w%4)..+31):
//   scorer:      warp 0 producer of packed rows; 1 TMEM owner and S issuer; 2-5 and 12-15 softmax (two per TMEM quarter,
//                64 keys each); 10, 11, 16, 17 unpack even chunks; 6-9 odd chunks, and both sets load a piece's Q-hat;
//                18 producer of keys
//   accumulator: warp 0 producer of packed rows; 1 TMEM owner and O issuer; 2-5 and 12-15 rescale / epilogue (two per
//                quarter, 256 columns each); 6-9 and 16-19 unpack; 10 returns consumed P slots; 11 notes the cuts
// Every wait is bounded and its expiry ends the kernel in order, as in
// sm100_attend.cuh.
#pragma once

#include "sm100_attend.cuh"
#include "sm100_pieces.cuh"
#include "sm100_unpack.cuh"

namespace mla {
namespace sm100 {
namespace pk {

constexpr int kTile = 128;  // keys of a score tile
constexpr int kUnit = 64;   // keys of a P slot and of an accumulator stage
constexpr int kThreads = 640;

constexpr int kRawRow = kPackNib + kPackScale;    // codes and scales of a row as they lie in memory: 288 bytes
constexpr int kRawBox = kUnit * kRawRow;          // 64 keys, 18 KB
// scorer: raw stages of 128 keys
constexpr int kRawStages = 2;
constexpr int kRawBytes = 2 * kRawBox;            // 36 KB
constexpr int kChunks = 4;
constexpr int kChunkBytes = kTile * 128;          // 16 KB: 128 keys x 64 bf16 latents, SW128
constexpr int kSlots = 3;
constexpr int kSlotP = kHeads * 128;              // 128 heads x 64 keys fp16, SW128
constexpr int kSlotBytes = kSlotP + kHeads * 8;   // + {rescale factor, sum of p} per head
constexpr int kOffChunk = kRawStages * kRawBytes;
constexpr int kOffRope = kOffChunk + kChunks * kChunkBytes;
constexpr int kOffQ = kOffRope + kChunkBytes;     // Q-hat's RoPE part (and the loaders' transposes), [128][128 B] SW128
constexpr int kOffStage = kOffQ + kHeads * 128;
constexpr int kOffRed = kOffStage + kSlots * kSlotBytes;    // [2 tiles][2 halves][128 rows]
constexpr int kOffFlag = kOffRed + 2 * 2 * kHeads * 4;      // [2 tiles][4 quarters][2]
constexpr int kScorerEnd = kOffFlag + 2 * 4 * 2 * 4;
// accumulator: raw stages of 64 keys
constexpr int kARawStages = kRawStages;
constexpr int kARawBytes = kRawBox;
constexpr int kVStages = 2;
constexpr int kVChunk = kUnit * 128;
constexpr int kVBytes = 8 * kVChunk;                        // 64 keys x 512 fp16 latents
constexpr int kOffV = kARawStages * kARawBytes;
constexpr int kOffSlots = kOffV + kVStages * kVBytes;
constexpr int kAccumEnd = kOffSlots + kSlots * kSlotBytes;
constexpr int kOffBars = ((kScorerEnd > kAccumEnd ? kScorerEnd : kAccumEnd) + 15) & ~15;
constexpr int kSmem = kOffBars + 512 + 1024;
static_assert(kRawBytes % 1024 == 0 && kARawBytes % 1024 == 0 && kSlotBytes % 1024 == 0, "1024-byte boundaries");
static_assert(kSmem <= 232448, "packed attention shared memory exceeds 227 KB");

constexpr int kTmemQ = 0;    // scorer: latent part of Q-hat, two bf16 per column
constexpr int kTmemS = 256;  // scorer: two score buffers of 128 columns
constexpr float kPShift = 7.0f;

enum {
    // scorer
    kRawFull = 0,                      // packed rows loaded (tx)
    kRawEmpty = kRawFull + kRawStages, // read by the eight unpacking warps
    kChFull = kRawEmpty + kRawStages,  // chunk unpacked (4 warps)
    kChEmpty = kChFull + kChunks,      // chunk multiplied (MMA commit)
    kRopeFull = kChEmpty + kChunks,    // keys loaded (tx)
    kRopeEmpty,                        // keys multiplied (MMA commit)
    kSFull,                            // S(g) complete (MMA commit)
    kSFree = kSFull + 2,               // S buffer read (8 warps)
    kQFull = kSFree + 2,               // Q-hat of a piece in place (8 warps)
    kQRead,                            // last S of a piece complete
    kSlotFree,                         // accumulator's P slot consumed (remote)
    // accumulator
    kARawFull = kSlotFree + kSlots,
    kARawEmpty = kARawFull + kARawStages,
    kVFull = kARawEmpty + kARawStages,  // unit unpacked (8 warps)
    kVEmpty = kVFull + kVStages,        // unit multiplied (MMA commit)
    kPFull = kVEmpty + kVStages,        // P of a unit landed (tx)
    kPDone = kPFull + kSlots,           // O of a unit complete (MMA commit)
    kRescaled = kPDone + kSlots,        // O rows ready for a unit (8 warps)
    kOFull = kRescaled + kSlots,
    kOFree,
    kDrain,
    kBars
};
static_assert(8 * (kBars + 2) <= 512, "barrier block too small");

struct Args {
    const int32_t* seqlens;
    const int32_t* n_seen;  // or NULL; only checked here
    int B, q_len, T_max;
    int ovh, min_units;  // of the split, in tiles
    float scale_log2;
    const __nv_bfloat16* q_hat;  // [B][q_len][128][576]
    __nv_bfloat16* o_lat;        // [B][q_len][128][512]
    int o_lat_v8;
    float* part_o;
    float* part_lse;
    float* lse;                  // [B][q_len][128] or NULL
    int4* cuts;                  // what the merge has to do, by sequence (cuts_by_seq) or by group: {sequence or -1, first, last group}
    int cuts_by_seq;
    int* status;
    uint64_t wait_limit_ns;
    int withhold_tile;           // test hook (>= 0): the loaders stop before this 64-key tile (see mla.h)
};

// mapRaw: codes and scales [B][T_max][144 x 16 bits], box of whole such rows x 64;
// mapRope: keys [B][T_max][64] bf16, box 64 x 64 rows, SW128.
__global__ void __launch_bounds__(kThreads, 1)
    packed_attend_kernel(const __grid_constant__ CUtensorMap mapRaw, const __grid_constant__ CUtensorMap mapRope, Args args) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ int s_scratch[64];
    __shared__ PieceShare s_share;
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* base_ptr = smem_raw + (base - raw);
    auto bar = [&](int i) { return base + kOffBars + 8u * i; };
    const uint32_t abort_addr = bar(kBars + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(base_ptr + kOffBars + 8 * (kBars + 1));
    const uint64_t lim = args.wait_limit_ns;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = cluster_ctarank() & 1;
    const uint32_t peer = rank ^ 1;
    const int cl = (int)cluster_id_x();
    const int q_len = args.q_len;
    const int grp = cl / q_len, qi = cl % q_len;

    if (threadIdx.x == 0) {
        auto init = [&](int first, int n, int count) {
            for (int i = 0; i < n; ++i) mbar_init(bar(first + i), count);
        };
        if (rank == 0) {
            init(kRawFull, kRawStages, 1);
            init(kRawEmpty, kRawStages, 8);
            init(kChFull, kChunks, 4);
            init(kChEmpty, kChunks, 1);
            init(kRopeFull, 1, 1);
            init(kRopeEmpty, 1, 1);
            init(kSFull, 2, 1);
            init(kSFree, 2, 8);
            init(kQFull, 1, 8);
            init(kQRead, 1, 1);
            init(kSlotFree, kSlots, 1);
        } else {
            init(kARawFull, kARawStages, 1);
            init(kARawEmpty, kARawStages, 8);
            init(kVFull, kVStages, 8);
            init(kVEmpty, kVStages, 1);
            init(kPFull, kSlots, 1);
            init(kPDone, kSlots, 1);
            init(kRescaled, kSlots, 8);
            init(kOFull, 1, 1);
            init(kOFree, 1, 8);
        }
        mbar_init(bar(kDrain), 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tensormap(&mapRaw);
        prefetch_tensormap(&mapRope);
    }
    if (warp == 1) {
        tmem_alloc(bar(kBars), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(base_ptr + kOffBars + 8 * kBars);
    pdl_wait();
    if (threadIdx.x == 0) pdl_trigger();
    // The clusters form groups of q_len, one cluster a query token; groups past the last whole one idle.
    const int groups = (int)(gridDim.x / 2) / q_len;
    const Batch batch = {args.seqlens, args.B, q_len, args.T_max, kTile, args.ovh};
    plan_share(batch, groups, grp, args.min_units, true, s_scratch, &s_share);
    const bool active = grp < groups;
    // Sequences with an invalid length: zeros, and -infinity for the log-sum-exps.
    for (int b = blockIdx.x; b < args.B; b += gridDim.x) {
        if (args.n_seen && threadIdx.x == 0 && args.n_seen[b] < q_len) atomicOr(args.status, MLA_STATUS_BAD_SEQLEN);
        if (batch.valid(batch.len(b))) continue;
        if (threadIdx.x == 0) {
            atomicOr(args.status, MLA_STATUS_BAD_SEQLEN);
            if (args.cuts_by_seq) args.cuts[b] = make_int4(-1, 0, 0, 0);
        }
        uint4* o = reinterpret_cast<uint4*>(args.o_lat + (size_t)b * q_len * kHeads * kLat);
        for (int i = threadIdx.x; i < q_len * kHeads * kLat / 8; i += kThreads) o[i] = make_uint4(0, 0, 0, 0);
        for (int i = threadIdx.x; args.lse && i < q_len * kHeads; i += kThreads)
            args.lse[(size_t)b * q_len * kHeads + i] = -CUDART_INF_F;
    }

    const int quarter = warp & 3;
    const int m = quarter * 32 + lane;
    const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
    const bool softmax_warp = (warp >= 2 && warp <= 5) || (warp >= 12 && warp <= 15);
    const int kh = warp >= 12 ? 1 : 0;
    int n_load = 0;  // loads issued (a producer's lane 0), for the teardown
    auto wait = [&](int i, int phase) { return warp_wait_fast<false>(bar(i), phase & 1, lim); };
    auto wait_peer = [&](int i, int phase) { return warp_wait_fast<true>(bar(i), phase & 1, lim); };  // completed by the other CTA

    // The pieces of the group: sequence, tiles k0..k1-1, and whether they are all of it.
    Pieces it(&s_share);
    int seq = 0, T = 0, k0 = 0, k1 = 0;
    bool whole = false, ok = true;
    if (!active) {
        // idle cluster (the cluster count is not a multiple of q_len)
    } else if (warp == 0) {
        // ======================================================== producer of packed rows (both CTAs), 64 rows a copy
        const int per = rank == 0 ? 2 : 1;  // copies of a stage
        const int full = rank == 0 ? (int)kRawFull : (int)kARawFull, empty = rank == 0 ? (int)kRawEmpty : (int)kARawEmpty;
        while (ok && it.next(seq, T, k0, k1, whole)) {
#pragma unroll 1
            for (int t = 2 * k0; t < 2 * k1; t += per, ++n_load) {
                if (args.withhold_tile >= 0 && n_load * per >= args.withhold_tile) break;
                const int st = n_load % kRawStages;
                if (!wait(empty + st, n_load / kRawStages + 1) || *abort_flag) { ok = false; break; }
                if (lane == 0) {
                    const uint32_t dst = base + st * per * kRawBox;
                    mbar_arrive_expect_tx(bar(full + st), per * kRawBox);
                    for (int r = 0; r < per; ++r)
                        tma_load_3d(dst + r * kRawBox, &mapRaw, bar(full + st), 0, (t + r) * kUnit, seq);
                }
                __syncwarp();
            }
        }
    } else if (rank == 0 && warp == 18) {
        // ======================================================== scorer: producer of RoPE keys
        while (ok && it.next(seq, T, k0, k1, whole)) {
#pragma unroll 1
            for (int t = k0; t < k1; ++t, ++n_load) {
                if (!wait(kRopeEmpty, n_load + 1) || *abort_flag) { ok = false; break; }
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar(kRopeFull), kChunkBytes);
                    for (int r = 0; r < 2; ++r)
                        tma_load_3d(base + kOffRope + r * kUnit * 128, &mapRope, bar(kRopeFull), 0, t * kTile + r * kUnit, seq);
                }
                __syncwarp();
            }
        }
    } else if (rank == 0 && warp == 1) {
        // ======================================================== scorer: S issuer
        constexpr uint32_t idS = idesc_bf16_f32(kHeads, kTile, false, false);
        const uint64_t dChunk = smem_desc(base + kOffChunk, 16, 1024, kSw128);
        const uint64_t dRope = smem_desc(base + kOffRope, 16, 1024, kSw128);
        const uint64_t dQ = smem_desc(base + kOffQ, 16, 1024, kSw128);
        int g = 0;
        for (int seg = 0; ok && it.next(seq, T, k0, k1, whole); ++seg) {
            ok = wait(kQFull, seg);
#pragma unroll 1
            for (int t = k0; t < k1 && ok; ++t, ++g) {
                const int sb = g & 1;
                if (!wait(kSFree + sb, (g >> 1) + 1) || *abort_flag) { ok = false; break; }
                const uint32_t dS = tmem + kTmemS + kTile * sb;
                // eight chunks a tile: the ring of four returns to the same slots and phases every tile
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    ok = ok && wait(kChFull + c % kChunks, c / kChunks);
                    tc_fence_after();
                    if (ok && elect_one()) {
                        const uint64_t dB = dChunk + (((c % kChunks) * kChunkBytes) >> 4);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_f16_ts(dS, tmem + kTmemQ + 32 * c + 8 * k, dB + ((32 * k) >> 4), idS, (c | k) ? 1u : 0u);
                        mma_commit(bar(kChEmpty + c % kChunks));
                    }
                    __syncwarp();
                }
                if (!ok || !wait(kRopeFull, g)) { ok = false; break; }
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) mma_f16_ss(dS, dQ + ((32 * k) >> 4), dRope + ((32 * k) >> 4), idS, 1u);
                    mma_commit(bar(kRopeEmpty));
                    mma_commit(bar(kSFull + sb));
                    if (t == k1 - 1) mma_commit(bar(kQRead));
                }
                __syncwarp();
            }
        }
    } else if (rank == 0 && ((warp >= 6 && warp <= 11) || warp == 16 || warp == 17)) {
        // ======================================================== scorer: unpacking warps, a row of the tile a lane
        // Two sets of four warps take the even (10, 11, 16, 17) and the odd chunks
        // (6-9).  First they share a piece's Q-hat out in the same way: row m's 512
        // latent values -> TMEM columns 0..255, 64 values in turn, read coalesced
        // and transposed through the first set's own first chunk and the RoPE
        // part's buffer, where the second set's last block, the RoPE part, stays
        // as the shared-memory operand.
        const int odd = warp <= 9 ? 1 : 0;
        const int row = 32 * quarter + lane;
        const uint32_t row_at = base + kOffChunk + sw128(row, 0);
        const uint32_t qbuf = base + (odd ? kOffQ : kOffChunk) + quarter * 32 * 128;
        const int rr = lane >> 3, pc = lane & 7;
        int g = 0;
        for (int seg = 0; ok && it.next(seq, T, k0, k1, whole); ++seg) {
            const int u = seq * q_len + qi;
            const uint4* src = reinterpret_cast<const uint4*>(args.q_hat + ((size_t)u * kHeads + quarter * 32 + rr) * kRow) + pc;
            uint4 cur[8], nxt[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) cur[j] = __ldg(src + (size_t)(4 * j) * (kRow / 8) + 8 * odd);
            // the last S of the previous piece has read Q-hat and the chunks
            if (!wait(kQRead, seg + 1) || *abort_flag) { ok = false; break; }
            tc_fence_after();
#pragma unroll 1
            for (int i = 0; i < 4 + odd; ++i) {
                const int c = i < 4 ? 2 * i + odd : 8;
                if (i + 1 < 4 + odd) {
                    const int next = i + 1 < 4 ? c + 2 : 8;
#pragma unroll
                    for (int j = 0; j < 8; ++j) nxt[j] = __ldg(src + (size_t)(4 * j) * (kRow / 8) + 8 * next);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int r = 4 * j + rr;
                    st_shared_v4(qbuf + sw128(r, pc), cur[j].x, cur[j].y, cur[j].z, cur[j].w);
                }
                __syncwarp();
                if (c == 8) break;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t v[16];
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        ld_shared_v4u(qbuf + sw128(lane, 4 * h + q), v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                    tmem_st16(tmem + lane_addr + kTmemQ + 32 * c + 16 * h, v);
                }
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 8; ++j) cur[j] = nxt[j];
            }
            tmem_wait_st();
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kQFull));
#pragma unroll 1
            for (int t = k0; t < k1 && ok; ++t, ++g) {
                const int st = g % kRawStages;
                if (!wait(kRawFull + st, g / kRawStages) || *abort_flag) { ok = false; break; }
                const uint32_t raw_row = base + st * kRawBytes + row * kRawRow;
                RawChunk raw;
                raw.load(raw_row, odd);
#pragma unroll 1
                for (int c = odd; c < 8; c += 2) {
                    const int slot = c % kChunks;
                    if (!wait(kChEmpty + slot, c / kChunks + 1)) { ok = false; break; }
                    raw.unpack<false>(row_at + slot * kChunkBytes);
                    if (c + 2 < 8) raw.load(raw_row, c + 2);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(bar(kChFull + slot));
                        if (c >= 6) mbar_arrive(bar(kRawEmpty + st));
                    }
                }
            }
        }
    } else if (rank == 0 && softmax_warp) {
        // ======================================================== scorer: softmax warps
        // Half kh of a quarter's pair takes keys 64kh..64kh+63 of each score
        // row, which are P unit 2g + kh; the pair agrees on the row maximum
        // through shared memory at a named barrier, where both also learn
        // whether the other goes on (see sm100_attend.cuh).
        const uint32_t slot_peer = mapa(base + kOffSlots, peer);
        const uint32_t pfull_peer = mapa(bar(kPFull), peer);
        float* red = reinterpret_cast<float*>(base_ptr + kOffRed);
        volatile int* pair_ok = reinterpret_cast<volatile int*>(base_ptr + kOffFlag);
        const float sl2 = args.scale_log2;
        int g = 0;
        bool run = true;  // the pair's common decision
        while (run && it.next(seq, T, k0, k1, whole)) {
            float m_used = -CUDART_INF_F, l_part = 0.f;
            // query token qi of sequence b sees keys 0..T_b-q_len+qi
            const int n_keys = T - q_len + 1 + qi;
#pragma unroll 1
            for (int t = k0; t < k1; ++t, ++g) {
                const int sb = g & 1, unit = 2 * g + kh, slot = unit % kSlots;
                if (ok) ok = wait(kSFull + sb, g >> 1);
                tc_fence_after();
                const uint32_t s_addr = tmem + lane_addr + kTmemS + kTile * sb + kUnit * kh;
                const int seen = n_keys - (t * kTile + kUnit * kh);  // of this half's 64 keys
                if (ok && seen < kUnit) {  // keys past the query: their scores become -infinity
#pragma unroll 1
                    for (int j = seen < 0 ? 0 : seen; j < kUnit; ++j) tmem_st1(s_addr + j, 0xFF800000u);
                    tmem_wait_st();
                }
                // ---- the row maximum, then the weights: both passes read the scores from TMEM in short loops
                float mx = -CUDART_INF_F;
                if (ok) {
#pragma unroll 1
                    for (int j0 = 0; j0 < kUnit; j0 += 32) {
                        uint32_t v[32];
                        tmem_ld32(s_addr + j0, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; j += 2) mx = max3(mx, __uint_as_float(v[j]), __uint_as_float(v[j + 1]));
                    }
                }
                float* rg = red + (sb * 2) * kHeads;
                rg[kh * kHeads + m] = mx * sl2;
                volatile int* st_pair = pair_ok + (sb * 4 + quarter) * 2;
                if (lane == 0) st_pair[kh] = (ok && !*abort_flag) ? 1 : 0;
                named_bar_sync(1 + quarter, 64);
                if (!st_pair[0] || !st_pair[1]) {
                    run = ok = false;
                    break;
                }
                mx = fmaxf(rg[m], rg[kHeads + m]);
                float f = 1.0f;
                if (mx > m_used + 8.0f) {
                    if (t > k0) {
                        f = ex2(m_used - mx);
                        l_part *= f;
                    }
                    m_used = mx;
                }
                // p = 2^(s - m_used + 7)
                const float mb = m_used == -CUDART_INF_F ? 0.f : kPShift - m_used;
                // (A half meets a slot in every other of its phases, and a barrier's parity
                // tells only neighbouring phases apart.  The phase between was waited for
                // by the other half of the pair, one or two tiles ago, before the meeting
                // at the named barrier above.)
                if (ok && unit >= kSlots) ok = wait_peer(kSlotFree + slot, unit / kSlots + 1);
                if (ok) {
                    const uint32_t stg = base + kOffStage + slot * kSlotBytes;
                    // (two values an instruction where there is one for it)
                    const uint64_t sl2x2 = pack_f32x2(sl2, sl2), mbx2 = pack_f32x2(mb, mb);
                    uint64_t rs = 0;
#pragma unroll 1
                    for (int j0 = 0; j0 < kUnit; j0 += 16) {
                        uint32_t v[16], pk[8];
                        tmem_ld16(s_addr + j0, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            float p0, p1;
                            unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])), sl2x2, mbx2), p0, p1);
                            p0 = ex2(p0);
                            p1 = ex2(p1);
                            rs = add_f32x2(rs, pack_f32x2(p0, p1));
                            pk[j] = pack_f16(p0, p1);
                        }
                        st_shared_v4(stg + sw128(m, j0 / 8), pk[0], pk[1], pk[2], pk[3]);
                        st_shared_v4(stg + sw128(m, j0 / 8 + 1), pk[4], pk[5], pk[6], pk[7]);
                    }
                    float rs0, rs1;
                    unpack_f32x2(rs, rs0, rs1);
                    l_part += rs0 + rs1;
                    st_shared_v2(stg + kSlotP + 8 * m, __float_as_uint(kh ? 1.0f : f), __float_as_uint(l_part));
                    tc_fence_before();
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(bar(kSFree + sb));
                        const uint32_t dst = slot_peer + slot * kSlotBytes, pb = pfull_peer + 8 * slot;
                        const uint32_t po = quarter * 32 * 128, ao = kSlotP + quarter * 32 * 8;
                        bulk_copy_s2s(dst + po, stg + po, 32 * 128, pb);
                        bulk_copy_s2s(dst + ao, stg + ao, 32 * 8, pb);
                    }
                }
            }
            if (!run) break;
            float* rl = red + (((g - 1) & 1) * 2) * kHeads;
            named_bar_sync(1 + quarter, 64);  // the pair has read the last tile's maxima
            rl[kh * kHeads + m] = l_part;
            named_bar_sync(1 + quarter, 64);
            const float l_sum = rl[m] + rl[kHeads + m];
            if (ok && kh == 0) {
                if (!whole) {
                    const size_t pslot = (size_t)(grp + seq) * q_len + qi;
                    args.part_lse[pslot * kHeads + m] = !(l_sum <= 0.f) ? m_used - kPShift + log2f(l_sum) : -CUDART_INF_F;
                } else if (args.lse) {
                    args.lse[((size_t)seq * q_len + qi) * kHeads + m] = lse_natural(m_used - kPShift, l_sum);
                }
            }
        }
    } else if (rank == 1 && warp == 1) {
        // ======================================================== accumulator: O issuer
        constexpr uint32_t idO = idesc_f16_f32(kHeads, 256, false, true);
        const uint64_t dP = smem_desc(base + kOffSlots, 16, 1024, kSw128);
        const uint64_t dV = smem_desc(base + kOffV, kVChunk, 1024, kSw128);
        int u = 0;
        for (int seg = 0; ok && it.next(seq, T, k0, k1, whole); ++seg) {
            ok = wait(kOFree, seg + 1);  // the previous piece's O has been read
            const int u0 = u, u1 = u + 2 * (k1 - k0);
#pragma unroll 1
            for (; u < u1 && ok; ++u) {
                const int slot = u % kSlots, st = u % kVStages;
                if (!wait_peer(kPFull + slot, u / kSlots) || !wait(kRescaled + slot, u / kSlots) || !wait(kVFull + st, u / kVStages) ||
                    *abort_flag) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t a0 = dP + ((slot * kSlotBytes) >> 4);
                    const uint64_t b0 = dV + ((st * kVBytes) >> 4);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf)
                            mma_f16_ss(tmem + 256 * hf, a0 + ((32 * k) >> 4), b0 + ((4 * kVChunk * hf + 2048 * k) >> 4), idO,
                                       (u > u0 || k > 0) ? 1u : 0u);
                    mma_commit(bar(kPDone + slot));
                    mma_commit(bar(kVEmpty + st));
                    if (u == u1 - 1) mma_commit(bar(kOFull));
                }
                __syncwarp();
            }
        }
    } else if (rank == 1 && ((warp >= 6 && warp <= 9) || (warp >= 16 && warp <= 19))) {
        // ======================================================== accumulator: unpacking warps
        // Eight warps: 32 of the unit's 64 rows, a row a lane, and 128 of its latents each.
        const int w8 = warp < 10 ? warp - 6 : warp - 12, part = w8 >> 1;
        const int row = 32 * (w8 & 1) + lane;
        int u = 0;
        while (ok && it.next(seq, T, k0, k1, whole)) {
            const int u1 = u + 2 * (k1 - k0);
#pragma unroll 1
            for (; u < u1; ++u) {
                const int st = u % kARawStages, vs = u % kVStages;
                if (!wait(kARawFull + st, u / kARawStages) || *abort_flag) { ok = false; break; }
                const uint32_t src = base + st * kARawBytes + row * kRawRow;
                RawChunk raw;
                raw.load(src, 2 * part);
                if (!wait(kVEmpty + vs, u / kVStages + 1)) { ok = false; break; }
                const uint32_t dst = base + kOffV + vs * kVBytes + 2 * part * kVChunk + sw128(row, 0);
                raw.unpack<true>(dst);
                raw.load(src, 2 * part + 1);
                raw.unpack<true>(dst + kVChunk);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(kARawEmpty + st));
                    mbar_arrive(bar(kVFull + vs));
                }
            }
        }
    } else if (rank == 1 && warp == 10) {
        // ======================================================== accumulator: slot forwarder
        // Arms each P slot for the unit to come, then tells the scorer that it is free.
        Pieces all = it;
        int n_units = 0;
        while (all.next(seq, T, k0, k1, whole)) n_units += 2 * (k1 - k0);
        const uint32_t slotfree_peer = mapa(bar(kSlotFree), peer);
        if (lane == 0)
            for (int s = 0; s < kSlots && s < n_units; ++s) mbar_arrive_expect_tx(bar(kPFull + s), kSlotBytes);
#pragma unroll 1
        for (int u = 0; u + kSlots < n_units; ++u) {
            const int slot = u % kSlots;
            if (!wait(kPDone + slot, u / kSlots) || *abort_flag) { ok = false; break; }
            if (lane == 0) {
                mbar_arrive_expect_tx(bar(kPFull + slot), kSlotBytes);
                mbar_arrive_remote_relaxed(slotfree_peer + 8 * slot);
            }
        }
    } else if (rank == 1 && warp == 11) {
        // ======================================================== accumulator: what the merge has to know
        if (qi == 0) {
            int4 last = make_int4(-1, 0, 0, 0);
            while (it.next(seq, T, k0, k1, whole)) {
                if (k0 > 0) continue;
                last = make_int4(whole ? -1 : seq, grp, (it.pre - 1) / s_share.L, 0);
                if (args.cuts_by_seq && lane == 0) args.cuts[seq] = last;
            }
            if (!args.cuts_by_seq && lane == 0) args.cuts[grp] = last;
        }
    } else if (rank == 1 && softmax_warp) {
        // ======================================================== accumulator: rescale / epilogue warps
        // (volatile: read once and here, as the slot is written anew once the warps have arrived)
        const volatile float* slots = reinterpret_cast<const volatile float*>(base_ptr + kOffSlots);
        const uint32_t o_addr = tmem + lane_addr + 256 * kh;
        int u = 0;
        for (int seg = 0; ok && it.next(seq, T, k0, k1, whole); ++seg) {
            float l_sum = 0.f;
            const int u0 = u, u1 = u + 2 * (k1 - k0);
#pragma unroll 1
            for (; u < u1; ++u) {
                const int slot = u % kSlots;
                if (!wait_peer(kPFull + slot, u / kSlots) || *abort_flag) { ok = false; break; }
                const volatile float* rowdat = slots + (slot * kSlotBytes + kSlotP) / 4 + 2 * m;
                const float f = rowdat[0], l_part = rowdat[1];
                l_sum = ((u - u0) & 1) ? l_sum + l_part : l_part;
                // (the vote has both values, so that neither load is under way when the slot is given back; a sum is never negative)
                const bool scaled = __any_sync(0xffffffffu, f != 1.0f || l_part < 0.f);
                if (u > u0 && scaled) {
                    // O must hold everything before this unit when it is rescaled.  (The
                    // phases of this barrier that were not waited for are complete: P of
                    // unit u lands once the products of unit u - kSlots have returned its
                    // slot, and commits complete in order, so unit u - 1 - kSlots is done.)
                    if (!wait(kPDone + (u - 1) % kSlots, (u - 1) / kSlots)) { ok = false; break; }
                    tc_fence_after();
#pragma unroll 1
                    for (int c0 = 0; c0 < 256; c0 += 32) {
                        uint32_t v[32];
                        tmem_ld32(o_addr + c0, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * f);
                        tmem_st32(o_addr + c0, v);
                    }
                    tmem_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kRescaled + slot));
            }
            if (!ok || !wait(kOFull, seg)) { ok = false; break; }
            tc_fence_after();
            const float inv = l_sum > 0.f ? 1.f / l_sum : 0.f;
            const size_t pslot = (size_t)(grp + seq) * q_len + qi;
            __nv_bfloat16* o_dst = args.o_lat + (((size_t)seq * q_len + qi) * kHeads + m) * kLat + 256 * kh;
            float* p_dst = args.part_o + ((pslot * (kLat / 8) + 32 * kh) * kHeads + m) * 8;
#pragma unroll 1
            for (int c0 = 0; c0 < 256; c0 += 16) {
                uint32_t v[16];
                tmem_ld16(o_addr + c0, v);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * inv);
                if (whole) {
                    uint32_t o[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q) o[q] = pack_bf16(__uint_as_float(v[2 * q]), __uint_as_float(v[2 * q + 1]));
                    if (args.o_lat_v8) {
                        st_global_v8(o_dst + c0, o[0], o[1], o[2], o[3], o[4], o[5], o[6], o[7]);
                    } else {
                        *reinterpret_cast<uint4*>(o_dst + c0) = make_uint4(o[0], o[1], o[2], o[3]);
                        *reinterpret_cast<uint4*>(o_dst + c0 + 8) = make_uint4(o[4], o[5], o[6], o[7]);
                    }
                } else {
                    // column octets, as in mla_attend_kernel
#pragma unroll
                    for (int j = 0; j < 16; j += 8)
                        st_global_v8(p_dst + (size_t)((c0 + j) / 8) * kHeads * 8, v[j], v[j + 1], v[j + 2], v[j + 3], v[j + 4],
                                     v[j + 5], v[j + 6], v[j + 7]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kOFree));
        }
    }
    if (!ok) *abort_flag = 1;

    // ---- teardown, as in mla_attend_kernel: nothing this CTA issued may still run when it exits
    __syncthreads();
    const bool aborted = *abort_flag != 0;
    if (aborted && active && n_load > 0) {  // loads in flight (every lane of a producer warp counted them)
        if (warp == 0) {
            const int full = rank == 0 ? (int)kRawFull : (int)kARawFull;
            for (int n = n_load > kRawStages ? n_load - kRawStages : 0; n < n_load; ++n)
                mbar_wait(bar(full + n % kRawStages), (n / kRawStages) & 1, lim);
        } else {
            mbar_wait(bar(kRopeFull), (n_load - 1) & 1, lim);
        }
    }
    if (warp == 1 && elect_one()) mma_commit(bar(kDrain));  // (a commit covers the products of the thread that makes it)
    if (warp == 1) mbar_wait(bar(kDrain), 0, lim);
    if (aborted && threadIdx.x == 0) atomicOr(args.status, MLA_STATUS_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, kTmemCols);
    cluster_sync();
    const bool peer_aborted = ld_shared_cluster_u32(mapa(abort_addr, peer)) != 0;
    cluster_sync();
    if (aborted || peer_aborted) spin_ns(20000);
}

// The merge of sequences that were cut: o = sum_p 2^(lse_p - m) o_p / sum_p 2^(lse_p - m).
// The group that holds a cut sequence's first part has left its number and the
// last group of it.  A CTA merges kHeadsPer heads of one query token, kWays
// warps a head: each takes every kWays-th piece, a whole row of 512 columns at
// a time (four independent loads a lane), and the warps' states meet in shared
// memory.  16 warps for one head where there are few tokens (32 pieces of one
// sequence in two rounds; eight heads a CTA and one warp a head: 18 us), two
// for each of eight heads where there are many, most of them in few pieces.
struct MergeArgs {
    const int4* cuts;
    int q_len;
    const float* part_o;
    const float* part_lse;
    __nv_bfloat16* o_lat;
    float* lse;
};

template <int kHeadsPer, int kWays>
__global__ void __launch_bounds__(kHeadsPer * kWays * 32) packed_merge_kernel(MergeArgs a) {
    __shared__ float s_m[kHeadsPer * kWays], s_w[kHeadsPer * kWays];
    __shared__ float4 s_acc[kHeadsPer][kWays - 1][kLat / 4];
    const int blk = blockIdx.x / (kHeads / kHeadsPer);
    const int qi = blk % a.q_len;
    pdl_wait();
    pdl_trigger();
    const int4 cut = a.cuts[blk / a.q_len];
    if (cut.x < 0) return;
    const int p_lo = cut.y, p_hi = cut.z;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int hh = warp / kWays, way = warp % kWays;
    const int h = (blockIdx.x % (kHeads / kHeadsPer)) * kHeadsPer + hh;
    const size_t tok = (size_t)cut.x * a.q_len + qi;  // piece p is in slot p q_len + tok
    MergeState st;
    st.clear();
#pragma unroll 1
    for (int p = p_lo + way; p <= p_hi; p += kWays) {
        const size_t slot = tok + (size_t)p * a.q_len;
        // columns 4q..4q+3, q = lane + 32 j: octet q / 2, half q % 2
        const float4* src = reinterpret_cast<const float4*>(a.part_o) + (slot * (kLat / 8) * kHeads + h) * 2;
        float4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int q = lane + 32 * j;
            v[j] = __ldg(src + (size_t)(q / 2) * kHeads * 2 + (q % 2));
        }
        const float z = __ldg(a.part_lse + slot * kHeads + h);
        st.fold(z, z == -CUDART_INF_F ? 0.f : 1.f, v);
    }
    if (way > 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) s_acc[hh][way - 1][lane + 32 * j] = st.acc[j];
        if (lane == 0) {
            s_m[warp] = st.m;
            s_w[warp] = st.wsum;
        }
    }
    __syncthreads();
    if (way > 0) return;
#pragma unroll 1
    for (int w = 1; w < kWays; ++w) {
        float4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = s_acc[hh][w - 1][lane + 32 * j];
        st.fold(s_m[warp + w], s_w[warp + w], v);
    }
    if (a.lse && lane == 0) a.lse[tok * kHeads + h] = lse_natural(st.m, st.wsum);
    st.normalise();
    uint2* dst = reinterpret_cast<uint2*>(a.o_lat + (tok * kHeads + h) * kLat) + lane;
#pragma unroll
    for (int j = 0; j < 4; ++j) dst[32 * j] = make_uint2(pack_bf16(st.acc[j].x, st.acc[j].y), pack_bf16(st.acc[j].z, st.acc[j].w));
}

}  // namespace pk
}  // namespace sm100
}  // namespace mla
