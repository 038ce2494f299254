// Accumulated attention weights on tcgen05 / TMEM:
//   w_t = sum over queries i and heads h of exp(scale * q_hat_ih . row_t - lse_ih)
// for every cached row t of a sequence, added to decay * prev_t.
//
// The rows are the M dimension here: S^T = rows . Q-hat^T has one row of the
// cache in each TMEM lane and the 128 heads in its columns, so a thread sums
// the weights of its own row and nothing is exchanged between lanes, and the
// result needs no atomics.  Q-hat of one query token (144 KB) stays in shared
// memory as the B operand; the rows stream past it:
//   full-width rows: TMA fills a ring of 128 x 64 chunks, the A operand;
//   packed rows: TMA brings the raw rows, eight warps unpack them to bf16 and
//     store them straight into TMEM, from where the products read their A
//     operand (eight chunks of 32 columns: one tile), so unpacked rows cost no
//     shared-memory bandwidth; the keys are a shared-memory A operand.
// Bound: 128 flop a byte for full-width rows: HBM (3.3 us a 128-row tile and
// SM against 1.4 us of products); 354 for packed rows: the tensor cores.
//
// Split.  The tiles of all sequences are cut into equal ranges, one CTA an SM;
// a tile is one CTA's for all queries, so a row's sum is formed in one order and
// needs no atomics.  With several queries a CTA goes through its range in blocks of
// up to eight tiles, query by query, so that the rows' second and later readings
// come from L2; the sums of a block wait in shared memory.  Two sets of four
// warps take alternate tiles of a block.
// Where there are fewer tiles than SMs a query after the other would leave most
// of the SMs idle: there a cluster of CTAs (args.ranks) has a range of at most
// eight tiles, each CTA takes some of the queries, and at the end the CTAs' sums
// are added up through distributed shared memory, in the order of their ranks.
//
// Measured (B200, bursts of twenty calls, and in brackets calls in a row for
// seconds, at the power limit): 1 x 4096 full-width rows 11 us (two thirds of it
// the launch, Q-hat's load and the end); 8 x 65536..131072 rows 169 (189) us, 5.8
// (5.1) TB/s, 0.88 (0.79) of the copy's bandwidth; 64 x 2048..16384 packed rows
// with two queries 156 (184) us, 0.67 (0.57) of the products' rate.
//
// Every wait is bounded; no warp waits on a barrier without a limit before
// the common end, so a wait that expires ends the kernel in order.
#pragma once

#include <cuda_bf16.h>
#include <math_constants.h>

#include "sm100_attend.cuh"
#include "sm100_pieces.cuh"
#include "sm100_unpack.cuh"

namespace mla {
namespace sm100 {
namespace wt {

constexpr int kTile = 128;                // rows of a tile
constexpr int kUnit = 64;                 // rows of a raw copy
constexpr int kChunkBytes = kTile * 128;  // 128 rows x 64 bf16, SW128
constexpr int kQChunks = 9;
constexpr int kBlock = 8;                 // most tiles of a block when there are several queries
constexpr int kRawRow = kPackNib + kPackScale;
constexpr int kRawBytes = kUnit * kRawRow;  // 18 KB: 64 raw rows
constexpr int kSetWarps = 4;

template <bool kPacked>
struct Cfg {
    static constexpr int kThreads = kPacked ? 640 : 384;
    static constexpr int kRing = kPacked ? 8 : 4;  // chunks: TMEM columns / shared memory
    static constexpr int kRawStages = 3;
    // Blocks where a CTA has more than one: those of all CTAs have to stay in L2
    // until the last query has read them.  Eight tiles of full-width rows on every
    // SM are 175 MB: 9 x 56330 rows with two queries 199 us, in blocks of two 177
    // (four 184, one 215); of packed rows, 63 MB, no difference.
    static constexpr int kLongBlock = kPacked ? kBlock : 2;
    static constexpr int kOffRing = kQChunks * kChunkBytes;
    // packed: the keys' chunk, then the raw stages; full width: the ring
    static constexpr int kOffRaw = kOffRing + kChunkBytes;
    static constexpr int kOffSums = kPacked ? kOffRaw + kRawStages * kRawBytes : kOffRing + kRing * kChunkBytes;
    static constexpr int kOffLse = kOffSums + kBlock * kTile * 4;   // [8 warps][128]
    static constexpr int kOffBars = kOffLse + 2 * kSetWarps * kHeads * 4;
    static constexpr int kSmem = kOffBars + 512 + 1024;
    static_assert(kSmem <= 232448, "shared memory exceeds 227 KB");
    static_assert(kOffRaw % 1024 == 0, "alignment");
    // barriers
    enum {
        kQFull = 0,                    // Q-hat chunk loaded (tx)
        kQEmpty = kQFull + kQChunks,   // Q-hat chunk of the previous query multiplied (MMA commit)
        kChFull = kQEmpty + kQChunks,  // ring chunk in place (tx, or 4 warps)
        kChEmpty = kChFull + kRing,    // ring chunk multiplied (MMA commit)
        kSFull = kChEmpty + kRing,     // S of a set complete (MMA commit)
        kSFree = kSFull + 2,           // S of a set read (4 warps)
        kRawFull = kSFree + 2,         // raw rows loaded (tx)
        kRawEmpty = kRawFull + kRawStages,  // raw rows unpacked (8 warps)
        kKeyFull = kRawEmpty + kRawStages,  // keys loaded (tx)
        kKeyEmpty,                          // keys multiplied (MMA commit)
        kDrain,
        kBars
    };
    static_assert(8 * (kBars + 2) <= 480, "barrier block too small");
};
constexpr int kTmemS = 0;       // two buffers of 128 fp32 columns
constexpr int kTmemRing = 256;  // packed: eight chunks of 32 columns

struct Args {
    const int32_t* seqlens;
    const float* lse;   // [B][q_len][128]
    const float* prev;  // or NULL
    float* weights;
    int64_t stride_w;
    float decay, scale_log2;
    int B, q_len, T_max;
    int ranks;          // CTAs of a cluster that share the queries (1: no cluster)
    int* status;
    uint64_t wait_limit_ns;
    int withhold_tile;  // test hook (>= 0): the loader stops before this 64-row tile (see mla.h)
};

// mapQ: Q-hat [tokens][128 heads][576], box 64 x 128 x 1, SW128.
// full width: mapRows [B][T_max][576], box 64 x 128 rows, SW128 (mapKey unused);
// packed: mapRows the codes and scales [B][T_max][144 words], box 144 x 64 rows; mapKey the keys, box 64 x 64 rows, SW128.
template <bool kPacked>
__global__ void __launch_bounds__(Cfg<kPacked>::kThreads, 1)
    weights_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapRows,
                   const __grid_constant__ CUtensorMap mapKey, Args args) {
    using C = Cfg<kPacked>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int s_scratch[64];
    __shared__ PieceShare s_share;
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* base_ptr = smem_raw + (base - raw);
    auto bar = [&](int i) { return base + C::kOffBars + 8u * i; };
    volatile int* abort_flag = reinterpret_cast<volatile int*>(base_ptr + C::kOffBars + 8 * (C::kBars + 1));
    const uint64_t lim = args.wait_limit_ns;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int q_len = args.q_len;
    const int ranks = args.ranks, group = blockIdx.x / ranks, rank = blockIdx.x % ranks;

    if (threadIdx.x == 0) {
        auto init = [&](int first, int n, int count) {
            for (int i = 0; i < n; ++i) mbar_init(bar(first + i), count);
        };
        init(C::kQFull, kQChunks, 1);
        init(C::kQEmpty, kQChunks, 1);
        init(C::kChFull, C::kRing, kPacked ? 4 : 1);
        init(C::kChEmpty, C::kRing, 1);
        init(C::kSFull, 2, 1);
        init(C::kSFree, 2, kSetWarps);
        init(C::kRawFull, C::kRawStages, 1);
        init(C::kRawEmpty, C::kRawStages, 8);
        init(C::kKeyFull, 1, 1);
        init(C::kKeyEmpty, 1, 1);
        init(C::kDrain, 1, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tensormap(&mapQ);
        prefetch_tensormap(&mapRows);
        if (kPacked) prefetch_tensormap(&mapKey);
    }
    if (warp == 1) {
        tmem_alloc(bar(C::kBars), kTmemCols);
        tmem_relinquish();
    }
    pdl_wait();
    const Batch batch = {args.seqlens, args.B, q_len, args.T_max, kTile, 1};
    plan_share(batch, gridDim.x / ranks, group, 1, false, s_scratch, &s_share);
    Pieces it(&s_share);
    for (int b = blockIdx.x + gridDim.x * threadIdx.x; b < args.B; b += gridDim.x * blockDim.x)
        if (!batch.valid(batch.len(b))) atomicOr(args.status, MLA_STATUS_BAD_SEQLEN);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(base_ptr + C::kOffBars + 8 * C::kBars);
    auto wait = [&](int i, int phase) { return warp_wait_fast<false>(bar(i), phase & 1, lim); };

    bool ok = true, whole = false;
    int seq = 0, T = 0, k0 = 0, k1 = 0;
    int n_load = 0, n_pass = 0;  // loads and passes (query tokens of a block) begun
    int n_done = 0;              // tiles of the pieces before
    // Every role walks the same passes: tiles j0..j1-1 of a sequence against one of its query tokens.
    auto walk = [&](auto&& pass) {
        while (ok && it.next(seq, T, k0, k1, whole)) {
            const int step = q_len == 1 ? k1 - k0 : (s_share.L > kBlock ? C::kLongBlock : kBlock);
            for (int j0 = k0; j0 < k1 && ok; j0 += step) {
                const int j1 = j0 + step < k1 ? j0 + step : k1;
                for (int i = rank; i < q_len && ok; i += ranks, ++n_pass) ok = pass(j0, j1, i) && !*abort_flag;
            }
            n_done += k1 - k0;
        }
    };

    if (warp == 0) {
        // ======================================================== producer of rows
        walk([&](int j0, int j1, int) {
            if constexpr (kPacked) {
#pragma unroll 1
                for (int t = 2 * j0; t < 2 * j1; ++t, ++n_load) {
                    if (args.withhold_tile >= 0 && n_load >= args.withhold_tile) return true;
                    const int st = n_load % C::kRawStages;
                    if (!wait(C::kRawEmpty + st, n_load / C::kRawStages + 1)) return false;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(bar(C::kRawFull + st), kRawBytes);
                        tma_load_3d(base + C::kOffRaw + st * kRawBytes, &mapRows, bar(C::kRawFull + st), 0, t * kUnit, seq);
                    }
                    __syncwarp();
                }
            } else {
#pragma unroll 1
                for (int t = j0; t < j1; ++t)
#pragma unroll 1
                    for (int c = 0; c < kQChunks; ++c, ++n_load) {
                        if (args.withhold_tile >= 0 && n_load / kQChunks * 2 + 1 >= args.withhold_tile) return true;
                        const int st = n_load % C::kRing;
                        if (!wait(C::kChEmpty + st, n_load / C::kRing + 1)) return false;
                        if (lane == 0) {
                            mbar_arrive_expect_tx(bar(C::kChFull + st), kChunkBytes);
                            tma_load_3d(base + C::kOffRing + st * kChunkBytes, &mapRows, bar(C::kChFull + st), 64 * c, t * kTile, seq);
                        }
                        __syncwarp();
                    }
            }
            return true;
        });
    } else if (warp == 2) {
        // ======================================================== producer of Q-hat, chunk by chunk behind the last products of the pass before
        walk([&](int, int, int i) {
#pragma unroll 1
            for (int c = 0; c < kQChunks; ++c, ++n_load) {
                if (!wait(C::kQEmpty + c, n_pass + 1)) return false;
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar(C::kQFull + c), kChunkBytes);
                    tma_load_3d(base + c * kChunkBytes, &mapQ, bar(C::kQFull + c), 64 * c, 0, seq * q_len + i);
                }
                __syncwarp();
            }
            return true;
        });
    } else if (kPacked && warp == 3) {
        // ======================================================== producer of keys
        walk([&](int j0, int j1, int) {
#pragma unroll 1
            for (int t = j0; t < j1; ++t, ++n_load) {
                if (!wait(C::kKeyEmpty, n_load + 1)) return false;
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar(C::kKeyFull), kChunkBytes);
                    for (int r = 0; r < 2; ++r)
                        tma_load_3d(base + C::kOffRing + r * kUnit * 128, &mapKey, bar(C::kKeyFull), 0, t * kTile + r * kUnit, seq);
                }
                __syncwarp();
            }
            return true;
        });
    } else if (warp == 1) {
        // ======================================================== MMA issuer: S^T (128 rows x 128 heads) of tile after tile
        constexpr uint32_t idS = idesc_bf16_f32(kTile, kHeads, false, false);
        const uint64_t dQ = smem_desc(base, 16, 1024, kSw128);
        const uint64_t dRing = smem_desc(base + C::kOffRing, 16, 1024, kSw128);
        int used[2] = {0, 0};  // tiles each set has been given
        int n = 0;             // full width: ring chunks multiplied; packed: tiles
        walk([&](int j0, int j1, int) {
#pragma unroll 1
            for (int t = j0; t < j1; ++t) {
                const int set = (t - j0) & 1;
                const int uses = set ? used[1]++ : used[0]++;
                if (!wait(C::kSFree + set, uses + 1)) return false;
                const uint32_t dS = tmem + kTmemS + kHeads * set;
                if constexpr (kPacked) {
                    // The unpacking warps are up to a tile ahead, so this warp's own
                    // latency is what a tile takes: a wait for every chunk, with its
                    // 160 cycles, and a rolled loop made 530 cycles a chunk of the 256
                    // that its products need.  So lane c looks at chunk c's barriers, all
                    // in one test, and the chunks found in place are issued without more.
                    // A chunk that was not is waited for.
                    uint32_t ready = 0;
#pragma unroll
                    for (int c = 0; c < kQChunks; ++c) {
                        const bool key = c == 8;
                        if (!(ready >> c & 1u)) {
                            bool there = false;
                            if (lane < kQChunks) {
                                there = mbar_test(bar(lane == 8 ? (int)C::kKeyFull : (int)C::kChFull + lane), n & 1);
                                if (t == j0) there = there && mbar_test(bar(C::kQFull + lane), n_pass & 1);
                            }
                            ready = __ballot_sync(0xffffffffu, there);
                            if (!(ready >> c & 1u)) {
                                if (t == j0 && !wait(C::kQFull + c, n_pass)) return false;
                                if (!wait(key ? (int)C::kKeyFull : (int)C::kChFull + c, n)) return false;
                                ready |= 1u << c;
                            }
                            __syncwarp();
                            tc_fence_after();
                        }
                        if (elect_one()) {
                            const uint64_t dB = dQ + ((c * kChunkBytes) >> 4);
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                if (key) mma_f16_ss(dS, dRing + ((32 * k) >> 4), dB + ((32 * k) >> 4), idS, 1u);
                                else mma_f16_ts(dS, tmem + kTmemRing + 32 * c + 8 * k, dB + ((32 * k) >> 4), idS, (c | k) ? 1u : 0u);
                            }
                            mma_commit(key ? bar(C::kKeyEmpty) : bar(C::kChEmpty + c));
                            if (t == j1 - 1) mma_commit(bar(C::kQEmpty + c));
                            if (key) mma_commit(bar(C::kSFull + set));
                        }
                        __syncwarp();
                    }
                    ++n;
                } else {
#pragma unroll 1
                    for (int c = 0; c < kQChunks; ++c, ++n) {
                        if (t == j0 && !wait(C::kQFull + c, n_pass)) return false;
                        const int st = n % C::kRing;
                        if (!wait(C::kChFull + st, n / C::kRing)) return false;
                        tc_fence_after();
                        if (elect_one()) {
                            const uint64_t dA = dRing + ((st * kChunkBytes) >> 4), dB = dQ + ((c * kChunkBytes) >> 4);
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                mma_f16_ss(dS, dA + ((32 * k) >> 4), dB + ((32 * k) >> 4), idS, (c | k) ? 1u : 0u);
                            mma_commit(bar(C::kChEmpty + st));
                            if (t == j1 - 1) mma_commit(bar(C::kQEmpty + c));
                            if (c == kQChunks - 1) mma_commit(bar(C::kSFull + set));
                        }
                        __syncwarp();
                    }
                }
            }
            return true;
        });
    } else if (kPacked && warp >= 12) {
        // ======================================================== unpacking warps: a row a lane, into the row's own TMEM lane
        // Warps 12-15 take the even chunks, 16-19 the odd ones.
        const int quarter = warp & 3, odd = warp >= 16 ? 1 : 0, hi = quarter >> 1;
        const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
        const uint32_t never = (uint32_t)(q_len >> 31);  // 0, which the compiler does not know
        int n = 0;  // tiles
        walk([&](int j0, int j1, int) {
#pragma unroll 1
            for (int t = j0; t < j1; ++t, ++n) {
                // Every warp waits for both halves of the tile and returns both, though
                // it reads one: a barrier's parity only tells its phases apart to who
                // has seen the one before.  It returns them as soon as its codes are in
                // registers: held until the last chunk was unpacked, they left room for
                // half a tile ahead.
                const int st0 = 2 * n % C::kRawStages, st1 = (2 * n + 1) % C::kRawStages;
                if (!wait(C::kRawFull + st0, 2 * n / C::kRawStages) || !wait(C::kRawFull + st1, (2 * n + 1) / C::kRawStages))
                    return false;
                const uint32_t src = base + C::kOffRaw + (hi ? st1 : st0) * kRawBytes + (32 * (quarter & 1) + lane) * kRawRow;
                RawChunk r[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) r[k].load_once(src, odd + 2 * k);
                // An arrival overtakes loads that are still queued, and the next rows would
                // land under them: the vote has a word of every load, so it waits for all.
                uint32_t some = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k) some |= r[k].scales | r[k].w[0] | r[k].w[4];
                if (!__any_sync(0xffffffffu, (some & never) != 0) && lane == 0) {
                    mbar_arrive(bar(C::kRawEmpty + st0));
                    mbar_arrive(bar(C::kRawEmpty + st1));
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int c = odd + 2 * k;
                    if (!wait(C::kChEmpty + c, n + 1)) return false;
                    tc_fence_after();
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t v[16];
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            uint32_t x[8];
                            unpack16<false>(r[k].w[4 * h + 2 * g], r[k].w[4 * h + 2 * g + 1], (r[k].scales >> (16 * h + 8 * g)) & 0xFFu, x);
#pragma unroll
                            for (int j = 0; j < 8; ++j) v[8 * g + j] = x[j];
                        }
                        tmem_st16(tmem + lane_addr + kTmemRing + 32 * c + 16 * h, v);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(C::kChFull + c));
                }
            }
            return true;
        });
    } else if (warp >= 4 && warp < 12) {
        // ======================================================== weights: lane = row of the tile; set 0 (warps 4-7) the even tiles of a block
        const int set = warp >= 8 ? 1 : 0, quarter = warp & 3, row = quarter * 32 + lane;
        float* nlse = reinterpret_cast<float*>(base_ptr + C::kOffLse) + (warp - 4) * kHeads;
        float* sums = reinterpret_cast<float*>(base_ptr + C::kOffSums);
        const uint32_t nl_addr = smem_u32(nlse);
        const uint32_t s_addr = tmem + ((uint32_t)(quarter * 32) << 16) + kTmemS + kHeads * set;
        const uint64_t sl2x2 = pack_f32x2(args.scale_log2, args.scale_log2);
        int n = 0;  // tiles of this set
        walk([&](int j0, int j1, int i) {
            __syncwarp();
            bool uncounted = false;
            for (int h = lane; h < kHeads; h += 32) {
                const float z = args.lse[((size_t)seq * q_len + i) * kHeads + h];
                nlse[h] = z == -CUDART_INF_F ? -CUDART_INF_F : z * -1.4426950408889634f;
                uncounted |= z == -CUDART_INF_F;
            }
            uncounted = __any_sync(0xffffffffu, uncounted);
            __syncwarp();
#pragma unroll 1
            for (int t = j0 + set; t < j1; t += 2, ++n) {
                if (!wait(C::kSFull + set, n)) return false;
                tc_fence_after();
                uint64_t w2 = 0;
#pragma unroll 1
                for (int h = 0; h < kHeads; h += 16) {
                    uint32_t v[16];
                    tmem_ld16(s_addr + h, v);
                    tmem_wait_ld();
                    if (uncounted) {  // whatever such a query's score is, infinite or NaN
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (ld_shared_u32(nl_addr + 4 * (h + j)) == 0xFF800000u) v[j] = 0u;
                    }
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        uint32_t z[4];
                        ld_shared_v4u(nl_addr + 4 * (h + j), z[0], z[1], z[2], z[3]);
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {  // (two values an instruction where there is one for it)
                            float p0, p1;
                            unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(v[j + e]), __uint_as_float(v[j + e + 1])), sl2x2,
                                                   pack_f32x2(__uint_as_float(z[e]), __uint_as_float(z[e + 1]))),
                                         p0, p1);
                            w2 = add_f32x2(w2, pack_f32x2(ex2(p0), ex2(p1)));
                        }
                    }
                }
                float w0, w1;
                unpack_f32x2(w2, w0, w1);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::kSFree + set));
                // query i sees rows 0..T-q_len+i; what a row past it holds reached only its own lane
                const int r = t * kTile + row;
                float w = r < T - q_len + 1 + i ? w0 + w1 : 0.f;
                if (q_len > 1) {  // (a cluster's range fits the block: every tile has a place of its own)
                    float* s = sums + ((ranks > 1 ? n_done : 0) + t - j0) * kTile + row;
                    if (i > rank) w += *s;
                    *s = w;
                }
                if (ranks == 1 && i == q_len - 1 && r < T) {
                    const size_t at = (size_t)seq * args.stride_w + r;
                    args.weights[at] = args.prev ? fmaf(args.decay, args.prev[at], w) : w;
                }
            }
            return true;
        });
    }
    if (!ok) *abort_flag = 1;

    // ---- teardown: nothing this CTA issued may still run when it exits
    __syncthreads();
    pdl_trigger();
    const bool aborted = *abort_flag != 0;
    if (aborted && n_load > 0) {  // loads in flight (a producer warp's count; zero in the other roles)
        const int first = warp == 0 ? (kPacked ? (int)C::kRawFull : (int)C::kChFull) : (warp == 2 ? (int)C::kQFull : (int)C::kKeyFull);
        const int nst = warp == 0 ? (kPacked ? C::kRawStages : C::kRing) : (warp == 2 ? kQChunks : 1);
        for (int x = n_load > nst ? n_load - nst : 0; x < n_load; ++x) mbar_wait(bar(first + x % nst), (x / nst) & 1, lim);
    }
    if (warp == 1 && elect_one()) mma_commit(bar(C::kDrain));  // (a commit covers the products of the thread that makes it)
    if (warp == 1) mbar_wait(bar(C::kDrain), 0, lim);
    if (aborted && threadIdx.x == 0) atomicOr(args.status, MLA_STATUS_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, kTmemCols);
    if (ranks == 1) return;

    // ---- the cluster's sums: CTA k adds up tiles k, k + ranks, ...
    cluster_sync();
    bool any_aborted = false;
    for (int k = 0; k < ranks; ++k) any_aborted |= ld_shared_cluster_u32(mapa(bar(C::kBars + 1), k)) != 0;
    Pieces fin(&s_share);
    int n = 0;
    while (!any_aborted && fin.next(seq, T, k0, k1, whole)) {
        for (int t = k0; t < k1; ++t, ++n) {
            const int r = t * kTile + (int)threadIdx.x;
            if (n % ranks != rank || threadIdx.x >= kTile || r >= T) continue;
            const uint32_t place = base + C::kOffSums + (n * kTile + threadIdx.x) * 4;
            float w = 0.f;
            for (int k = 0; k < ranks; ++k) w += __uint_as_float(ld_shared_cluster_u32(mapa(place, k)));
            const size_t at = (size_t)seq * args.stride_w + r;
            args.weights[at] = args.prev ? fmaf(args.decay, args.prev[at], w) : w;
        }
    }
    __syncthreads();
    cluster_sync();  // (no CTA's shared memory is read after this)
}

}  // namespace wt
}  // namespace sm100
}  // namespace mla
