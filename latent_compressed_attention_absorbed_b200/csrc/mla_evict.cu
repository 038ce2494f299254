// Eviction from a cache by accumulated attention weight: which rows of every
// sequence stay, and the compaction of the cache to those rows.
//
// Of a sequence of T rows that is over the budget, the first n_sink rows, the
// last n_recent rows and the m = budget - n_sink - n_recent rows of the middle
// with the largest weights stay, in their order.  Equal weights: the lower
// row; -0 equals 0, a NaN counts as less than every number.
//
// evict_select_kernel: a cluster of CTAs per sequence finds the last weight
// that stays by a radix search over order-preserving 32-bit keys (up to three
// passes of 11, 11 and 10 bits: each counts the digits of the keys that share
// the prefix found so far, in shared memory, and the CTAs add their counts up
// through distributed shared memory), then lists the kept rows in order with
// one prefix sum.  The first and last rows take part with a key above every
// weight's.  A thread keeps its rows' keys in registers, so the weights are
// read once.
// evict_move_kernel: a CTA moves a chunk of kept rows.  It is bound by HBM:
// every kept row is read once and written once.
// Measured (B200): 1 x 4096 full-width rows to 4000 in 13 us (two launches
// and the passes' meetings), 64 x 1500..8192 to 2048 in 65 us (4.6 TB/s), 8 x
// 131072 to 32768 in 123 us (5.0 TB/s).  In place (single calls, the L2 written
// over between): 23, 92 and 191 us, and of packed rows 23, 51 and 98.
// In place, a kept row never moves to a higher index, and the rows that a
// chunk overwrites are kept rows of its own or of at most two earlier chunks
// (the kept rows inside an index range have consecutive ranks).  So a chunk
// loads its rows into registers, publishes that it has, waits until those
// chunks have, and stores.  Chunks are taken in order from a counter, so the
// chunks waited for are running or done, and every wait is bounded.
#include <cooperative_groups.h>
#include <limits.h>

#include "mla_packed_internal.h"
#include "sm100_host.h"
#include "sm100_ptx.cuh"

namespace mla {
namespace {

namespace cg = cooperative_groups;

constexpr int kSelBins = 2048;
constexpr int kSelRanks = 8;  // CTAs of a cluster
constexpr int kSlab = 16;  // rows a thread of the selection holds
constexpr int kMoveThreads = 256;
constexpr int kMovePieces = 8;  // 16-byte pieces a thread holds: chunks of up to 32 KB

// Larger weight <-> larger key, -0 as 0.  No number maps below 0x007FFFFF or
// above 0xFF800000: a NaN is 1, a row that stays in any case (the first and the
// last ones) kKeySafe, no row 0.
constexpr uint32_t kKeyNaN = 1u, kKeySafe = 0xFFFFFFFFu;
__device__ __forceinline__ uint32_t weight_key(float w) {
    const uint32_t u = __float_as_uint(w + 0.0f);
    const uint32_t k = u ^ (uint32_t)(((int32_t)u >> 31) | 0x80000000);
    return w != w ? kKeyNaN : k;
}

struct EvictScratch {
    int32_t* kept;    // [B][budget] rows kept, ascending
    int32_t* count;   // [B]
    int32_t* loaded;  // [B][chunks]: the chunk's rows are in registers
    int32_t* ticket;
    int chunks, chunk_rows;
};

// Block-wide exclusive prefix of a count (or two packed ones); `total` gets the
// sum.  One barrier; `sums` must not be in use by a scan one barrier ago.
template <int kWarps>
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t* sums, uint64_t& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    const uint64_t mine = lane < kWarps ? sums[lane] : 0;
    uint64_t w = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
    }
    total = __shfl_sync(0xffffffffu, w, 31);
    return __shfl_sync(0xffffffffu, w - mine, warp) + x - v;
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads) evict_select_kernel(EvictArgs a, EvictScratch s) {
    constexpr int kWarps = kThreads / 32, kBins = kSelBins / kThreads;  // bins a thread
    __shared__ __align__(16) int hist[3][kSelBins];  // one for each pass: a pass needs no second meeting to clear it
    __shared__ uint64_t sums[2][32];
    __shared__ uint64_t mine;    // this CTA's counts, read by the others
    __shared__ int found[3][3];  // of each pass: digit, keys above it, keys with it
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int b = blockIdx.x / ranks, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    sm100::pdl_wait();
    sm100::pdl_trigger();
    const int T = a.seqlens[b];
    const bool bad = T < 0 || T > a.T_max;
    if (blockIdx.x == 0 && tid == 0) *s.ticket = 0;
    if (rank == 0)
        for (int c = tid; c < s.chunks; c += kThreads) s.loaded[(size_t)b * s.chunks + c] = 0;
    const int n = bad ? 0 : (T < a.budget ? T : a.budget);
    int32_t* kept = s.kept + (size_t)b * a.budget;
    int32_t* kept_out = a.kept_out ? a.kept_out + (size_t)b * a.budget : nullptr;
    if (bad || T <= a.budget) {  // the same for the whole cluster
        if (bad && rank == 0 && tid == 0) atomicOr(a.status, MLA_STATUS_BAD_SEQLEN);
        for (int j = rank * kThreads + tid; j < a.budget; j += ranks * kThreads) {
            if (j < n) kept[j] = j;
            if (kept_out) kept_out[j] = j < n ? j : -1;
        }
    } else {
        const int lo = a.n_sink, hi = T - a.n_recent;  // the middle
        const float* w = a.weights + (size_t)b * a.stride_w;
        const bool wide = (reinterpret_cast<uintptr_t>(w) & 15) == 0;
        // This CTA's rows, and a slab of their keys in registers: a warp has 32
        // `each` consecutive rows, its lanes four at a time in turn (so that loads
        // and the kept rows' stores stay within a few lines).  One slab holds all
        // of them up to 16 rows a thread, and the weights are read once; beyond
        // that every pass reads them again, from L2.
        const int64_t per = (((int64_t)T + ranks - 1) / ranks + 3) & ~int64_t(3);
        const int64_t t_lo = min((int64_t)T, rank * per), t_hi = min((int64_t)T, t_lo + per);
        const int slabs = (int)((per + kSlab * kThreads - 1) / (kSlab * kThreads));
        const int each = slabs > 1 ? kSlab : (int)((per + 4 * kThreads - 1) / (4 * kThreads)) * 4;
        uint32_t key[kSlab];
        int held = -1;
        auto load_slab = [&](int slab) {
            if (held == slab) return;
            held = slab;
            const int64_t t0 = t_lo + ((int64_t)slab * kWarps + warp) * (32 * each) + 4 * lane;
            float4 f[kSlab / 4];
#pragma unroll
            for (int v = 0; v < kSlab / 4; ++v) {
                const int64_t t = t0 + 128 * v;
                f[v] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (4 * v >= each || t >= t_hi) continue;
                if (wide && t + 4 <= t_hi) {
                    f[v] = *reinterpret_cast<const float4*>(w + t);
                } else {
                    f[v].x = w[t];
                    if (t + 1 < t_hi) f[v].y = w[t + 1];
                    if (t + 2 < t_hi) f[v].z = w[t + 2];
                    if (t + 3 < t_hi) f[v].w = w[t + 3];
                }
            }
#pragma unroll
            for (int v = 0; v < kSlab / 4; ++v) {
                const int64_t t = t0 + 128 * v;
                const float x[4] = {f[v].x, f[v].y, f[v].z, f[v].w};
                const bool inside = 4 * v < each && t >= lo && t + 4 <= hi && t + 4 <= t_hi;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t k = weight_key(x[j]);
                    if (!inside) {
                        if (t + j < lo || t + j >= hi) k = kKeySafe;
                        if (4 * v >= each || t + j >= t_hi) k = 0u;
                    }
                    key[4 * v + j] = k;
                }
            }
        };
        // ---- the key of the budget-th row from above: `last`, of whose equals equal_left stay
        for (int i = tid; i < 3 * kSelBins; i += kThreads) (&hist[0][0])[i] = 0;
        __syncthreads();
        uint32_t last = 0u;
        int need = a.budget;
        int shift = 32;
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int bits = pass < 2 ? 11 : 10;
            const uint32_t above = shift == 32 ? 0u : 0xFFFFFFFFu << shift;
            shift -= bits;
            const uint32_t digits = (1u << bits) - 1;
            for (int slab = 0; slab < slabs; ++slab) {
                load_slab(slab);
#pragma unroll
                for (int i = 0; i < kSlab; ++i)
                    if (i < each && ((key[i] ^ last) & above) == 0) atomicAdd(&hist[pass][(key[i] >> shift) & digits], 1);
            }
            if (ranks > 1) cluster.sync();
            else __syncthreads();
            // kBins bins a thread, from the highest digit down
            int c[kBins];
            const int top = kSelBins - 1 - kBins * tid;
#pragma unroll
            for (int k = 0; k < kBins; ++k) c[k] = 0;
#pragma unroll
            for (int r = 0; r < kSelRanks; ++r) {  // (unrolled, so that the remote reads overlap)
                if (r >= ranks) break;
                const int* other = cluster.map_shared_rank(&hist[pass][0], r) + top - (kBins - 1);
#pragma unroll
                for (int k = 0; k < kBins; k += 2) {
                    const int2 two = *reinterpret_cast<const int2*>(other + kBins - 2 - k);
                    c[k] += two.y;
                    c[k + 1] += two.x;
                }
            }
            int sum = 0;
#pragma unroll
            for (int k = 0; k < kBins; ++k) sum += c[k];
            uint64_t total;
            int before = (int)block_scan<kWarps>(sum, sums[pass & 1], total);
            if (before < need && before + sum >= need) {
#pragma unroll
                for (int k = 0; k < kBins; ++k) {
                    if (before < need && before + c[k] >= need) {
                        found[pass][0] = top - k;
                        found[pass][1] = before;
                        found[pass][2] = c[k];
                    }
                    before += c[k];
                }
            }
            __syncthreads();
            last |= (uint32_t)found[pass][0] << shift;
            need -= found[pass][1];
            if (found[pass][2] == need && last > 0u) {  // all rows with this digit stay: everything from `last` up
                --last;
                need = 0;
                break;
            }
        }
        const int equal_left = need;
        // ---- the kept rows in order.  Counts are pairs: rows above the last key in the low half, rows with it in the high half.
        uint32_t over = 0, equal = 0;  // which of this lane's rows
        auto classify = [&]() {
            over = equal = 0;
#pragma unroll
            for (int i = 0; i < kSlab; ++i) {
                over |= key[i] > last ? 1u << i : 0u;
                equal |= key[i] == last ? 1u << i : 0u;
            }
        };
        auto warp_count = [&]() {  // (a warp's slab has 512 rows)
            const uint32_t c = __reduce_add_sync(0xffffffffu, (uint32_t)(__popc(equal) << 16 | __popc(over)));
            return (uint64_t)(c >> 16) << 32 | (c & 0xFFFFu);
        };
        uint64_t base = 0, total;
        __syncthreads();  // the last pass has read its sums
        if (ranks > 1) {  // what the CTAs before this one keep
            uint64_t own = 0;
            for (int slab = 0; slab < slabs; ++slab) {
                load_slab(slab);
                classify();
                own += warp_count();
            }
            block_scan<kWarps>(lane == 0 ? own : 0, sums[1], total);
            if (tid == 0) mine = total;
            cluster.sync();
#pragma unroll
            for (int r = 0; r < kSelRanks; ++r)
                if (r < rank) base += *cluster.map_shared_rank(&mine, r);
        }
        for (int slab = 0; slab < slabs; ++slab) {
            if (slabs > 1 || ranks == 1) {
                load_slab(slab);
                classify();
            }
            const uint64_t own = warp_count();
            uint64_t at = block_scan<kWarps>(lane == 0 ? own : 0, sums[slab & 1], total);
            at = base + __shfl_sync(0xffffffffu, at, 0);
            base += total;
            if (own == 0) continue;
            const int t0 = (int)(t_lo + ((int64_t)slab * kWarps + warp) * (32 * each) + 4 * lane);
#pragma unroll
            for (int v = 0; v < kSlab / 4; ++v) {
                if (4 * v >= each) break;
                const uint32_t o4 = over >> (4 * v) & 15u, e4 = equal >> (4 * v) & 15u;
                const uint32_t c = __popc(e4) << 16 | __popc(o4);
                uint32_t inc = c;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t up = __shfl_up_sync(0xffffffffu, inc, o);
                    if (lane >= o) inc += up;
                }
                int x = (int)(uint32_t)at + (int)((inc - c) & 0xFFFFu), y = (int)(at >> 32) + (int)((inc - c) >> 16);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bool is_over = o4 >> j & 1, is_equal = e4 >> j & 1;
                    const int slot = x + min(y, equal_left);
                    // (slot < budget holds for weights that nobody changes meanwhile)
                    if ((is_over || (is_equal && y < equal_left)) && slot < a.budget) {
                        kept[slot] = t0 + 128 * v + j;
                        if (kept_out) kept_out[slot] = t0 + 128 * v + j;
                    }
                    x += is_over;
                    y += is_equal;
                }
                const uint32_t all = __shfl_sync(0xffffffffu, inc, 31);
                at += (uint64_t)(all >> 16) << 32 | (all & 0xFFFFu);
            }
        }
    }
    // seqlens_out may be seqlens: every CTA of the cluster has read it by now,
    // and no CTA's shared memory is read after this
    cluster.sync();
    if (rank == 0 && tid == 0) {
        s.count[b] = n;
        a.seqlens_out[b] = n;
    }
}

template <typename U>  // the unit rows are copied in: the widest that divides a row
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(EvictArgs a, EvictScratch s) {
    __shared__ int s_ticket;
    __shared__ int s_wait[2];
    const int tid = threadIdx.x;
    sm100::pdl_wait();
    sm100::pdl_trigger();
    if (tid == 0) s_ticket = a.in_place ? atomicAdd(s.ticket, 1) : (int)blockIdx.x;
    __syncthreads();
    const int b = s_ticket / s.chunks, chunk = s_ticket % s.chunks;
    const int j0 = chunk * s.chunk_rows;
    const int total = s.count[b];
    const int n = total - j0 < s.chunk_rows ? total - j0 : s.chunk_rows;
    int* loaded = s.loaded + (size_t)b * s.chunks;
    if (n <= 0) return;  // no row of this sequence waits for an empty chunk
    const int32_t* kept = s.kept + (size_t)b * a.budget;
    const int units = a.row_bytes / (int)sizeof(U);
    const uint8_t* src = a.src + (int64_t)b * a.src_b;
    uint8_t* dst = a.dst + (int64_t)b * a.dst_b;
    const bool same_rows = a.src == a.dst;  // then the strides are the same too
    const bool same_weights = a.weights == a.weights_out;
    // nothing before the chunk's last row was dropped: in place, nothing moves
    const bool still = kept[j0 + n - 1] == j0 + n - 1;
    const bool move_rows = !(still && same_rows), move_weights = !(still && same_weights);
    U v[kMovePieces];
    float w = 0.f;
    if (move_rows) {
#pragma unroll
        for (int i = 0; i < kMovePieces; ++i) {
            const int e = i * kMoveThreads + tid;
            if (e < n * units) v[i] = reinterpret_cast<const U*>(src + (int64_t)kept[j0 + e / units] * a.src_t)[e % units];
        }
    }
    if (move_weights)
        if (tid < n) w = a.weights[(size_t)b * a.stride_w + kept[j0 + tid]];
    if (a.in_place) {
        // the ranks of the kept rows among those this chunk overwrites
        if (tid < 2) {
            const int edge = tid == 0 ? j0 : j0 + n;
            int lo = 0, hi = total;
            while (lo < hi) {
                const int mid = (lo + hi) / 2;
                if (kept[mid] < edge) lo = mid + 1;
                else hi = mid;
            }
            s_wait[tid] = lo;
        }
        __threadfence();
        __syncthreads();  // every thread's loads are done
        if (tid == 0) {
            if (chunk != a.withhold_chunk) atomicExch(&loaded[chunk], 1);
            const int c0 = s_wait[0] / s.chunk_rows, c1 = (s_wait[1] - 1) / s.chunk_rows;
            bool ok = true;
            for (int c = c0; c <= c1 && c < chunk && s_wait[1] > s_wait[0]; ++c) {
                const uint64_t start = sm100::global_timer_ns();
                while (atomicAdd(&loaded[c], 0) == 0) {
                    if (sm100::global_timer_ns() - start > a.wait_limit_ns) {
                        ok = false;
                        break;
                    }
                }
            }
            __threadfence();
            s_wait[0] = ok;
        }
        __syncthreads();
        if (!s_wait[0]) {
            if (tid == 0) atomicOr(a.status, MLA_STATUS_TIMEOUT);
            return;
        }
    }
    if (move_rows) {
#pragma unroll
        for (int i = 0; i < kMovePieces; ++i) {
            const int e = i * kMoveThreads + tid;
            if (e < n * units) reinterpret_cast<U*>(dst + (int64_t)(j0 + e / units) * a.dst_t)[e % units] = v[i];
        }
    }
    if (move_weights)
        if (tid < n) a.weights_out[(size_t)b * a.stride_w_out + j0 + tid] = w;
}

int unit_bytes(int row_bytes) { return row_bytes % 16 == 0 ? 16 : (row_bytes % 4 == 0 ? 4 : 2); }
int rows_per_chunk(int row_bytes) {
    const int rows = kMoveThreads * kMovePieces / (row_bytes / unit_bytes(row_bytes));
    return rows < 1 ? 1 : (rows > kMoveThreads ? kMoveThreads : rows);
}

size_t evict_layout(int B, int budget, int row_bytes, EvictScratch* s, void* base) {
    Carve c(base);
    s->chunk_rows = rows_per_chunk(row_bytes);
    s->chunks = (budget + s->chunk_rows - 1) / s->chunk_rows;
    s->kept = (int32_t*)c.take((size_t)B * budget * 4);
    s->count = (int32_t*)c.take((size_t)B * 4);
    s->loaded = (int32_t*)c.take((size_t)B * s->chunks * 4);
    s->ticket = (int32_t*)c.take(4);
    return c.off;
}

}  // namespace

size_t evict_workspace(int B, int budget, int row_bytes) {
    EvictScratch s;
    return evict_layout(B, budget, row_bytes, &s, nullptr);
}

cudaError_t evict_launch(const EvictArgs& args, void* workspace, cudaStream_t st) {
    EvictArgs a = args;
    if (a.wait_limit_ns == 0) a.wait_limit_ns = MLA_WAIT_LIMIT_NS;
    EvictScratch s;
    evict_layout(a.B, a.budget, a.row_bytes, &s, workspace);
    const int64_t blocks = (int64_t)a.B * s.chunks;
    if (blocks > INT_MAX) return cudaErrorInvalidValue;
    // Up to 8192 rows a sequence is one CTA's, of 512 threads (sixteen rows each;
    // its barriers cost less than those of 1024).  Above, eight CTAs of 1024: the
    // loads and counters of one would hold it up.  One CTA and eight, rows selected
    // and 16-byte rows moved, us: 1 x 8192 rows 15.5 and 25.9, 64 x 8192 22.6 and 93.6;
    // 1 x 16384 26.5 and 26.3; 1 x 131072 147 and 30, 8 x 131072 163 and 46.  (Eight
    // are slow where there are many sequences: 64 x 4096 rows in a cache of 131072 are
    // 18 and 92.  Callers who know a bound on the lengths pass it as T_max.)
    cudaError_t e = a.T_max <= 512 * kSlab
                        ? launch_pdl(evict_select_kernel<512>, dim3((unsigned)a.B), dim3(512), 0, st, 1, a, s)
                        : launch_pdl(evict_select_kernel<1024>, dim3((unsigned)a.B * kSelRanks), dim3(1024), 0, st, kSelRanks, a, s);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)blocks), block(kMoveThreads);
    switch (unit_bytes(a.row_bytes)) {
        case 16: return launch_pdl(evict_move_kernel<uint4>, grid, block, 0, st, 1, a, s);
        case 4: return launch_pdl(evict_move_kernel<uint32_t>, grid, block, 0, st, 1, a, s);
        default: return launch_pdl(evict_move_kernel<uint16_t>, grid, block, 0, st, 1, a, s);
    }
}

}  // namespace mla
