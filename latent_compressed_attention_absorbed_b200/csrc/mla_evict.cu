// Eviction from a cache by accumulated attention weight: which rows of every
// sequence stay, and the compaction of the cache to those rows.
//
// Of a sequence of T rows that is over the budget, the first n_sink rows, the
// last n_recent rows and the m = budget - n_sink - n_recent rows of the middle
// with the largest weights stay, in their order.  Equal weights: the lower
// row; -0 equals 0, a NaN counts as less than every number.
//
// evict_select_kernel: a cluster of CTAs per sequence finds the m-th largest
// weight by a radix search over order-preserving 32-bit keys (three passes of
// 11, 11 and 10 bits: each pass counts the digits of the keys that share the
// prefix found so far, in shared memory, and the CTAs add their counts up
// through distributed shared memory), then lists the kept rows in order with
// one prefix sum.  The weights are read from HBM once; the later passes hit L2.
// evict_move_kernel: a CTA moves a chunk of kept rows.  It is bound by HBM:
// every kept row is read once and written once.
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

constexpr int kSelThreads = 1024;
constexpr int kSelBins = 2048;
constexpr int kSlab = 16;  // rows a thread of the selection holds
constexpr int kMoveThreads = 256;
constexpr int kMovePieces = 8;  // 16-byte pieces a thread holds: chunks of up to 32 KB

// Larger weight <-> larger key; NaN 0, -0 as 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.0f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

struct EvictScratch {
    int32_t* kept;    // [B][budget] rows kept, ascending
    int32_t* count;   // [B]
    int32_t* loaded;  // [B][chunks]: the chunk's rows are in registers
    int32_t* ticket;
    int chunks, chunk_rows;
};

// Block-wide exclusive prefix of two counts; `total` gets their sums.
__device__ __forceinline__ void block_scan2(int& a, int& b, int2* warp_sums, int2& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = a, y = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x1 = __shfl_up_sync(0xffffffffu, x, o), y1 = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) {
            x += x1;
            y += y1;
        }
    }
    __syncthreads();  // warp_sums of the previous scan have been read
    if (lane == 31) warp_sums[warp] = make_int2(x, y);
    __syncthreads();
    int2 w = warp_sums[lane];  // 32 warps
    int wx = w.x, wy = w.y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x1 = __shfl_up_sync(0xffffffffu, wx, o), y1 = __shfl_up_sync(0xffffffffu, wy, o);
        if (lane >= o) {
            wx += x1;
            wy += y1;
        }
    }
    total = make_int2(__shfl_sync(0xffffffffu, wx, 31), __shfl_sync(0xffffffffu, wy, 31));
    const int bx = __shfl_sync(0xffffffffu, wx - w.x, warp), by = __shfl_sync(0xffffffffu, wy - w.y, warp);
    const int ax = x - a, ay = y - b;
    a = bx + ax;
    b = by + ay;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(EvictArgs a, EvictScratch s) {
    __shared__ int hist[kSelBins];
    __shared__ int2 warp_sums[32];
    __shared__ int2 mine;     // this CTA's counts, read by the others
    __shared__ int found[2];  // digit, keys above it
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int b = blockIdx.x / ranks, tid = threadIdx.x;
    sm100::pdl_wait();
    sm100::pdl_trigger();
    const int T = a.seqlens[b];
    const bool bad = T < 0 || T > a.T_max;
    if (blockIdx.x == 0 && tid == 0) *s.ticket = 0;
    if (rank == 0)
        for (int c = tid; c < s.chunks; c += kSelThreads) s.loaded[(size_t)b * s.chunks + c] = 0;
    const int n = bad ? 0 : (T < a.budget ? T : a.budget);
    int32_t* kept = s.kept + (size_t)b * a.budget;
    int32_t* kept_out = a.kept_out ? a.kept_out + (size_t)b * a.budget : nullptr;
    if (bad || T <= a.budget) {  // the same for the whole cluster
        if (bad && rank == 0 && tid == 0) atomicOr(a.status, MLA_STATUS_BAD_SEQLEN);
        for (int j = rank * kSelThreads + tid; j < a.budget; j += ranks * kSelThreads) {
            if (j < n) kept[j] = j;
            if (kept_out) kept_out[j] = j < n ? j : -1;
        }
    } else {
        const int lo = a.n_sink, hi = T - a.n_recent;  // the middle
        const int m = a.budget - a.n_sink - a.n_recent;
        const float* w = a.weights + (size_t)b * a.stride_w;
        const bool wide = (reinterpret_cast<uintptr_t>(w) & 15) == 0;
        // This CTA's rows, and a slab of them in registers: `each` consecutive
        // rows a thread.  One slab holds all of them up to 16384 rows a CTA, so
        // that the weights are read once; beyond that every pass reads them
        // again, from L2.
        const int64_t per = (((int64_t)T + ranks - 1) / ranks + 3) & ~int64_t(3);
        const int64_t t_lo = min((int64_t)T, rank * per), t_hi = min((int64_t)T, t_lo + per);
        const int slabs = (int)((per + kSlab * kSelThreads - 1) / (kSlab * kSelThreads));
        const int each = slabs > 1 ? kSlab : (int)((per + 4 * kSelThreads - 1) / (4 * kSelThreads)) * 4;
        uint32_t key[kSlab];
        uint32_t middle = 0, there = 0;  // which of them are in the middle, which are rows at all
        int held = -1;
        auto load_slab = [&](int slab) {
            if (held == slab) return;
            held = slab;
            middle = there = 0;
            const int64_t t0 = t_lo + ((int64_t)slab * kSelThreads + tid) * each;
#pragma unroll
            for (int v = 0; v < kSlab / 4; ++v) {
                const int64_t t = t0 + 4 * v;
                float x[4] = {0.f, 0.f, 0.f, 0.f};
                if (4 * v < each && t < t_hi) {
                    if (wide && t + 4 <= t_hi) {
                        const float4 f = *reinterpret_cast<const float4*>(w + t);
                        x[0] = f.x; x[1] = f.y; x[2] = f.z; x[3] = f.w;
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (t + j < t_hi) x[j] = w[t + j];
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    key[4 * v + j] = weight_key(x[j]);
                    if (4 * v < each && t + j < t_hi) {
                        there |= 1u << (4 * v + j);
                        if (t + j >= lo && t + j < hi) middle |= 1u << (4 * v + j);
                    }
                }
            }
        };
        // ---- the m-th largest key of the middle
        uint32_t last = 0xFFFFFFFFu;
        int equal_left = 0;  // how many of the keys equal to it stay
        if (m > 0) {
            uint32_t prefix = 0;
            int need = m;
            int shift = 32;
            for (int pass = 0; pass < 3; ++pass) {
                const int bits = pass < 2 ? 11 : 10;
                const uint32_t above = shift == 32 ? 0u : 0xFFFFFFFFu << shift;
                shift -= bits;
                for (int i = tid; i < kSelBins; i += kSelThreads) hist[i] = 0;
                __syncthreads();
                for (int slab = 0; slab < slabs; ++slab) {
                    load_slab(slab);
#pragma unroll
                    for (int i = 0; i < kSlab; ++i)
                        if ((middle >> i & 1) && ((key[i] ^ prefix) & above) == 0)
                            atomicAdd(&hist[(key[i] >> shift) & ((1 << bits) - 1)], 1);
                }
                if (ranks > 1) cluster.sync();
                else __syncthreads();
                // two bins a thread, from the highest digit down
                int c0 = 0, c1 = 0;
                const int d0 = kSelBins - 1 - 2 * tid;
                for (int r = 0; r < ranks; ++r) {
                    const int* other = cluster.map_shared_rank(hist, r);
                    const int2 two = *reinterpret_cast<const int2*>(other + d0 - 1);
                    c0 += two.y;
                    c1 += two.x;
                }
                int before = c0 + c1, none = 0;
                int2 total;
                block_scan2(before, none, warp_sums, total);
                if (before < need && before + c0 >= need) {
                    found[0] = d0;
                    found[1] = before;
                } else if (before + c0 < need && before + c0 + c1 >= need) {
                    found[0] = d0 - 1;
                    found[1] = before + c0;
                }
                // every CTA has read the counts; found is set
                if (ranks > 1) cluster.sync();
                else __syncthreads();
                prefix |= (uint32_t)found[0] << shift;
                need -= found[1];
                __syncthreads();
            }
            last = prefix;
            equal_left = need;
        }
        // ---- the kept rows in order.  over: rows that stay whatever else does; equal: rows of the last weight.
        auto classify = [&](uint32_t& over, uint32_t& equal) {
            over = there & ~middle;
            equal = 0;
            if (m > 0) {
#pragma unroll
                for (int i = 0; i < kSlab; ++i) {
                    if (key[i] > last) over |= middle & (1u << i);
                    if (key[i] == last) equal |= middle & (1u << i);
                }
            }
        };
        int base_over = 0, base_equal = 0;
        uint32_t over, equal;
        int2 total;
        if (ranks > 1) {  // what the CTAs before this one keep
            int x = 0, y = 0;
            for (int slab = 0; slab < slabs; ++slab) {
                load_slab(slab);
                classify(over, equal);
                x += __popc(over);
                y += __popc(equal);
            }
            block_scan2(x, y, warp_sums, total);
            if (tid == 0) mine = total;
            cluster.sync();
            for (int r = 0; r < rank; ++r) {
                const int2 o = *cluster.map_shared_rank(&mine, r);
                base_over += o.x;
                base_equal += o.y;
            }
        }
        for (int slab = 0; slab < slabs; ++slab) {
            load_slab(slab);
            classify(over, equal);
            int x = __popc(over), y = __popc(equal);
            block_scan2(x, y, warp_sums, total);
            x += base_over;
            y += base_equal;
            const int64_t t0 = t_lo + ((int64_t)slab * kSelThreads + tid) * each;
#pragma unroll
            for (int i = 0; i < kSlab; ++i) {
                const bool is_over = over >> i & 1, is_equal = equal >> i & 1;
                if (is_over || (is_equal && y < equal_left)) {
                    const int slot = x + min(y, equal_left);
                    kept[slot] = (int32_t)(t0 + i);
                    if (kept_out) kept_out[slot] = (int32_t)(t0 + i);
                }
                x += is_over;
                y += is_equal;
            }
            base_over += total.x;
            base_equal += total.y;
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
            atomicExch(&loaded[chunk], 1);
            const int c0 = s_wait[0] / s.chunk_rows, c1 = (s_wait[1] - 1) / s.chunk_rows;
            bool ok = true;
            for (int c = c0; c <= c1 && c < chunk && s_wait[1] > s_wait[0]; ++c) {
                const uint64_t start = sm100::global_timer_ns();
                while (atomicAdd(&loaded[c], 0) == 0) {
                    if (sm100::global_timer_ns() - start > MLA_WAIT_LIMIT_NS) {
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

cudaError_t evict_launch(const EvictArgs& a, void* workspace, cudaStream_t st) {
    EvictScratch s;
    evict_layout(a.B, a.budget, a.row_bytes, &s, workspace);
    const int64_t blocks = (int64_t)a.B * s.chunks;
    if (blocks > INT_MAX) return cudaErrorInvalidValue;
    // One CTA a sequence up to 8192 rows (eight a thread), eight above: a single
    // CTA's shared-memory counters and its share of L2 would hold it up, while
    // the eight meetings of a cluster cost about 8 us.
    const int ranks = a.T_max <= 8 * kSelThreads ? 1 : 8;
    cudaError_t e = launch_pdl(evict_select_kernel, dim3((unsigned)(a.B * ranks)), dim3(kSelThreads), 0, st, ranks, a, s);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)blocks), block(kMoveThreads);
    switch (unit_bytes(a.row_bytes)) {
        case 16: return launch_pdl(evict_move_kernel<uint4>, grid, block, 0, st, 1, a, s);
        case 4: return launch_pdl(evict_move_kernel<uint32_t>, grid, block, 0, st, 1, a, s);
        default: return launch_pdl(evict_move_kernel<uint16_t>, grid, block, 0, st, 1, a, s);
    }
}

}  // namespace mla
