// Cutting the tiles of a ragged batch into equal shares, planned by every CTA
// for itself from the sequence lengths, so that no planning launch comes first.
//
// A sequence of T rows costs its tiles and `ovh` more units (what a piece of it
// costs apart from its tiles); the costs in order make a line of units, and
// group g works on units g L .. (g+1) L - 1.
#pragma once

#include <limits.h>
#include <stdint.h>

#include "mla.h"

namespace mla {
namespace sm100 {

struct Batch {
    const int32_t* seqlens;
    int B, q_len, T_max, tile, ovh;
    __device__ __forceinline__ int len(int b) const { return seqlens[b]; }
    __device__ __forceinline__ bool valid(int T) const { return T >= q_len && T <= T_max; }
    __device__ __forceinline__ int cost(int T) const { return valid(T) ? (T + tile - 1) / tile + ovh : 0; }
};

// What a block has planned, in shared memory (a walker keeps only its place in
// registers, as most roles have none to spare).
struct PieceShare {
    Batch batch;
    int L, lo, hi;   // units a group; the units of this group
    int first, pre;  // the sequence unit lo falls in, and the units before it
};

// A walk over the pieces of one group, in order.
struct Pieces {
    const PieceShare* s;
    int b, pre;
    __device__ __forceinline__ explicit Pieces(const PieceShare* share) : s(share), b(share->first), pre(share->pre) {}
    // The next piece: tiles k0..k1-1 of sequence `seq` of T rows; whole: all of them.
    __device__ bool next(int& seq, int& T, int& k0, int& k1, bool& whole) {
        const Batch& batch = s->batch;
        while (b < batch.B && pre < s->hi) {
            const int len = batch.len(b), c = batch.cost(len);
            const int tiles = c > 0 ? c - batch.ovh : 0;
            int from = s->lo - pre - batch.ovh, to = s->hi - pre - batch.ovh;
            from = from < 0 ? 0 : from;
            to = to > tiles ? tiles : to;
            const int cur = b++;
            pre += c;
            if (to > from) {
                seq = cur;
                T = len;
                k0 = from;
                k1 = to;
                whole = from == 0 && to == tiles;
                return true;
            }
        }
        return false;
    }
};

// Plans group g's share (all threads of the block; `out` and 64 ints of scratch
// in shared memory; first = B where there is no unit g L).
//   min_units: smallest share.  whole_equal: a batch of equal valid lengths is
//   cut at sequence boundaries when that makes the share at most a quarter larger.
__device__ __forceinline__ void plan_share(const Batch& batch, int groups, int g, int min_units, bool whole_equal,
                                           int* scratch, PieceShare* out) {
    const int n = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = n >> 5;
    const int per = (batch.B + n - 1) / n;
    const int b0 = tid * per;
    int sum = 0, lo_c = INT_MAX, hi_c = 0;
    for (int b = b0; b < b0 + per && b < batch.B; ++b) {
        const int c = batch.cost(batch.len(b));
        lo_c = min(lo_c, c);
        hi_c = max(hi_c, c);
        sum += c;
    }
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    lo_c = __reduce_min_sync(0xffffffffu, lo_c);
    hi_c = __reduce_max_sync(0xffffffffu, hi_c);
    if (lane == 31) scratch[warp] = inc;
    if (lane == 0) scratch[32 + warp] = lo_c == hi_c && lo_c > 0 ? lo_c : (lo_c == INT_MAX ? -1 : 0);
    if (tid == 0) {
        out->batch = batch;
        out->first = batch.B;
        out->pre = 0;
    }
    __syncthreads();
    // every warp adds the warps' sums up for itself
    const int ws = lane < warps ? scratch[lane] : 0, we = lane < warps ? scratch[32 + lane] : -1;
    const int total = __reduce_add_sync(0xffffffffu, ws);
    const int before = __reduce_add_sync(0xffffffffu, lane < warp ? ws : 0);
    const int e_max = __reduce_max_sync(0xffffffffu, we);
    const int e_min = __reduce_min_sync(0xffffffffu, we < 0 ? INT_MAX : we);
    const int equal = e_max == e_min ? e_max : 0;  // the one cost of every sequence, 0 if they differ
    int L = (total + groups - 1) / groups;
    if (whole_equal && equal > 0) {
        const int whole = ((batch.B + groups - 1) / groups) * equal;
        if (whole <= L + L / 4) L = whole;
    }
    L = max(max(L, min_units), 1);
    const int64_t unit = (int64_t)g * L;
    if (tid == 0) {
        out->L = L;
        out->lo = g * L;
        out->hi = g * L + L;
    }
    int pre = before + inc - sum;
    if (unit >= pre && unit < (int64_t)pre + sum) {
        int b = b0;
        for (;; ++b) {
            const int c = batch.cost(batch.len(b));
            if (unit < (int64_t)pre + c) break;
            pre += c;
        }
        out->first = b;
        out->pre = pre;
    }
    __syncthreads();
}

}  // namespace sm100
}  // namespace mla
