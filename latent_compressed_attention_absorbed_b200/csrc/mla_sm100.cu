// Host launchers of the sm_100a path (bf16 storage, V3 head geometry:
// H = 128, d_c = 512, d_r = 64, d_n = 128, d_v = 128).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <string.h>

#include <utility>

#include "mla_internal.h"
#include "mla_rope.cuh"
#include "sm100_host.h"
#include "sm100_attend.cuh"
#include "sm100_gemm.cuh"
#include "sm100_gemv.cuh"
#include "sm100_packed_attend.cuh"
#include "sm100_weights.cuh"
#include "mla_packed_internal.h"

#ifdef MLA_TRACE
// Copies the attention kernel's timing trace (4096 tiles x 16 stamps) to host
// memory; only in builds compiled with -DMLA_TRACE.
extern "C" int mla_trace_read(void* host, size_t bytes) {
    return cudaMemcpyFromSymbol(host, mla::sm100::g_mla_trace, bytes) == cudaSuccess ? 0 : -4;
}
extern "C" int mla_trace_read_all(void* host, size_t bytes) {
    return cudaMemcpyFromSymbol(host, mla::sm100::g_mla_trace_all, bytes) == cudaSuccess ? 0 : -4;
}
extern "C" int mla_trace_read_kt(void* host, size_t bytes) {
    return cudaMemcpyFromSymbol(host, mla::sm100::g_mla_ktrace, bytes) == cudaSuccess ? 0 : -4;
}
extern "C" int mla_trace_clear_kt(void) {
    unsigned long long init[mla::sm100::kKtN][3];
    for (int k = 0; k < mla::sm100::kKtN; ++k) {
        init[k][0] = init[k][1] = ~0ull;
        init[k][2] = 0;
    }
    return cudaMemcpyToSymbol(mla::sm100::g_mla_ktrace, init, sizeof(init)) == cudaSuccess ? 0 : -4;
}
extern "C" int mla_trace_clear(void) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, mla::sm100::g_mla_trace) != cudaSuccess) return -4;
    if (cudaMemset(p, 0, sizeof(mla::sm100::g_mla_trace)) != cudaSuccess) return -4;
    if (cudaGetSymbolAddress(&p, mla::sm100::g_mla_trace_all) != cudaSuccess) return -4;
    return cudaMemset(p, 0, sizeof(mla::sm100::g_mla_trace_all)) == cudaSuccess ? 0 : -4;
}
#endif

namespace mla {

using namespace sm100;

namespace {

// ------------------------------------------------------------------ append

// One warp per new token: 16-byte copies of the 512 latent values and the
// RoPE rotation of the 64-wide key at its position (one pair per lane).
__global__ void append_v3_kernel(const __nv_bfloat16* __restrict__ c_kv, const __nv_bfloat16* __restrict__ k_rope,
                                 const int32_t* __restrict__ pos, int B, int n_tok, CacheView cache, RopeTable rope,
                                 int* status) {
    MLA_KT(kKtAppend, 0);
    const int gw = (blockIdx.x * blockDim.x + threadIdx.x) / 32;
    const int lane = threadIdx.x & 31;
    if (gw >= B * n_tok) return;
    const int b = gw / n_tok, i = gw % n_tok;
    const int p0 = pos[b];
    if (p0 < 0 || p0 + n_tok > cache.T_max) {
        if (lane == 0 && i == 0) atomicOr(status, MLA_STATUS_BAD_POS);
        return;
    }
    const int t = p0 + i;
    __nv_bfloat16* row = static_cast<__nv_bfloat16*>(cache.data) + (size_t)b * cache.stride_b + (size_t)t * cache.stride_t;
    const uint4* src = reinterpret_cast<const uint4*>(c_kv + (size_t)gw * kLat);
    uint4* dst = reinterpret_cast<uint4*>(row);
    dst[lane] = src[lane];
    dst[lane + 32] = src[lane + 32];
    const __nv_bfloat162 k2 = reinterpret_cast<const __nv_bfloat162*>(k_rope + (size_t)gw * kRope)[lane];
    float y0, y1;
    mla_rope_rotate(__low2float(k2), __high2float(k2), rope.inv_freq[lane], t, &y0, &y1);
    reinterpret_cast<__nv_bfloat162*>(row + kLat)[lane] = __floats2bfloat162_rn(y0, y1);
    MLA_KT(kKtAppend, 2);
}

DoneFlags g_smem_absorb, g_smem_project, g_smem_attend[2], g_smem_packed;
DoneFlags g_smem_weights[2];
DoneFlags g_smem_absorb_gemv[4], g_smem_project_gemv[4];

constexpr int kAbsorbStages = 2;
// Rows of the A tile a GEMM CTA loads: all 128 when the batch fills them,
// else the batch rounded up to 16 (the MMA still computes 128 rows; the rows
// past the batch are never stored).
int plan_ovh(int overhead_tiles) { return overhead_tiles < 0 ? 2 : overhead_tiles; }
int plan_min_units(int min_tiles) { return min_tiles > 0 ? (min_tiles < kMaxUnits ? min_tiles : kMaxUnits) : 2; }
int gemm_a_rows(int rows) { return rows >= 128 ? 128 : ((rows + 15) / 16) * 16; }
constexpr int kProjStages = 4;
constexpr int kProjNT = 64;

}  // namespace

bool sm100_supported(const Problem& p, int q_len) {
    if (p.dtype != MLA_DTYPE_BF16 || p.H != kHeads || p.d_c != kLat || p.d_r != kRope || p.d_n != 128 ||
        p.d_v != 128)
        return false;
    if (q_len < 1 || q_len > 16) return false;
    int dev = 0, major = 0, minor = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    return major == 10 && minor == 0;
}

int sm100_default_pairs() { return device_sm_count() / 2; }

cudaError_t sm100_append(const Problem& p, const void* c_kv, const void* k_rope, const int32_t* pos, int n_tok,
                         const CacheView& cache, int* status, cudaStream_t st) {
    const int warps = p.B * n_tok;
    const int threads = 128;
    const int blocks = (warps * 32 + threads - 1) / threads;
    append_v3_kernel<<<blocks, threads, 0, st>>>((const __nv_bfloat16*)c_kv, (const __nv_bfloat16*)k_rope, pos, p.B,
                                                 n_tok, cache, p.rope, status);
    return cudaGetLastError();
}

cudaError_t sm100_absorb(const Problem& p, const void* q_nope, const void* q_rope, const void* W_UK,
                         const int32_t* seqlens, void* q_hat, cudaStream_t st, const PlanRequest* plan) {
    const int rows = p.B * p.q_len;
    CUtensorMap mA, mB;
    // A: q_nope viewed as [rows][H][128]; box 64 x 1 x 128 rows.
    if (!make_map(&mA, q_nope, 128, kHeads, rows, 128 * 2, (uint64_t)kHeads * 128 * 2, 64, 1, gemm_a_rows(rows),
                  CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    // B: W_UK viewed as [H][128 (d)][512 (c)]; box 64 c x 64 d x 1.
    if (!make_map(&mB, W_UK, kLat, 128, kHeads, kLat * 2, (uint64_t)128 * kLat * 2, 64, 64, 1,
                  CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    using Cfg = GemmCfg<2, 256, true, kAbsorbStages, true>;
    auto kern = head_gemm_kernel<2, 256, true, kAbsorbStages, true>;
    cudaError_t e = set_smem(kern, Cfg::kSmem, g_smem_absorb);
    if (e != cudaSuccess) return e;
    GemmArgs a;
    a.rows = rows;
    a.H = kHeads;
    a.ld_out = kRow;
    a.out_col0 = 0;
    a.out = (__nv_bfloat16*)q_hat;
    a.out_v8 = (reinterpret_cast<uintptr_t>(q_hat) & 31u) == 0;
    a.q_rope = (const __nv_bfloat16*)q_rope;
    a.seqlens = seqlens;
    a.q_len = p.q_len;
    a.rope = p.rope;
    a.status = device_status_ptr();
    a.a_rows = gemm_a_rows(rows);
    a.plan = nullptr;
    if (plan) {
        a.plan = static_cast<Plan*>(plan->plan);
        a.plan_B = p.B;
        a.plan_T_max = plan->T_max;
        a.plan_clusters = plan->clusters;
        a.plan_ovh = plan_ovh(plan->overhead_tiles);
        a.plan_min_units = plan_min_units(plan->min_tiles);
        a.plan_olat = static_cast<__nv_bfloat16*>(plan->o_lat);
    }
    dim3 grid(kHeads, kLat / 256, (rows + 127) / 128);
    return launch_pdl(kern, grid, dim3(128), Cfg::kSmem, st, 1, mA, mB, a);
}

cudaError_t sm100_project(const Problem& p, const void* o_lat, const void* W_UV, int rows, void* out,
                          cudaStream_t st) {
    CUtensorMap mA, mB;
    // A: o_lat viewed as [rows][H][512]; box 64 x 1 x 128.
    if (!make_map(&mA, o_lat, kLat, kHeads, rows, kLat * 2, (uint64_t)kHeads * kLat * 2, 64, 1, gemm_a_rows(rows),
                  CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    // B: W_UV viewed as [H][128 (d)][512 (c)]; box 64 c x NT d x 1 (K-major).
    if (!make_map(&mB, W_UV, kLat, 128, kHeads, kLat * 2, (uint64_t)128 * kLat * 2, 64, kProjNT, 1,
                  CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    using Cfg = GemmCfg<8, kProjNT, false, kProjStages, false>;
    auto kern = head_gemm_kernel<8, kProjNT, false, kProjStages, false>;
    cudaError_t e = set_smem(kern, Cfg::kSmem, g_smem_project);
    if (e != cudaSuccess) return e;
    GemmArgs a;
    memset(&a, 0, sizeof(a));
    a.plan = nullptr;
    a.rows = rows;
    a.H = kHeads;
    a.ld_out = 128;
    a.out_col0 = 0;
    a.out = (__nv_bfloat16*)out;
    a.out_v8 = (reinterpret_cast<uintptr_t>(out) & 31u) == 0;
    a.status = device_status_ptr();
    a.q_len = 1;
    a.a_rows = gemm_a_rows(rows);
    dim3 grid(kHeads, 128 / kProjNT, (rows + 127) / 128);
    return launch_pdl(kern, grid, dim3(128), Cfg::kSmem, st, 1, mA, mB, a);
}

// Small batches (rows <= kGemvMaxRows): CUDA-core matrix-vector kernels with
// the weight slices staged in shared memory; R = rows rounded up to 1, 2, 4, 8.
template <int R>
static cudaError_t absorb_gemv_launch(const AbsorbGemvArgs& a, cudaStream_t st) {
    static_assert(R == 1 || R == 2 || R == 4 || R == 8, "row count");
    constexpr int idx = R == 1 ? 0 : R == 2 ? 1 : R == 4 ? 2 : 3;
    cudaError_t e = set_smem(absorb_gemv_kernel<R>, absorb_gemv_smem<R>(), g_smem_absorb_gemv[idx]);
    if (e != cudaSuccess) return e;
    // W_UK [128 heads][128][512]: one box of 256 latent columns x 128 rows per CTA
    CUtensorMap mapW;
    if (!make_map(&mapW, a.W_UK, kLat, 128, kHeads, (uint64_t)kLat * 2, (uint64_t)128 * kLat * 2, 256, 128, 1,
                  CU_TENSOR_MAP_SWIZZLE_NONE))
        return cudaErrorInvalidValue;
    return launch_pdl(absorb_gemv_kernel<R>, dim3(kHeads + 1, 2), dim3(128), absorb_gemv_smem<R>(), st, 1, mapW, a);
}
template <int R>
static cudaError_t project_gemv_launch(const ProjectGemvArgs& a, cudaStream_t st) {
    constexpr int idx = R == 1 ? 0 : R == 2 ? 1 : R == 4 ? 2 : 3;
    cudaError_t e = set_smem(project_gemv_kernel<R>, project_gemv_smem<R>(), g_smem_project_gemv[idx]);
    if (e != cudaSuccess) return e;
    // W_UV [128 heads][128][512]: eight SW128 boxes of 64 latent columns x 128 rows per CTA
    CUtensorMap mapW;
    if (!make_map(&mapW, a.W_UV, kLat, 128, kHeads, (uint64_t)kLat * 2, (uint64_t)128 * kLat * 2, 64, 128, 1,
                  CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    return launch_pdl(project_gemv_kernel<R>, dim3(kHeads), dim3(512), project_gemv_smem<R>(), st, 1, mapW, a);
}

cudaError_t sm100_absorb_small(const Problem& p, const void* q_nope, const void* q_rope, const void* W_UK,
                               const int32_t* seqlens, void* q_hat, cudaStream_t st, const PlanRequest* plan) {
    const int rows = p.B * p.q_len;
    if (rows < 1 || rows > kGemvMaxRows) return cudaErrorInvalidValue;
    AbsorbGemvArgs a;
    memset(&a, 0, sizeof(a));
    a.q_nope = (const __nv_bfloat16*)q_nope;
    a.q_rope = (const __nv_bfloat16*)q_rope;
    a.W_UK = (const __nv_bfloat16*)W_UK;
    a.seqlens = seqlens;
    a.rows = rows;
    a.q_len = p.q_len;
    a.q_hat = (__nv_bfloat16*)q_hat;
    a.rope = p.rope;
    a.status = device_status_ptr();
    a.plan = nullptr;
    if (plan) {
        a.plan = static_cast<Plan*>(plan->plan);
        a.plan_B = p.B;
        a.plan_T_max = plan->T_max;
        a.plan_clusters = plan->clusters;
        a.plan_ovh = plan_ovh(plan->overhead_tiles);
        a.plan_min_units = plan_min_units(plan->min_tiles);
        a.plan_olat = static_cast<__nv_bfloat16*>(plan->o_lat);
    }
    if (rows == 1) return absorb_gemv_launch<1>(a, st);
    if (rows == 2) return absorb_gemv_launch<2>(a, st);
    if (rows <= 4) return absorb_gemv_launch<4>(a, st);
    return absorb_gemv_launch<8>(a, st);
}

// Clusters of the attention grid: at least one per query token (a group of
// q_len clusters streams one sequence piece, one cluster per token).
static int attend_clusters(int pairs, int q_len) { return pairs < q_len ? q_len : pairs; }

// Workspace of the attention step: plan, fp32 partials and LSEs.
static size_t attend_layout(const Problem& p, int pairs, size_t* off_part, size_t* off_lse) {
    const int clusters = attend_clusters(pairs, p.q_len);
    Carve c(nullptr);
    const size_t units = (size_t)p.B * p.q_len;  // one per query token
    c.take(sizeof(Plan) + sizeof(int) * (kPlanMaxGroups + 2 * units + 1));
    const size_t slots = (size_t)clusters + units;
    *off_part = c.off;
    c.take(slots * kHeads * kLat * sizeof(float));
    *off_lse = c.off;
    c.take(slots * kHeads * sizeof(float));
    return c.off;
}

void* sm100_plan_ptr(void* attend_workspace) { return attend_workspace; }

size_t sm100_attend_workspace_bytes(const Problem& p, int num_pairs) {
    size_t a, b;
    return attend_layout(p, num_pairs, &a, &b);
}

cudaError_t sm100_attend(const Problem& p, const void* q_hat, const CacheView& cache, const int32_t* seqlens,
                         void* o_lat, void* workspace, size_t ws_bytes, int num_pairs, int overhead_tiles,
                         int min_tiles, int* status, cudaStream_t st, const Events* events, bool plan_ready,
                         bool combine, const void* prefetch, size_t prefetch_bytes, const mla_decode_opts_t* opts,
                         float* lse) {
    const int clusters = attend_clusters(num_pairs, p.q_len);
    if (clusters / p.q_len > kPlanMaxGroups) return cudaErrorInvalidValue;
    size_t off_part, off_lse;
    const size_t need = attend_layout(p, clusters, &off_part, &off_lse);
    if (ws_bytes < need) return cudaErrorInvalidValue;
    char* ws = static_cast<char*>(workspace);
    Plan* plan = reinterpret_cast<Plan*>(ws);
    // The cache as [B][T_max][576]: boxes of 64 columns x 64 keys (SW128); the
    // scoring CTA loads all nine of a row tile, the accumulating CTA the eight
    // latent ones.
    CUtensorMap mRow;
    const uint64_t sb = (uint64_t)cache.stride_b * 2, stt = (uint64_t)cache.stride_t * 2;
    if (!make_map(&mRow, cache.data, kRow, cache.T_max, p.B, stt, sb, 64, kNk, 1, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;

    cudaError_t e;
    if (!plan_ready) {
        mla_plan_kernel<<<1, 32, 0, st>>>(seqlens, p.B, p.q_len, cache.T_max, clusters, plan_ovh(overhead_tiles),
                                          plan_min_units(min_tiles), plan, status, (__nv_bfloat16*)o_lat, lse);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }

    const auto attend = lse ? mla_attend_kernel<true> : mla_attend_kernel<false>;
    e = set_smem(attend, kAttSmem, g_smem_attend[lse != nullptr]);
    if (e != cudaSuccess) return e;
    AttendArgs a;
    a.plan = plan;
    a.seqlens = seqlens;
    a.q_len = p.q_len;
    a.scale_log2 = p.scale * 1.4426950408889634f;
    a.q_hat = (const __nv_bfloat16*)q_hat;
    a.o_lat = (__nv_bfloat16*)o_lat;
    a.o_lat_v8 = (reinterpret_cast<uintptr_t>(o_lat) & 31u) == 0;
    a.prefetch = static_cast<const uint8_t*>(prefetch);
    a.prefetch_bytes = prefetch ? prefetch_bytes : 0;
    a.part_o = reinterpret_cast<float*>(ws + off_part);
    a.part_lse = reinterpret_cast<float*>(ws + off_lse);
    a.lse = lse;
    a.status = status;
    a.wait_limit_ns = (opts && opts->wait_limit_ns > 0) ? (uint64_t)opts->wait_limit_ns : MLA_WAIT_LIMIT_NS;
    a.withhold_tile = (opts && opts->withhold_tile > 0) ? opts->withhold_tile : -1;
    a.cache = static_cast<const uint8_t*>(cache.data);
    a.stride_b = cache.stride_b * 2;
    a.stride_t = cache.stride_t * 2;
    a.T_max = cache.T_max;

    if (events) events->record(MLA_EV_ATTEND_BEGIN, st);
    e = launch_pdl(attend, dim3(clusters * 2), dim3(kAttThreads), kAttSmem, st, 2, mRow, a);
    if (e != cudaSuccess) return e;
    if (events) events->record(MLA_EV_ATTEND_END, st);

    // Split units number at most min(B * q_len, clusters); one CTA covers
    // eight heads of one unit.
    const int units = p.B * p.q_len;
    const int max_split = units < clusters ? units : clusters;
    if (combine)
        e = launch_pdl(mla_combine_kernel, dim3(max_split * (kHeads / 8)), dim3(256), 0, st, 1, (const Plan*)plan,
                       (const float*)a.part_o, (const float*)a.part_lse, (__nv_bfloat16*)o_lat, lse);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

cudaError_t sm100_attend_packed(const Problem& p, const void* q_hat, const CacheView& cache, const int32_t* seqlens,
                                const int32_t* n_seen, void* o_lat, float* lse, void* workspace, size_t ws_bytes, int num_pairs, int* status,
                                const mla_decode_opts_t* opts, cudaStream_t st) {
    const int clusters = attend_clusters(num_pairs, p.q_len);
    if (clusters / p.q_len > kPlanMaxGroups) return cudaErrorInvalidValue;
    size_t off_part, off_lse;
    if (ws_bytes < attend_layout(p, clusters, &off_part, &off_lse)) return cudaErrorInvalidValue;
    char* ws = static_cast<char*>(workspace);
    CUtensorMap mRaw, mRope;
    const uint64_t stt = (uint64_t)cache.stride_t;
    const uint64_t sb = p.B > 1 ? (uint64_t)cache.stride_b : stt * (uint64_t)cache.T_max;
    const uint8_t* rows = static_cast<const uint8_t*>(cache.data);
    if (!make_map_words(&mRaw, rows, pk::kRawRow / 2, cache.T_max, p.B, stt, sb, pk::kRawRow / 2, pk::kUnit, 1,
                        CU_TENSOR_MAP_SWIZZLE_NONE) ||
        !make_map(&mRope, rows + kPackRope, kRope, cache.T_max, p.B, stt, sb, kRope, pk::kUnit, 1, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    cudaError_t e;
    e = set_smem(pk::packed_attend_kernel, pk::kSmem, g_smem_packed);
    if (e != cudaSuccess) return e;
    pk::Args a;
    a.seqlens = seqlens;
    a.n_seen = n_seen;
    a.B = p.B;
    a.q_len = p.q_len;
    a.T_max = cache.T_max;
    a.ovh = opts && opts->overhead_tiles >= 0 ? opts->overhead_tiles : 1;
    a.min_units = opts && opts->min_tiles > 0 ? plan_min_units(opts->min_tiles) : 1;
    a.scale_log2 = p.scale * 1.4426950408889634f;
    a.q_hat = (const __nv_bfloat16*)q_hat;
    a.o_lat = (__nv_bfloat16*)o_lat;
    a.o_lat_v8 = (reinterpret_cast<uintptr_t>(o_lat) & 31u) == 0;
    const int groups = clusters / p.q_len;
    a.cuts = reinterpret_cast<int4*>(ws);  // (in the plan's place)
    a.cuts_by_seq = p.B < groups;
    a.part_o = reinterpret_cast<float*>(ws + off_part);
    a.part_lse = reinterpret_cast<float*>(ws + off_lse);
    a.lse = lse;
    a.status = status;
    a.wait_limit_ns = (opts && opts->wait_limit_ns > 0) ? (uint64_t)opts->wait_limit_ns : MLA_WAIT_LIMIT_NS;
    a.withhold_tile = (opts && opts->withhold_tile > 0) ? opts->withhold_tile : -1;
    e = launch_pdl(pk::packed_attend_kernel, dim3(clusters * 2), dim3(pk::kThreads), pk::kSmem, st, 2, mRaw, mRope, a);
    if (e != cudaSuccess) return e;
    if (groups < 2) return cudaSuccess;  // nothing is cut
    pk::MergeArgs m;
    m.cuts = a.cuts;
    m.q_len = p.q_len;
    m.part_o = a.part_o;
    m.part_lse = a.part_lse;
    m.o_lat = a.o_lat;
    m.lse = lse;
    const int tokens = (a.cuts_by_seq ? p.B : groups - 1) * p.q_len;
    if (tokens <= 8)
        return launch_pdl(pk::packed_merge_kernel<1, 16>, dim3(tokens * kHeads), dim3(512), 0, st, 1, m);
    return launch_pdl(pk::packed_merge_kernel<8, 2>, dim3(tokens * (kHeads / 8)), dim3(512), 0, st, 1, m);
}

// How many CTAs of a cluster share the queries of a tile (see sm100_weights.cuh),
// and the clusters that run at once: the split with the least estimated time, in
// tiles, of which one takes 2.6 us, a pass over a block `pass` more for Q-hat's
// load, and the joining of a cluster's sums `join`.  A cluster's range must fit
// the eight tiles whose sums it holds, by the cache's size, as the lengths lie on
// the device.  One CTA against a cluster, in us: 1 x 600 packed rows with 16
// queries 55 and 13, 1 x 4096 with 2 11.2 and 9.3, with 16 56 and 23; but 16 x
// 2000 with 2 15.6 and 18.0, which the rule leaves to one.  In a cache much longer
// than its sequences the rule sees no clusters (1 x 600 rows with 16 queries: 13 us
// by T_max 600, 56 to 64 by 131072), so callers who know a bound pass it as T_max.
template <bool kPacked>
static void weights_split(const Problem& p, int T_max, int* ranks, int* clusters) {
    using C = wt::Cfg<kPacked>;
    static std::atomic<int> most[4][kMaxDev];  // clusters of 2, 4 and 8 CTAs that run at once (0: not asked yet)
    const int sms = device_sm_count();
    *ranks = 1;
    *clusters = sms;
    int dev = 0;
    if (p.q_len == 1 || cudaGetDevice(&dev) != cudaSuccess || dev >= kMaxDev) return;
    constexpr double pass = 0.2, join = 0.75;
    const int64_t units = (int64_t)p.B * ((T_max + wt::kTile - 1) / wt::kTile + 1);  // (one more a sequence, as plan_share has it)
    const int64_t alone = (units + sms - 1) / sms;
    double best = p.q_len * (double)(alone + pass * ((alone + wt::kBlock - 1) / wt::kBlock));
    for (int k = 1; k <= 3 && (1 << k) <= p.q_len; ++k) {
        int n = most[k][dev].load(std::memory_order_relaxed);
        if (n == 0) {
            cudaLaunchConfig_t cfg;
            memset(&cfg, 0, sizeof(cfg));
            cudaLaunchAttribute attr;
            attr.id = cudaLaunchAttributeClusterDimension;
            attr.val.clusterDim.x = 1 << k;
            attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
            cfg.gridDim = dim3((sms >> k) << k);
            cfg.blockDim = dim3(C::kThreads);
            cfg.dynamicSmemBytes = C::kSmem;
            cfg.attrs = &attr;
            cfg.numAttrs = 1;
            int found = 0;
            if (cudaOccupancyMaxActiveClusters(&found, wt::weights_kernel<kPacked>, &cfg) != cudaSuccess || found < 1) {
                cudaGetLastError();
                found = -1;
            }
            n = found;
            most[k][dev].store(n, std::memory_order_relaxed);
        }
        if (n < 1) continue;
        const int64_t share = (units + n - 1) / n;
        if (share > wt::kBlock) continue;
        const double t = ((p.q_len + (1 << k) - 1) >> k) * (share + pass) + join;
        if (t < best) {
            best = t;
            *ranks = 1 << k;
            *clusters = n;
        }
    }
}

template <bool kPacked>
static cudaError_t weights_launch(const CUtensorMap& mQ, const CUtensorMap& mRows, const CUtensorMap& mKey, const Problem& p,
                                  wt::Args& a, cudaStream_t st) {
    using C = wt::Cfg<kPacked>;
    cudaError_t e = set_smem(wt::weights_kernel<kPacked>, C::kSmem, g_smem_weights[kPacked]);
    if (e != cudaSuccess) return e;
    int clusters;
    weights_split<kPacked>(p, a.T_max, &a.ranks, &clusters);
    return launch_pdl(wt::weights_kernel<kPacked>, dim3(clusters * a.ranks), dim3(C::kThreads), C::kSmem, st, a.ranks, mQ, mRows, mKey, a);
}

cudaError_t sm100_weights(const Problem& p, bool packed, const void* q_hat, const float* lse, const CacheView& cache,
                          const int32_t* seqlens, float decay, const float* prev, float* weights, int64_t stride_w,
                          int* status, const mla_decode_opts_t* opts, cudaStream_t st) {
    CUtensorMap mQ, mRows, mKey;
    if (!make_map(&mQ, q_hat, kRow, kHeads, (uint64_t)p.B * p.q_len, kRow * 2, (uint64_t)kHeads * kRow * 2, 64, kHeads, 1,
                  CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    const uint64_t es = packed ? 1 : 2;
    const uint64_t stt = (uint64_t)cache.stride_t * es;
    const uint64_t sb = p.B > 1 ? (uint64_t)cache.stride_b * es : stt * (uint64_t)cache.T_max;
    const uint8_t* rows = static_cast<const uint8_t*>(cache.data);
    bool made;
    if (packed) {
        made = make_map_words(&mRows, rows, wt::kRawRow / 2, cache.T_max, p.B, stt, sb, wt::kRawRow / 2, wt::kUnit, 1,
                              CU_TENSOR_MAP_SWIZZLE_NONE) &&
               make_map(&mKey, rows + kPackRope, kRope, cache.T_max, p.B, stt, sb, kRope, wt::kUnit, 1, CU_TENSOR_MAP_SWIZZLE_128B);
    } else {
        made = make_map(&mRows, rows, kRow, cache.T_max, p.B, stt, sb, 64, wt::kTile, 1, CU_TENSOR_MAP_SWIZZLE_128B);
        mKey = mRows;
    }
    if (!made) return cudaErrorInvalidValue;
    wt::Args a;
    a.seqlens = seqlens;
    a.lse = lse;
    a.prev = prev;
    a.weights = weights;
    a.stride_w = stride_w;
    a.decay = decay;
    a.scale_log2 = p.scale * 1.4426950408889634f;
    a.B = p.B;
    a.q_len = p.q_len;
    a.T_max = cache.T_max;
    a.status = status;
    a.wait_limit_ns = (opts && opts->wait_limit_ns > 0) ? (uint64_t)opts->wait_limit_ns : MLA_WAIT_LIMIT_NS;
    a.withhold_tile = (opts && opts->withhold_tile > 0) ? opts->withhold_tile : -1;
    return packed ? weights_launch<true>(mQ, mRows, mKey, p, a, st) : weights_launch<false>(mQ, mRows, mKey, p, a, st);
}

cudaError_t sm100_project_small(const Problem& p, void* attend_workspace, int num_pairs, const void* o_lat,
                                const void* W_UV, void* out, cudaStream_t st) {
    const int rows = p.B * p.q_len;
    if (rows < 1 || rows > kGemvMaxRows) return cudaErrorInvalidValue;
    size_t off_part, off_lse;
    attend_layout(p, num_pairs, &off_part, &off_lse);
    char* ws = static_cast<char*>(attend_workspace);
    ProjectGemvArgs a;
    a.plan = reinterpret_cast<const Plan*>(ws);
    a.o_lat = (const __nv_bfloat16*)o_lat;
    a.part_o = reinterpret_cast<const float*>(ws + off_part);
    a.part_lse = reinterpret_cast<const float*>(ws + off_lse);
    a.W_UV = (const __nv_bfloat16*)W_UV;
    a.rows = rows;
    a.out = (__nv_bfloat16*)out;
    a.status = device_status_ptr();
    if (rows == 1) return project_gemv_launch<1>(a, st);
    if (rows == 2) return project_gemv_launch<2>(a, st);
    if (rows <= 4) return project_gemv_launch<4>(a, st);
    return project_gemv_launch<8>(a, st);
}

}  // namespace mla
