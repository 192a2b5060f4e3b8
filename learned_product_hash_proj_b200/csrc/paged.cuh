// paged.cuh -- plan, workspace layout and device helpers of the dense
// operators: packed prompts and the paged key/value cache.
#pragma once

#include "internal.cuh"
#include "tc.cuh"

namespace mono {

constexpr int kPagedMaxRows = 16384;
constexpr int kPagedMaxCtas = 320;   // CTAs of the one-token attention, two partial results each
constexpr int kPagedHeads = 16;      // query heads of one key/value head that a CTA handles together

// error codes after those of internal.cuh
enum PagedErr : unsigned { kDevErrBadPage = 6, kDevErrBadLen = 7, kDevErrNoPage = 8 };

// 64-bit words at the start of the workspace; the error word sits where record_error expects it
enum PagedCounter { kPagedHeld = 0, kPagedCopied = 1, kPagedShort = 2, kPagedTiles = 3, kPagedErr = kCntErr };

enum PagedRegion {
    kPgCounters = 0,
    kPgMarks,    // first[] uint32, then held[] and whole[] bytes, one per page, padded to 16 pages; all ones: unmarked
    kPgFree,     // [pages] int32 free pages in ascending order (update)
    kPgFresh,    // [rows] int32: position in the free list of each row's first new page
    kPgPairs,    // [max(rows, pages)] int2 (from, to) pages to copy
    kPgPrefix,   // [rows+1] int32 key tiles before each row (one-token attention)
    kPgPartO,    // [2*kPagedMaxCtas, 16, d] fp32 unnormalised partial outputs
    kPgPartML,   // [2*kPagedMaxCtas, 16] float2 (max, sum) of each
    kPgWork,     // [tokens*pack/128 + rows + 1] query tiles of a prompt call (32 bytes each), longest first
    kPgN
};

struct PagedPlan {
    mono_paged_config cfg;
    int es;            // bytes of a stored element
    float scale_log2;  // softmax scale times log2(e)
    size_t off[kPgN];
    size_t ws_bytes;
};

// log2 of the query heads of one key/value head that share a row tile of the bf16 prompt kernel
inline int prompt_pack_log2(const mono_paged_config &c) {
    int log2 = 0;
    while (log2 < 4 && (c.Hq / c.Hkv) % (2 << log2) == 0) ++log2;
    return log2;
}

// query tiles of a prompt call, by the rows of a tile and the heads that share it, over all heads
inline long long prompt_items(const mono_paged_config &c, int n, int total_q) {
    const int pack = c.dtype == MONO_BF16 ? prompt_pack_log2(c) : 0, rows = c.dtype == MONO_BF16 ? 128 >> pack : 64;
    return ((long long)total_q / rows + n) * (c.Hq >> pack);
}

inline size_t marks_bytes(int pages) { return ((size_t)pages + 15) / 16 * 16 * 6; }
inline char *pg_ptr(const PagedPlan &p, void *ws, int region) { return (char *)ws + p.off[region]; }

// A cumulative length read from the caller, kept inside [0, total].
__device__ __forceinline__ int cu_at(const int32_t *cu, int i, int total) { return min(max(cu[i], 0), total); }

// Rows of sequence s: the first and how many, inside [0, total] whatever the caller's lengths say.  Lengths that lead
// outside or do not ascend are recorded.
struct Span {
    int at, n;
};
__device__ __forceinline__ Span cu_span(const int32_t *cu, int s, int total, unsigned long long *counters) {
    const int a = cu[s], b = cu[s + 1];
    if (a < 0 || b < a || b > total) record_error(counters, kDevErrBadLen);
    const int at = min(max(a, 0), total);
    return {at, max(0, min(max(b, 0), total) - at)};
}

// Block-wide exclusive scan of one int per thread (NT threads, a multiple of 32); *total receives the sum.  Sums are
// taken modulo 2^32.  s_w: NT/32 + 1 ints of shared memory, free again after the next __syncthreads.
template <int NT>
__device__ __forceinline__ int block_scan(int v, int *s_w, int *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned x = (unsigned)v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s_w[warp] = (int)x;
    __syncthreads();
    if (warp == 0) {
        unsigned w = lane < NT / 32 ? (unsigned)s_w[lane] : 0u;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        if (lane < NT / 32) s_w[lane] = (int)w;
    }
    __syncthreads();
    *total = s_w[NT / 32 - 1];
    return (int)(x - (unsigned)v + (warp > 0 ? (unsigned)s_w[warp - 1] : 0u));
}

// The sequence and first row of query tile `tile` when every sequence is cut into tiles of `qt` rows, the last
// (with causal masking the longest) tile of each sequence first.  Called by all NT threads; false past the end.
template <int NT>
__device__ __forceinline__ bool find_tile(const int32_t *cu_q, int n, int total_q, int qt, int tile, int *s_w,
                                          int *s_out, int *seq, int *row0, unsigned long long *counters) {
    const int per = (n + NT - 1) / NT;
    const int s0 = min(n, (int)threadIdx.x * per), s1 = min(n, s0 + per);
    if (threadIdx.x == 0) s_out[0] = -1;
    int mine = 0;
    for (int s = s0; s < s1; ++s) mine += (cu_span(cu_q, s, total_q, counters).n + qt - 1) / qt;
    int all;
    int pre = block_scan<NT>(mine, s_w, &all);
    if (tile >= all) return false;
    for (int s = s0; s < s1; ++s) {
        const int t = (cu_span(cu_q, s, total_q, counters).n + qt - 1) / qt;
        if (tile >= pre && tile < pre + t) {
            s_out[0] = s;
            s_out[1] = (t - 1 - (tile - pre)) * qt;
        }
        pre += t;
    }
    __syncthreads();
    *seq = s_out[0];
    *row0 = s_out[1];
    return *seq >= 0;  // (every tile has its sequence unless lengths that do not ascend overflow the count)
}

cudaError_t launch_paged_append(const PagedPlan &p, int layer, int n, int total, const void *K, const void *V,
                                const int32_t *cu, const int32_t *table, const int32_t *lens, void *Kp, void *Vp,
                                void *ws, cudaStream_t s);
cudaError_t launch_paged_update(const PagedPlan &p, int n_in, const int32_t *table, const int32_t *lens, int n_out,
                                const int32_t *parents, const int32_t *grow, int32_t *table_out, int32_t *lens_out,
                                void *Kp, void *Vp, void *ws, cudaStream_t s);
cudaError_t launch_paged_compact(const PagedPlan &p, int n, const int32_t *table, const int32_t *lens,
                                 int32_t *table_out, void *Kp, void *Vp, void *ws, cudaStream_t s);
cudaError_t launch_paged_attend(const PagedPlan &p, int layer, int n, const void *Q, const int32_t *table,
                                const int32_t *lens, const void *Kp, const void *Vp, void *O, void *ws,
                                cudaStream_t s);
cudaError_t launch_prompt_tc(const PagedPlan &p, int n, int total_q, int total_k, const void *Q, const void *K,
                             const void *V, const int32_t *cu_q, const int32_t *cu_k, void *O, void *ws,
                             cudaStream_t s);
cudaError_t launch_prompt_simt(const PagedPlan &p, int n, int total_q, int total_k, const void *Q, const void *K,
                               const void *V, const int32_t *cu_q, const int32_t *cu_k, void *O, void *ws,
                               cudaStream_t s);

// A kernel launched so that it may start while the kernel before it on the
// stream, this library's or not, still ends: every kernel launched so waits for
// its predecessor itself (tc::grid_dep_wait) before it touches global memory.
// (Its inputs are not __restrict__: loads that the compiler may take for
// invariant could move ahead of that wait.)
template <typename... KArgs, typename... Args>
inline cudaError_t launch_after_cluster(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                                        int cluster, Args... args) {
    cudaLaunchConfig_t lc = {};
    lc.gridDim = grid;
    lc.blockDim = block;
    lc.dynamicSmemBytes = smem;
    lc.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    lc.attrs = at;
    lc.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&lc, kern, (KArgs)args...);
}
template <typename... KArgs, typename... Args>
inline cudaError_t launch_after(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                                Args... args) {
    return launch_after_cluster(kern, grid, block, smem, s, 1, args...);
}

}  // namespace mono

struct mono_paged_plan_s {
    mono::PagedPlan p;
};
