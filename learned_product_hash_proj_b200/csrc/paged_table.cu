// paged_table.cu -- the paged cache's bookkeeping: writing new keys and
// values into pages, the page table's step (fork, continue, cut back, drop)
// and closing the pool's holes, each with the page copies it needs.
//
// All of it is integer work and copies, so results do not depend on timing:
// marks are set by idempotent stores or atomicMin, and every list is built by
// a scan in ascending order.
#include <limits.h>

#include <algorithm>

#include "paged.cuh"

namespace mono {

namespace {

constexpr unsigned kNoRow = 0xffffffffu;

struct Marks {
    unsigned *first;       // lowest output row whose kept tokens end inside the page; compact: the page's new id
    unsigned char *held;   // 0: an input row holds the page
    unsigned char *whole;  // 0: an output row goes on past the page
};

Marks marks_of(const PagedPlan &p, void *ws) {
    char *m = pg_ptr(p, ws, kPgMarks);
    const size_t n = ((size_t)p.cfg.pages + 15) / 16 * 16;
    return {(unsigned *)m, (unsigned char *)m + 4 * n, (unsigned char *)m + 5 * n};
}

// a row's length, inside [0, width*page]
__device__ __forceinline__ int len_at(const int32_t *lens, int i, int cap, unsigned long long *counters) {
    const int n = lens[i];
    if (n < 0 || n > cap) record_error(counters, kDevErrBadLen);
    return min(max(n, 0), cap);
}

// what an output row of the update takes from its parent: kept tokens and length
struct RowStep {
    int parent, kept, len;
};
__device__ __forceinline__ RowStep row_step(const int32_t *lens, const int32_t *parents, const int32_t *grow, int i,
                                            int n_in, int cap, unsigned long long *counters) {
    RowStep r;
    r.parent = parents[i];
    if (r.parent < -1 || r.parent >= n_in) {
        record_error(counters, kDevErrBadLen);
        r.parent = -1;
    }
    const int n = r.parent >= 0 ? len_at(lens, r.parent, cap, counters) : 0;
    const long long after = (long long)n + grow[i];
    if (after > cap) record_error(counters, kDevErrBadLen);
    r.len = (int)min(max(after, 0ll), (long long)cap);
    r.kept = min(n, r.len);
    return r;
}

// ---------------------------------------------------------------------------
// marks: one block per input row, then one per output row
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(128) k_page_mark(const int32_t *__restrict__ table, const int32_t *__restrict__ lens,
                                                   const int32_t *__restrict__ parents,
                                                   const int32_t *__restrict__ grow, Marks mk, int n_in, int width,
                                                   int page, int pages, unsigned long long *__restrict__ counters) {
    tc::grid_dep_launch();
    const int cap = width * page;
    if ((int)blockIdx.x < n_in) {
        const int i = blockIdx.x;
        const int n = (len_at(lens, i, cap, counters) + page - 1) / page;
        for (int e = threadIdx.x; e < n; e += 128) {
            const int id = table[(size_t)i * width + e];
            if ((unsigned)id < (unsigned)pages) mk.held[id] = 0;
            else record_error(counters, kDevErrBadPage);
        }
        return;
    }
    const int i = blockIdx.x - n_in;
    const RowStep r = row_step(lens, parents, grow, i, n_in, cap, counters);
    if (r.parent < 0) return;
    const int full = r.kept / page;
    for (int e = threadIdx.x; e < full; e += 128) {
        const int id = table[(size_t)r.parent * width + e];
        if ((unsigned)id < (unsigned)pages) mk.whole[id] = 0;
    }
    if (threadIdx.x == 0 && r.kept % page) {
        const int id = table[(size_t)r.parent * width + full];
        if ((unsigned)id < (unsigned)pages) atomicMin(&mk.first[id], (unsigned)i);
    }
}

// whether output row i needs its own copy of the page `id` that its kept tokens end in
__device__ __forceinline__ bool takes_copy(const Marks &mk, int id, int pages, int i) {
    return (unsigned)id < (unsigned)pages && (mk.whole[id] == 0 || mk.first[id] != (unsigned)i);
}

// Ascending list of the pages below `limit` whose held byte says `want_held`, by one block of 1024 threads;
// returns their number.  Each thread takes runs of 16 pages, one 16-byte load each.
template <typename F>
__device__ __forceinline__ int list_pages(const unsigned char *held, int from, int limit, bool want_held, int *s_w,
                                          F put) {
    int base = 0;
    for (int p0 = from & ~15; p0 < limit; p0 += 16 * 1024) {
        const int p = p0 + 16 * threadIdx.x;
        unsigned bits = 0;
        if (p < limit) {
            const uint4 v = *(const uint4 *)(held + p);  // the marks are padded to 16 pages
            const unsigned w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const int id = p + k;
                const bool is_held = ((w[k >> 2] >> (8 * (k & 3))) & 0xffu) == 0;
                if (id >= from && id < limit && is_held == want_held) bits |= 1u << k;
            }
        }
        int total;
        int at = base + block_scan<1024>(__popc(bits), s_w, &total);
        while (bits) {
            put(at++, p + __ffs(bits) - 1);
            bits &= bits - 1;
        }
        base += total;
        __syncthreads();
    }
    return base;
}

// ---------------------------------------------------------------------------
// update: free list, each row's share of it, and the pages to copy.  A block of 1024 threads; the marks are complete.
// fresh[i]: where row i's new pages start in the free list, as its complement if the first is a copy of its tail.
// The rows may ask for more than 2^31 pages together, though for less than 2^32 (rows * width of a plan): positions
// are counted without a sign, and those behind the pool, which no page answers to, are stored as `pages`.
// ---------------------------------------------------------------------------
template <typename F, typename G>
__device__ __forceinline__ void assign_pages(F step_of, G tail_of, const Marks &mk, int32_t *freelist, int32_t *fresh,
                                             int2 *pairs, int n_out, int page, int pages, unsigned long long *counters,
                                             int *s_w) {
    const int nfree = list_pages(mk.held, 0, pages, false, s_w, [&](int at, int id) { freelist[at] = id; });
    __syncthreads();  // the list's stores are read by other threads below
    unsigned base = 0;
    int ncopy = 0;
    for (int i0 = 0; i0 < n_out; i0 += 1024) {
        const int i = i0 + threadIdx.x;
        int need = 0, tail = -1;
        bool copy = false;
        if (i < n_out) {
            const RowStep r = step_of(i);
            need = (r.len + page - 1) / page - (r.kept + page - 1) / page;
            if (r.kept % page) {
                tail = tail_of(i, r);
                copy = takes_copy(mk, tail, pages, i);
            }
        }
        int total, ctotal;
        const unsigned pos = base + (unsigned)block_scan<1024>(need + (copy ? 1 : 0), s_w, &total);
        const int at = (int)min(pos, (unsigned)pages);
        __syncthreads();
        if (i < n_out) fresh[i] = copy ? ~at : at;
        copy = copy && at < nfree;  // a row's copied page is its first new one
        const int cat = ncopy + block_scan<1024>(copy ? 1 : 0, s_w, &ctotal);
        __syncthreads();
        if (copy) pairs[cat] = make_int2(tail, freelist[at]);
        base += (unsigned)total;
        ncopy += ctotal;
    }
    if (threadIdx.x == 0) {
        counters[kPagedHeld] = (unsigned long long)(pages - nfree);
        counters[kPagedCopied] = (unsigned long long)ncopy;
        const unsigned over = base > (unsigned)nfree ? base - (unsigned)nfree : 0u;
        counters[kPagedShort] = (unsigned long long)min(over, (unsigned)INT_MAX);
        if (over) record_error(counters, kDevErrNoPage);
    }
}

// ---------------------------------------------------------------------------
// compact: the held pages from L on and the holes below L, paired in order; a moved page's new id in mk.first.
// A block of 1024 threads.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void pair_holes(const Marks &mk, int2 *pairs, int pages, unsigned long long *counters,
                                           int *s_w) {
    const int live = list_pages(mk.held, 0, pages, true, s_w, [](int, int) {});
    const int holes = list_pages(mk.held, 0, live, false, s_w, [&](int at, int id) { pairs[at].y = id; });
    __syncthreads();
    // as many held pages lie at or above L as there are holes below it
    list_pages(mk.held, live, pages, true, s_w, [&](int at, int id) {
        pairs[at].x = id;
        mk.first[id] = (unsigned)pairs[at].y;
    });
    if (threadIdx.x == 0) {
        counters[kPagedHeld] = (unsigned long long)live;
        counters[kPagedCopied] = (unsigned long long)holes;
        counters[kPagedShort] = 0;
    }
}

// large pools and tables: marks in the workspace, set by k_page_mark
__global__ void __launch_bounds__(1024) k_page_assign(const int32_t *table,
                                                      const int32_t *lens,
                                                      const int32_t *parents,
                                                      const int32_t *grow, Marks mk, int32_t *freelist,
                                                      int32_t *fresh, int2 *pairs, int n_in, int n_out, int width,
                                                      int page, int pages, unsigned long long *counters) {
    __shared__ int s_w[33];
    tc::grid_dep_launch();
    tc::grid_dep_wait();
    assign_pages([&](int i) { return row_step(lens, parents, grow, i, n_in, width * page, counters); },
                 [&](int, const RowStep &r) { return table[(size_t)r.parent * width + r.kept / page]; }, mk, freelist,
                 fresh, pairs, n_out, page, pages, counters, s_w);
}

__global__ void __launch_bounds__(1024) k_page_holes(Marks mk, int2 *pairs, int pages, unsigned long long *counters) {
    __shared__ int s_w[33];
    tc::grid_dep_launch();
    tc::grid_dep_wait();
    pair_holes(mk, pairs, pages, counters, s_w);
}

// Small pools and tables: marks and row steps in shared memory, and all of the planning in one block, a warp per row.
// (Four rows over 256 pages: with clearing, marking and assigning as three launches 12.3 us, so 7.2, the copies
// included; at 160 rows over 4096 pages both take 20.2 us, 12 of them the copies of 38 pages of 1 MB.)
constexpr int kPlanPages = 24576;          // marks: 6 bytes each
constexpr int kPlanRows = 2048;            // 16 bytes each of the output's, 4 each of the input's
constexpr long long kPlanEntries = 65536;  // table entries that the block looks at, at most

size_t plan_smem(int pages, int n_in, int n_out) {
    return marks_bytes(pages) + (size_t)n_out * (sizeof(RowStep) + 4) + (size_t)n_in * 4;
}
bool plan_small(const mono_paged_config &c, int n_in, int n_out) {
    return c.pages <= kPlanPages && n_in <= kPlanRows && n_out <= kPlanRows && (long long)(n_in + n_out) * c.width <= kPlanEntries;
}

template <bool UPDATE>
__global__ void __launch_bounds__(1024) k_page_plan(const int32_t *table,
                                                    const int32_t *lens,
                                                    const int32_t *parents,
                                                    const int32_t *grow, unsigned *first, int32_t *freelist,
                                                    int32_t *fresh, int2 *pairs, int n_in, int n_out, int width,
                                                    int page, int pages, unsigned long long *counters) {
    extern __shared__ __align__(16) uint8_t s_marks[];
    __shared__ int s_w[33];
    const int padded = (pages + 15) / 16 * 16, cap = width * page;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Marks mk = {(unsigned *)s_marks, s_marks + 4 * padded, s_marks + 5 * padded};
    RowStep *s_step = (RowStep *)(s_marks + 6 * padded);
    int *s_tail = (int *)(s_step + n_out), *s_np = s_tail + n_out;  // pages that kept tokens end in, pages of input rows
    for (int i = threadIdx.x; i < padded * 6 / 16; i += 1024) ((uint4 *)s_marks)[i] = make_uint4(~0u, ~0u, ~0u, ~0u);
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    for (int i = threadIdx.x; i < n_in; i += 1024) s_np[i] = (len_at(lens, i, cap, counters) + page - 1) / page;
    if (UPDATE)
        for (int i = threadIdx.x; i < n_out; i += 1024)
            s_step[i] = row_step(lens, parents, grow, i, n_in, cap, counters);
    __syncthreads();
#pragma unroll 4
    for (int i = warp; i < n_in; i += 32) {
        const int np = s_np[i];
        for (int e = lane; e < np; e += 32) {
            const int id = table[i * width + e];
            if ((unsigned)id < (unsigned)pages) mk.held[id] = 0;
            else record_error(counters, kDevErrBadPage);
        }
    }
    if (UPDATE) {
#pragma unroll 4
        for (int i = warp; i < n_out; i += 32) {
            const RowStep r = s_step[i];
            const int full = r.kept / page, np = (r.kept + page - 1) / page;  // kept is 0 without a parent
            for (int e = lane; e < np; e += 32) {
                const int id = table[r.parent * width + e];
                if (e == full) s_tail[i] = id;
                if ((unsigned)id >= (unsigned)pages) continue;
                if (e < full) mk.whole[id] = 0;
                else atomicMin(&mk.first[id], (unsigned)i);
            }
        }
        __syncthreads();
        assign_pages([&](int i) { return s_step[i]; }, [&](int i, const RowStep &) { return s_tail[i]; }, mk, freelist,
                     fresh, pairs, n_out, page, pages, counters, s_w);
    } else {
        __syncthreads();
        pair_holes(mk, pairs, pages, counters, s_w);
        __syncthreads();
        for (int i = threadIdx.x; i < pages; i += 1024) first[i] = mk.first[i];
    }
}

// ---------------------------------------------------------------------------
// page copies: every (pair, layer, K or V) as chunks of 16 KB, spread over the grid
// ---------------------------------------------------------------------------
constexpr int kCopyChunk = 16384;

__device__ __forceinline__ void copy_pages(const int2 *pairs, int npairs, char *Kp, char *Vp, int layers, int pages,
                                           int page_bytes, int block, int nblocks) {
    const int per = (page_bytes + kCopyChunk - 1) / kCopyChunk;
    const long long total = (long long)npairs * layers * 2 * per;
    for (long long w = block; w < total; w += nblocks) {
        const int c = (int)(w % per);
        const long long r = w / per;
        const int kv = (int)(r & 1), layer = (int)((r >> 1) % layers);
        const int2 pr = pairs[(r >> 1) / layers];
        char *pool = (kv ? Vp : Kp) + (size_t)layer * pages * page_bytes;
        const int n16 = (min(page_bytes - c * kCopyChunk, kCopyChunk)) / 16;
        const uint4 *src = (const uint4 *)(pool + (size_t)pr.x * page_bytes + c * kCopyChunk);
        uint4 *dst = (uint4 *)(pool + (size_t)pr.y * page_bytes + c * kCopyChunk);
        constexpr int N = kCopyChunk / (256 * 16);
        uint4 v[N];
#pragma unroll
        for (int k = 0; k < N; ++k)
            if ((int)threadIdx.x + 256 * k < n16) v[k] = __ldcs(src + threadIdx.x + 256 * k);
#pragma unroll
        for (int k = 0; k < N; ++k)
            if ((int)threadIdx.x + 256 * k < n16) __stcs(dst + threadIdx.x + 256 * k, v[k]);
    }
}

// The first row_blocks blocks write the table, `per` threads a row, the others copy pages.
inline int threads_per_row(int width) { return width <= 256 ? 32 : 256; }

// update
__global__ void __launch_bounds__(256) k_page_apply(const int32_t *table, const int32_t *lens,
                                                    const int32_t *parents,
                                                    const int32_t *grow, int32_t *freelist,
                                                    int32_t *fresh, int2 *pairs, int32_t *table_out,
                                                    int32_t *lens_out, char *Kp, char *Vp, int n_in,
                                                    int n_out, int width, int page, int pages, int layers,
                                                    int page_bytes, int row_blocks, int per,
                                                    unsigned long long *counters) {
    tc::grid_dep_wait();
    const int nfree = pages - (int)counters[kPagedHeld];
    const int cap = width * page;
    if ((int)blockIdx.x >= row_blocks) {
        copy_pages(pairs, (int)counters[kPagedCopied], Kp, Vp, layers, pages, page_bytes, blockIdx.x - row_blocks,
                   gridDim.x - row_blocks);
        return;
    }
    const int i = blockIdx.x * (256 / per) + threadIdx.x / per, lane = threadIdx.x % per;
    if (i < n_out) {
        const RowStep r = row_step(lens, parents, grow, i, n_in, cap, counters);
        const int nkeep = (r.kept + page - 1) / page, nall = (r.len + page - 1) / page;
        const int f = fresh[i], at = f < 0 ? ~f : f, first_new = nkeep - (f < 0 ? 1 : 0);
        for (int e = lane; e < width; e += per) {
            int id = -1;
            if (e < first_new) {
                id = table[(size_t)r.parent * width + e];
                if ((unsigned)id >= (unsigned)pages) id = -1;
            } else if (e < nall) {
                const int k = at + e - first_new;
                if (k < nfree) id = freelist[k];
            }
            table_out[(size_t)i * width + e] = id;
        }
        if (lane == 0) lens_out[i] = r.len;
    }
}

// compact: the table with the new ids and the copies
__global__ void __launch_bounds__(256) k_page_move(const int32_t *table, const int32_t *lens,
                                                   const unsigned *first, int2 *pairs, int32_t *table_out,
                                                   char *Kp, char *Vp, int n, int width, int page, int pages,
                                                   int layers, int page_bytes, int row_blocks, int per,
                                                   unsigned long long *counters) {
    tc::grid_dep_wait();
    if ((int)blockIdx.x >= row_blocks) {
        copy_pages(pairs, (int)counters[kPagedCopied], Kp, Vp, layers, pages, page_bytes, blockIdx.x - row_blocks,
                   gridDim.x - row_blocks);
        return;
    }
    const int i = blockIdx.x * (256 / per) + threadIdx.x / per, lane = threadIdx.x % per;
    if (i < n) {
        const int nall = (len_at(lens, i, width * page, counters) + page - 1) / page;
        for (int e = lane; e < width; e += per) {
            int id = e < nall ? table[(size_t)i * width + e] : -1;
            if ((unsigned)id >= (unsigned)pages) id = -1;
            else if (first[id] != kNoRow) id = (int)first[id];
            table_out[(size_t)i * width + e] = id;
        }
    }
}

// ---------------------------------------------------------------------------
// append: T tokens per block.  The block first asks for its tokens' rows of K and V, up to 16 KB each, which lie in
// order; while they are under way a warp finds each token's row by a 32-way search of the cumulative lengths and its
// place through the table; then the rows go to their head-major pages (each (token, head) row of d elements is
// contiguous on both sides).  A thread steps through the pieces by a fixed stride, without divisions.
// ---------------------------------------------------------------------------
constexpr int kAppendMax = 64;     // tokens of a block
// (volatile: it stays behind the wait for the kernel before)
__device__ __forceinline__ uint4 ld_stream(const uint4 *p) {
    uint4 v;
    asm volatile("ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

constexpr int kAppendBatch = 4;    // 16-byte pieces of K, and of V, that a thread has under way

__global__ void __launch_bounds__(256, 3) k_page_append(const uint4 *K, const uint4 *V,
                                                     const int32_t *cu, const int32_t *table,
                                                     const int32_t *lens, uint4 *Kp, uint4 *Vp, int n,
                                                     int total, int T, int width, int page, int pages, int Hkv,
                                                     int per_log2, unsigned long long *counters) {
    __shared__ long long s_at[kAppendMax];  // first row (page, head 0) of the token in the pool, or -1
    tc::grid_dep_wait();
    const int t0 = blockIdx.x * T, nt = min(T, total - t0);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tok = Hkv << per_log2, pieces = nt * tok;  // 16-byte pieces of a token, and of all
    const size_t from = (size_t)t0 * tok;
    uint4 k[kAppendBatch], v[kAppendBatch];
    auto load = [&](int x0) {
#pragma unroll
        for (int j = 0; j < kAppendBatch; ++j) {
            const int x = x0 + 256 * j;
            if (x < pieces) {
                k[j] = ld_stream(K + from + x);
                v[j] = ld_stream(V + from + x);
            }
        }
    };
    load(threadIdx.x);
    for (int i = warp; i < nt; i += 8) {
        const int t = t0 + i;
        // the last row whose first token is at or before t: [lo, hi) narrows to one
        int lo = 0, hi = n;
        while (hi - lo > 1) {
            const int step = (hi - lo + 31) / 32;
            const int at = lo + lane * step;
            const bool at_or_before = at < hi && cu_at(cu, at, total) <= t;
            const unsigned b = __ballot_sync(0xffffffffu, at_or_before);
            if (!b) { hi = lo; break; }
            lo += (31 - __clz(b)) * step;
            hi = min(hi, lo + step);
        }
        if (lane == 0) {
            long long at = -1;
            if (hi > lo) {
                const int a = cu_at(cu, lo, total), b = cu_at(cu, lo + 1, total);
                if (t >= a && t < b) {
                    const long long pos = (long long)lens[lo] - (b - a) + (t - a);
                    if (pos < 0 || pos >= (long long)width * page) {
                        record_error(counters, kDevErrBadLen);
                    } else {
                        const int id = table[(size_t)lo * width + (int)(pos / page)];
                        if ((unsigned)id < (unsigned)pages) at = (long long)id * Hkv * page + (int)(pos % page);
                        else record_error(counters, kDevErrBadPage);
                    }
                }
            }
            s_at[i] = at;
        }
    }
    __syncthreads();
    // piece y of token i, carried along as x advances by 256
    const int di = 256 / tok, dy = 256 - di * tok, mask = (1 << per_log2) - 1;
    int i = threadIdx.x / tok, y = threadIdx.x - i * tok;
    for (int x0 = threadIdx.x; x0 < pieces; x0 += 256 * kAppendBatch) {
        if (x0 != (int)threadIdx.x) load(x0);
#pragma unroll
        for (int j = 0; j < kAppendBatch; ++j) {
            if (x0 + 256 * j < pieces) {
                const long long at = s_at[i];
                if (at >= 0) {
                    const size_t to = ((size_t)(at + (long long)(y >> per_log2) * page) << per_log2) + (y & mask);
                    Kp[to] = k[j];
                    Vp[to] = v[j];
                }
            }
            i += di;
            y += dy;
            if (y >= tok) {
                y -= tok;
                ++i;
            }
        }
    }
    for (int r = blockIdx.x * 256 + threadIdx.x; r < n; r += gridDim.x * 256) cu_span(cu, r, total, counters);
}

// The attribute is the kernel's, not the call's: host threads whose calls meet all set the largest size of any call.
template <typename F>
cudaError_t allow_plan_smem(F *kern, size_t smem) {
    if (smem <= 48 * 1024) return cudaSuccess;
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)plan_smem(kPlanPages, kPlanRows, kPlanRows));
}

cudaError_t sm_count(int *sms) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    return cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
}

}  // namespace

cudaError_t launch_paged_append(const PagedPlan &p, int layer, int n, int total, const void *K, const void *V,
                                const int32_t *cu, const int32_t *table, const int32_t *lens, void *Kp, void *Vp,
                                void *ws, cudaStream_t s) {
    const mono_paged_config &c = p.cfg;
    int sms = 0;
    cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    const int row_bytes = c.d * p.es;
    const size_t layer_bytes = (size_t)c.pages * c.Hkv * c.page * row_bytes;
    int per_log2 = 0;
    while ((16 << per_log2) < row_bytes) ++per_log2;
    // tokens per block: one batch of every thread, fewer where the call would not fill the SMs
    int T = std::max(1, std::min(kAppendMax, (256 * kAppendBatch) / (c.Hkv << per_log2)));
    while (T > 1 && (total + T - 1) / T < 2 * sms) T /= 2;
    e = launch_after(k_page_append, dim3((total + T - 1) / T), dim3(256), 0, s, (const uint4 *)K, (const uint4 *)V, cu,
                     table, lens, (uint4 *)((char *)Kp + layer * layer_bytes),
                     (uint4 *)((char *)Vp + layer * layer_bytes), n, total, T, c.width, c.page, c.pages, c.Hkv, per_log2,
                     (unsigned long long *)pg_ptr(p, ws, kPgCounters));
    count_launches(1);
    return e;
}

cudaError_t launch_paged_update(const PagedPlan &p, int n_in, const int32_t *table, const int32_t *lens, int n_out,
                                const int32_t *parents, const int32_t *grow, int32_t *table_out, int32_t *lens_out,
                                void *Kp, void *Vp, void *ws, cudaStream_t s) {
    const mono_paged_config &c = p.cfg;
    const Marks mk = marks_of(p, ws);
    unsigned long long *counters = (unsigned long long *)pg_ptr(p, ws, kPgCounters);
    int32_t *freelist = (int32_t *)pg_ptr(p, ws, kPgFree), *fresh = (int32_t *)pg_ptr(p, ws, kPgFresh);
    int2 *pairs = (int2 *)pg_ptr(p, ws, kPgPairs);
    const int page_bytes = c.Hkv * c.page * c.d * p.es;
    int sms = 0;
    cudaError_t e;
    if ((e = sm_count(&sms)) != cudaSuccess) return e;
    const bool small = plan_small(c, n_in, n_out);
    if (small) {
        const size_t smem = plan_smem(c.pages, n_in, n_out);
        if ((e = allow_plan_smem(k_page_plan<true>, smem)) != cudaSuccess) return e;
        if ((e = launch_after(k_page_plan<true>, dim3(1), dim3(1024), smem, s, table, lens, parents, grow,
                              (unsigned *)nullptr, freelist, fresh, pairs, n_in, n_out, c.width, c.page, c.pages,
                              counters)) != cudaSuccess)
            return e;
    } else {
        if ((e = cudaMemsetAsync(mk.first, 0xff, marks_bytes(c.pages), s)) != cudaSuccess) return e;
        k_page_mark<<<n_in + n_out, 128, 0, s>>>(table, lens, parents, grow, mk, n_in, c.width, c.page, c.pages,
                                                 counters);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        if ((e = launch_after(k_page_assign, dim3(1), dim3(1024), 0, s, table, lens, parents, grow, mk, freelist, fresh,
                              pairs, n_in, n_out, c.width, c.page, c.pages, counters)) != cudaSuccess)
            return e;
    }
    // At most one copied page per row, few of them in use: 16 CTAs per SM, which take chunks in turn.  (64 per SM: a
    // batch of 160 rows with 38 copies 20.0 -> 21.4 us, most CTAs finding nothing.)
    const long long chunks = (long long)n_out * c.layers * 2 * ((page_bytes + kCopyChunk - 1) / kCopyChunk);
    const int grid = (int)std::min<long long>(chunks, 16ll * sms);
    const int per = threads_per_row(c.width), row_blocks = (n_out + 256 / per - 1) / (256 / per);
    if ((e = launch_after(k_page_apply, dim3(row_blocks + grid), dim3(256), 0, s, table, lens, parents, grow, freelist,
                          fresh, pairs, table_out, lens_out, (char *)Kp, (char *)Vp, n_in, n_out, c.width, c.page,
                          c.pages, c.layers, page_bytes, row_blocks, per, counters)) != cudaSuccess)
        return e;
    count_launches(small ? 2 : 3);
    return cudaSuccess;
}

cudaError_t launch_paged_compact(const PagedPlan &p, int n, const int32_t *table, const int32_t *lens,
                                 int32_t *table_out, void *Kp, void *Vp, void *ws, cudaStream_t s) {
    const mono_paged_config &c = p.cfg;
    const Marks mk = marks_of(p, ws);
    unsigned long long *counters = (unsigned long long *)pg_ptr(p, ws, kPgCounters);
    int2 *pairs = (int2 *)pg_ptr(p, ws, kPgPairs);
    const int page_bytes = c.Hkv * c.page * c.d * p.es;
    int sms = 0;
    cudaError_t e;
    if ((e = sm_count(&sms)) != cudaSuccess) return e;
    const bool small = plan_small(c, n, 0);
    if (small) {
        const size_t smem = plan_smem(c.pages, n, 0);
        if ((e = allow_plan_smem(k_page_plan<false>, smem)) != cudaSuccess) return e;
        const int32_t *none = nullptr;
        if ((e = launch_after(k_page_plan<false>, dim3(1), dim3(1024), smem, s, table, lens, none, none, mk.first,
                              (int32_t *)nullptr, (int32_t *)nullptr, pairs, n, 0, c.width, c.page, c.pages, counters)) !=
            cudaSuccess)
            return e;
    } else {
        if ((e = cudaMemsetAsync(mk.first, 0xff, marks_bytes(c.pages), s)) != cudaSuccess) return e;
        k_page_mark<<<n, 128, 0, s>>>(table, lens, (const int32_t *)nullptr, (const int32_t *)nullptr, mk, n, c.width,
                                      c.page, c.pages, counters);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        if ((e = launch_after(k_page_holes, dim3(1), dim3(1024), 0, s, mk, pairs, c.pages, counters)) != cudaSuccess)
            return e;
    }
    // 64 CTAs per SM, most of them with one chunk: 700 pages of 0.5 MB 122 us, with 8 per SM 133 us
    const long long moves = std::min<long long>(c.pages / 2, (long long)n * c.width);
    const long long chunks = moves * c.layers * 2 * ((page_bytes + kCopyChunk - 1) / kCopyChunk);
    const int grid = (int)std::min<long long>(chunks, 64ll * sms);
    const int per = threads_per_row(c.width), row_blocks = (n + 256 / per - 1) / (256 / per);
    if ((e = launch_after(k_page_move, dim3(row_blocks + grid), dim3(256), 0, s, table, lens, mk.first, pairs, table_out,
                          (char *)Kp, (char *)Vp, n, c.width, c.page, c.pages, c.layers, page_bytes, row_blocks, per,
                          counters)) != cudaSuccess)
        return e;
    count_launches(small ? 2 : 3);
    return cudaSuccess;
}

}  // namespace mono
