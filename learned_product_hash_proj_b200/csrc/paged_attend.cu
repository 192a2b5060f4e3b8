// paged_attend.cu -- attention of one new token per sequence over its paged
// key/value cache.
//
//   o_h = sum_j softmax_j(scale <q_h, k_j>) v_j     over the row's tokens j
//
// Every key and value is used by the Hq/Hkv query heads of its group only, so
// the kernel is bound by reading the pages.  The work of a call is the list of
// key tiles of every (row, kv head, chunk of 16 query heads), in that order;
// the grid's CTAs take equal runs of it, whatever the lengths, so that a batch
// of very different lengths, or one long sequence, keeps every SM reading.  A
// producer warp follows the table and brings each tile's K and V pages in by
// TMA (128-byte swizzle) through a ring of shared-memory stages, ahead of
// four consumer warps that take a quarter of the tile's keys each with a
// running maximum and sum of their own.  Where a run covers only part of a
// (row, head), its result goes to the workspace as (unnormalised o, max, sum)
// in fp32, and a second kernel joins the parts.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>

#include "paged.cuh"

namespace mono {

namespace {

using bf16 = __nv_bfloat16;

constexpr int kThreads = 160;  // 4 consumer warps and the producer

template <typename T, int D>
struct Shape {
    static constexpr int ES = sizeof(T);
    // keys per tile: 16 KB of K (bf16, d = 64 in tiles of 64 keys: 374 us where 128 take 326; 8 rows of 65,536
    // tokens, 16 heads)
    static constexpr int TILE = 16 * 1024 / (D * ES);
    static constexpr int SL = TILE / 4;                   // keys per consumer warp
    static constexpr int SLICE = SL < 16 ? SL : 16;       // that it takes at a time
    static constexpr int EB = 128 / ES;                   // elements per 128-byte block of a row
    static constexpr int NB = D / EB;                     // blocks per row
    static constexpr int KB = TILE * D * ES;              // bytes of a K (or V) tile: [NB][TILE][128]
    // Bytes under way: with 96 KB per CTA (two per SM) the SMs' shares of the memory drift apart, with equal work the
    // last CTA ended 14 % behind the middle one, with 64 KB 4 % (16 rows of 65,536 tokens, 4 heads of 128: 326 and
    // 315 us).  fp32 rows, whose tiles take longer to work off, prefer 96 KB (165 and 162 us).
    static constexpr int STAGES = (ES == 2 ? 64 : 96) * 1024 / (2 * KB);
    static constexpr int RING = STAGES * 2 * KB;
    static constexpr int MERGE = 2 * kPagedHeads * D * 4;  // two warps' outputs; fp32: q and probabilities meanwhile
    static constexpr int BYTES = RING + MERGE + 512;        // and the Small below: two CTAs per SM at most sizes
};

// the small shared variables, behind the ring and the join buffer
struct Small {
    uint64_t full[6], empty[6];
    float2 ml[2][kPagedHeads];
    int mask[6];  // which pages of the stage's tile were there to be read
    int scan[kThreads / 32 + 1], start[3];
};
static_assert(sizeof(Small) <= 512, "behind the ring");

struct Maps {
    CUtensorMap k, v;
};

struct Args {
    const void *q;
    const int32_t *table, *lens;
    void *o;
    float *part_o;
    float2 *part_ml;
    int32_t *prefix;
    unsigned long long *counters;
    int n, Hq, Hkv, G, HC, width, page, pages;
    float scale_log2;
};

__device__ __forceinline__ int row_len(const Args &a, int r) { return min(max(a.lens[r], 0), a.width * a.page); }

// sync of the four consumer warps
__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
// c (16x8 fp32) += a (16x16) b (16x8)
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// The state of one consumer warp over one (row, head chunk): running maximum (in units of log2), sum and
// unnormalised output of its heads.  The warps' states of a segment are joined in shared memory.

// bf16: S = Q K^T and O = P V by m16n8k16, the 16 rows being the query heads.  P goes in as two bf16 terms (16
// significant bits; one term would round each probability to 8 bits), which costs nothing here: the tensor pipe is
// idle most of the time.
template <int D>
struct StateBf16 {
    static constexpr int NT = D / 8;
    uint32_t q[D / 16][4];
    float o[NT][4];
    float m[2], l[2];

    __device__ __forceinline__ void begin(const Args &a, int row, int h0, int nh, uint8_t *, int lane, int) {
        const bf16 *Q = (const bf16 *)a.q + ((size_t)row * a.Hq + h0) * D;
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int h = g + 8 * (x & 1), c = 16 * k + 2 * t + 8 * (x >> 1);
                q[k][x] = h < nh ? *(const uint32_t *)(Q + (size_t)h * D + c) : 0u;
            }
#pragma unroll
        for (int i = 0; i < NT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
    }

    // keys k0 .. k0+15 of the tile, the first `valid` (> 0) of which exist
    __device__ __forceinline__ void tile(uint8_t *sK, uint8_t *sV, int k0, int valid, float scale, uint8_t *, int lane,
                                         int) {
        using S = Shape<bf16, D>;
        if (valid < 16) {  // whatever the page holds behind the row's end must not meet a zero probability
            for (int i = lane; i < (16 - valid) * S::NB * 8; i += 32) {
                const int c = i & 7, b = (i >> 3) % S::NB, r = k0 + valid + (i >> 3) / S::NB;
                *(uint4 *)(sV + b * (S::TILE * 128) + r * 128 + 16 * c) = make_uint4(0, 0, 0, 0);
            }
            __syncwarp();
        }
        float s[2][4] = {};
        {
            // matrices of an x4 load: keys 0-7 and 8-15 (lane bit 4) x the two halves of 16 elements (lane bit 3)
            const int r = k0 + (lane & 7) + ((lane >> 4) << 3);
            const uint32_t base = tc::smem_u32(sK) + r * 128;
            const int hi = (lane >> 3) & 1;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const int c = 2 * (k & 3) + hi;
                uint32_t b[4];
                ldsm4(b, base + (k >> 2) * (S::TILE * 128) + ((c ^ (r & 7)) << 4));
                mma16816(s[0], q[k], b[0], b[1]);
                mma16816(s[1], q[k], b[2], b[3]);
            }
        }
        const int t = lane & 3;
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const bool seen = 8 * n + 2 * t + (x & 1) < valid;
                s[n][x] = seen ? s[n][x] * scale : -INFINITY;
                mx[x >> 1] = fmaxf(mx[x >> 1], s[n][x]);
            }
        float f[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
            mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
            const float mn = fmaxf(m[r], mx[r]);
            f[r] = m[r] == mn ? 1.f : exp2f(m[r] - mn);  // (also where both are -inf)
            m[r] = mn;
        }
        if (__any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                o[i][0] *= f[0];
                o[i][1] *= f[0];
                o[i][2] *= f[1];
                o[i][3] *= f[1];
            }
            l[0] *= f[0];
            l[1] *= f[1];
        }
        uint32_t ph[4], pl[4];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float mr = m[r] == -INFINITY ? 0.f : m[r];
                const float p0 = exp2f(s[n][2 * r] - mr), p1 = exp2f(s[n][2 * r + 1] - mr);
                l[r] += p0 + p1;
                const uint32_t h = pack_bf16(p0, p1);
                ph[2 * n + r] = h;
                pl[2 * n + r] = pack_bf16(p0 - bf_lo(h), p1 - bf_hi(h));
            }
        {
            const int r = k0 + (lane & 15);
            const uint32_t base = tc::smem_u32(sV) + r * 128;
            const int hi = lane >> 4;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const int c = 2 * (k & 3) + hi;
                uint32_t b[4];
                ldsm4t(b, base + (k >> 2) * (S::TILE * 128) + ((c ^ (r & 7)) << 4));
                mma16816(o[2 * k], ph, b[0], b[1]);
                mma16816(o[2 * k + 1], ph, b[2], b[3]);
                mma16816(o[2 * k], pl, b[0], b[1]);
                mma16816(o[2 * k + 1], pl, b[2], b[3]);
            }
        }
    }

    __device__ __forceinline__ void finish_sum() {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        }
    }
    __device__ __forceinline__ void put(float *buf, float2 *ml, int lane) const {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x) buf[(4 * i + x) * 32 + lane] = o[i][x];
        if ((lane & 3) == 0) {
            ml[lane >> 2] = make_float2(m[0], l[0]);
            ml[8 + (lane >> 2)] = make_float2(m[1], l[1]);
        }
    }
    __device__ __forceinline__ void join(const float *buf, const float2 *ml, int lane) {
        float fa[2], fb[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float2 b = ml[8 * r + (lane >> 2)];
            const float mn = fmaxf(m[r], b.x), ms = mn == -INFINITY ? 0.f : mn;
            fa[r] = exp2f(m[r] - ms);
            fb[r] = exp2f(b.x - ms);
            l[r] = l[r] * fa[r] + b.y * fb[r];
            m[r] = mn;
        }
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x)
                o[i][x] = o[i][x] * fa[x >> 1] + buf[(4 * i + x) * 32 + lane] * fb[x >> 1];
    }
    __device__ __forceinline__ void write_out(const Args &a, int row, int h0, int nh, int lane) const {
        bf16 *O = (bf16 *)a.o + ((size_t)row * a.Hq + h0) * D;
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            if (g + 8 * r >= nh) continue;
            const float inv = l[r] > 0.f ? 1.f / l[r] : 0.f;
#pragma unroll
            for (int i = 0; i < NT; ++i)
                *(uint32_t *)(O + (size_t)(g + 8 * r) * D + 8 * i + 2 * t) =
                    pack_bf16(o[i][2 * r] * inv, o[i][2 * r + 1] * inv);
        }
    }
    __device__ __forceinline__ void write_part(float *po, float2 *pml, int nh, int lane) const {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            if (g + 8 * r >= nh) continue;
            if (t == 0) pml[g + 8 * r] = make_float2(m[r], l[r]);
#pragma unroll
            for (int i = 0; i < NT; ++i)
                *(float2 *)(po + (size_t)(g + 8 * r) * D + 8 * i + 2 * t) = make_float2(o[i][2 * r], o[i][2 * r + 1]);
        }
    }
};

// fp32 storage: fp32 FMAs.  For the scores a lane owns a key and 32 of the elements (one 128-byte block of its row),
// for the output D/32 elements of every key; q and the probabilities are read as broadcasts from shared memory.
template <int D, int GP>
struct StateF32 {
    using S = Shape<float, D>;
    static constexpr int DPL = D / 32, SL = S::SLICE, PARTS = 32 / SL;
    static_assert(PARTS == S::NB, "one block of a row per lane");
    float o[GP][DPL];
    float m[GP], l[GP];

    static __device__ __forceinline__ float *s_q(uint8_t *merge) { return (float *)merge; }  // [GP][D]
    static __device__ __forceinline__ float *s_p(uint8_t *merge, int warp) {                 // [SL][GP]
        return (float *)(merge + kPagedHeads * D * 4) + warp * (SL * GP);
    }

    __device__ __forceinline__ void begin(const Args &a, int row, int h0, int nh, uint8_t *merge, int lane, int warp) {
        const float *Q = (const float *)a.q + ((size_t)row * a.Hq + h0) * D;
        for (int i = warp * 32 + lane; i < GP * D; i += 128) s_q(merge)[i] = i < nh * D ? Q[i] : 0.f;
        consumer_sync();
#pragma unroll
        for (int h = 0; h < GP; ++h) {
            m[h] = -INFINITY;
            l[h] = 0.f;
#pragma unroll
            for (int j = 0; j < DPL; ++j) o[h][j] = 0.f;
        }
    }

    __device__ __forceinline__ void tile(uint8_t *sK, uint8_t *sV, int k0, int valid, float scale, uint8_t *merge,
                                         int lane, int warp) {
        const int key = lane % SL, part = lane / SL;
        float s[GP] = {};
        {
            const int r = k0 + key;
            const uint8_t *krow = sK + part * (S::TILE * 128) + r * 128;
            const float *q = s_q(merge) + part * 32;
            // (the parts' pieces of q lie 128 bytes apart: each part starts elsewhere, so that they meet no bank twice)
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const int c = (x + part * (8 / PARTS)) & 7;
                const float4 k = *(const float4 *)(krow + ((c ^ (r & 7)) << 4));
#pragma unroll
                for (int h = 0; h < GP; ++h) {
                    const float4 y = *(const float4 *)(q + h * D + 4 * c);
                    s[h] = fmaf(y.x, k.x, s[h]);
                    s[h] = fmaf(y.y, k.y, s[h]);
                    s[h] = fmaf(y.z, k.z, s[h]);
                    s[h] = fmaf(y.w, k.w, s[h]);
                }
            }
        }
        float *sp = s_p(merge, warp);
        // step by step over all heads, whose exchanges then overlap
#pragma unroll
        for (int x = SL; x < 32; x <<= 1)
#pragma unroll
            for (int h = 0; h < GP; ++h) s[h] += __shfl_xor_sync(0xffffffffu, s[h], x);
        float mx[GP];
#pragma unroll
        for (int h = 0; h < GP; ++h) mx[h] = s[h] = key < valid ? s[h] * scale : -INFINITY;
#pragma unroll
        for (int x = 1; x < SL; x <<= 1)
#pragma unroll
            for (int h = 0; h < GP; ++h) mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], x));
#pragma unroll
        for (int h = 0; h < GP; ++h) {
            const float mn = fmaxf(m[h], mx[h]), ms = mn == -INFINITY ? 0.f : mn;
            const float f = tc::ex2_fast(m[h] - ms);
            m[h] = mn;
            s[h] = tc::ex2_fast(s[h] - ms);
            l[h] = l[h] * f + (part == 0 ? s[h] : 0.f);
#pragma unroll
            for (int j = 0; j < DPL; ++j) o[h][j] *= f;
        }
        if (part == 0) {
#pragma unroll
            for (int h = 0; h < GP; ++h) sp[key * GP + h] = s[h];
        }
        __syncwarp();
        const int b = lane * DPL / 32, e = (lane * DPL) % 32;  // this lane's block and element in it
#pragma unroll 4
        for (int k = 0; k < valid; ++k) {
            const int r = k0 + k;
            const uint8_t *v = sV + b * (S::TILE * 128) + r * 128 + (((e >> 2) ^ (r & 7)) << 4) + (e & 3) * 4;
            float x[DPL];
            if constexpr (DPL == 4) {
                const float4 y = *(const float4 *)v;
                x[0] = y.x; x[1] = y.y; x[2] = y.z; x[3] = y.w;
            } else {
                const float2 y = *(const float2 *)v;
                x[0] = y.x; x[1] = y.y;
            }
            float p[GP];
            if constexpr (GP % 4 == 0) {
#pragma unroll
                for (int h = 0; h < GP; h += 4) *(float4 *)(p + h) = *(const float4 *)(sp + k * GP + h);
            } else {
#pragma unroll
                for (int h = 0; h < GP; ++h) p[h] = sp[k * GP + h];
            }
#pragma unroll
            for (int h = 0; h < GP; ++h)
#pragma unroll
                for (int j = 0; j < DPL; ++j) o[h][j] = fmaf(p[h], x[j], o[h][j]);
        }
        __syncwarp();  // the probabilities are overwritten by the next tile
    }

    __device__ __forceinline__ void finish_sum() {
#pragma unroll
        for (int h = 0; h < GP; ++h)
#pragma unroll
            for (int x = 1; x < 32; x <<= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], x);
    }
    __device__ __forceinline__ void put(float *buf, float2 *ml, int lane) const {
#pragma unroll
        for (int h = 0; h < GP; ++h) {
#pragma unroll
            for (int j = 0; j < DPL; ++j) buf[(h * DPL + j) * 32 + lane] = o[h][j];
            if (lane == 0) ml[h] = make_float2(m[h], l[h]);
        }
    }
    __device__ __forceinline__ void join(const float *buf, const float2 *ml, int lane) {
#pragma unroll
        for (int h = 0; h < GP; ++h) {
            const float2 b = ml[h];
            const float mn = fmaxf(m[h], b.x), ms = mn == -INFINITY ? 0.f : mn;
            const float fa = exp2f(m[h] - ms), fb = exp2f(b.x - ms);
            l[h] = l[h] * fa + b.y * fb;
            m[h] = mn;
#pragma unroll
            for (int j = 0; j < DPL; ++j) o[h][j] = o[h][j] * fa + buf[(h * DPL + j) * 32 + lane] * fb;
        }
    }
    __device__ __forceinline__ void write_out(const Args &a, int row, int h0, int nh, int lane) const {
        float *O = (float *)a.o + ((size_t)row * a.Hq + h0) * D;
#pragma unroll
        for (int h = 0; h < GP; ++h) {
            if (h >= nh) break;
            const float inv = l[h] > 0.f ? 1.f / l[h] : 0.f;
#pragma unroll
            for (int j = 0; j < DPL; ++j) O[h * D + lane * DPL + j] = o[h][j] * inv;
        }
    }
    __device__ __forceinline__ void write_part(float *po, float2 *pml, int nh, int lane) const {
#pragma unroll
        for (int h = 0; h < GP; ++h) {
            if (h >= nh) break;
            if (lane == 0) pml[h] = make_float2(m[h], l[h]);
#pragma unroll
            for (int j = 0; j < DPL; ++j) po[h * D + lane * DPL + j] = o[h][j];
        }
    }
};

// A run of the work list, walked segment by segment ((row, kv head, head chunk)).
struct Walk {
    int row, sub, tiles, tile;  // row, (kv head, chunk) within it, its key tiles, next tile
    __device__ __forceinline__ void skip_empty(const Args &a, int tile_keys) {
        while (tiles == 0 && row + 1 < a.n) {
            ++row;
            tiles = (row_len(a, row) + tile_keys - 1) / tile_keys;
        }
    }
    // one tile on; true where that began another segment
    __device__ __forceinline__ bool next(const Args &a, int tile_keys) {
        if (++tile < tiles) return false;
        tile = 0;
        if (++sub == a.Hkv * a.HC) {
            sub = 0;
            tiles = 0;
            skip_empty(a, tile_keys);
        }
        return true;
    }
};

template <typename T, int D, typename State>
__global__ void __launch_bounds__(kThreads, 2) k_paged_attend(const __grid_constant__ Maps maps, const Args a) {
    using S = Shape<T, D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    Small &sm = *(Small *)(smem + S::RING + S::MERGE);
    if (threadIdx.x == kThreads - 32) {
        tc::prefetch_map(&maps.k);
        tc::prefetch_map(&maps.v);
    }
    tc::grid_dep_wait();
    tc::grid_dep_launch();  // (after the wait: the join reads the lengths before it waits for this kernel)
    if (tc::smem_u32(smem) & 1023) {
        if (threadIdx.x == 0) record_error(a.counters, kDevErrSmemAlign);
        return;
    }
    uint8_t *merge = smem + S::RING;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int HH = a.Hkv * a.HC;

    // this CTA's run [u0, u1) of the tile list, and where it starts
    const int per = (a.n + kThreads - 1) / kThreads;
    const int r0 = min(a.n, (int)threadIdx.x * per), r1 = min(a.n, r0 + per);
    int mine = 0;
    for (int r = r0; r < r1; ++r) {
        const int len = a.lens[r];
        if (blockIdx.x == 0 && (len < 0 || len > a.width * a.page)) record_error(a.counters, kDevErrBadLen);
        mine += (row_len(a, r) + S::TILE - 1) / S::TILE;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::STAGES; ++i) {
            tc::mbar_init(&sm.full[i], 1);
            tc::mbar_init(&sm.empty[i], 4);
        }
        tc::fence_mbar_init();
    }
    int tiles_all;
    int pre = block_scan<kThreads>(mine, sm.scan, &tiles_all);
    const long long total = (long long)tiles_all * HH;
    const int ctas = (int)min(total, (long long)gridDim.x);  // of a tile at least each
    const bool idle = (int)blockIdx.x >= ctas;
    const long long u0 = idle ? 0 : total * blockIdx.x / ctas, u1 = idle ? 0 : total * (blockIdx.x + 1) / ctas;
    for (int r = r0; r < r1; ++r) {
        const int t = (row_len(a, r) + S::TILE - 1) / S::TILE;
        if (blockIdx.x == 0) a.prefix[r] = pre;
        if (u0 < u1 && t > 0 && u0 >= (long long)pre * HH && u0 < (long long)(pre + t) * HH) {
            sm.start[0] = r;
            sm.start[1] = pre;
            sm.start[2] = t;
        }
        pre += t;
    }
    if (blockIdx.x == 0 && threadIdx.x == kThreads - 1) a.prefix[a.n] = tiles_all;
    __syncthreads();
    if (u0 >= u1) return;
    Walk w;
    {
        const long long in_row = u0 - (long long)sm.start[1] * HH;
        w.row = sm.start[0];
        w.tiles = sm.start[2];
        w.sub = (int)(in_row / w.tiles);
        w.tile = (int)(in_row % w.tiles);
    }
    const int count = (int)(u1 - u0);
    bool ok = true;

    if (warp == 4) {
        // ---------------- producer ----------------
        // lane l brings page l of the tile; its id is read one tile ahead
        const int box = min(a.page, S::TILE), np = S::TILE / box;
        auto lookup = [&](const Walk &x) {
            int id = -1;
            const int key = x.tile * S::TILE + lane * box;
            if (lane < np && key < row_len(a, x.row)) {
                id = a.table[(size_t)x.row * a.width + key / a.page];
                if ((unsigned)id >= (unsigned)a.pages) {
                    record_error(a.counters, kDevErrBadPage);
                    id = -1;
                }
            }
            return id;
        };
        int id = lookup(w);
        int last[S::STAGES];
#pragma unroll
        for (int s = 0; s < S::STAGES; ++s) last[s] = -1;
        for (int i = 0; i < count; ++i) {
            const int s = i % S::STAGES, v = i / S::STAGES;
            const Walk cur = w;
            w.next(a, S::TILE);
            const int id_next = i + 1 < count ? lookup(w) : -1;
            if (v > 0 && !__all_sync(0xffffffffu, tc::mbar_wait(&sm.empty[s], (v - 1) & 1))) {
                ok = false;
                break;
            }
            const unsigned mask = __ballot_sync(0xffffffffu, id >= 0);
            if (lane == 0) {
                sm.mask[s] = (int)mask;
                if (mask) tc::mbar_expect_tx(&sm.full[s], __popc(mask) * box * D * S::ES * 2);
                else tc::mbar_arrive(&sm.full[s]);
            }
            __syncwarp();
            if (id >= 0) {
                uint8_t *sK = smem + s * (2 * S::KB);
                const int y = (id * a.Hkv + cur.sub / a.HC) * a.page + (cur.tile * S::TILE + lane * box) % a.page;
#pragma unroll
                for (int b = 0; b < S::NB; ++b) {
                    uint8_t *at = sK + b * (S::TILE * 128) + lane * box * 128;
                    tc::tma_load_2d(at, &maps.k, b * S::EB, y, &sm.full[s]);
                    tc::tma_load_2d(at + S::KB, &maps.v, b * S::EB, y, &sm.full[s]);
                }
            }
#pragma unroll
            for (int x = 0; x < S::STAGES; ++x)
                if (x == s) last[x] = v;
            id = id_next;
        }
        // every copy issued has landed before the CTA may exit
#pragma unroll
        for (int s = 0; s < S::STAGES; ++s)
            if (last[s] >= 0 && !tc::mbar_wait(&sm.full[s], last[s] & 1)) ok = false;
    } else {
        // ---------------- consumers ----------------
        State st;
        const int k0 = warp * S::SL;
        const int box = min(a.page, S::TILE);
        int i = 0;
        bool first_seg = true;
        while (i < count) {
            const Walk seg = w;
            const int kv = seg.sub / a.HC, h0 = kv * a.G + (seg.sub % a.HC) * kPagedHeads;
            const int nh = min(kPagedHeads, a.G - (seg.sub % a.HC) * kPagedHeads);
            const int len = row_len(a, seg.row);
            const bool whole = seg.tile == 0 && count - i >= seg.tiles;
            st.begin(a, seg.row, h0, nh, merge, lane, warp);
            bool another = false;
            while (i < count && !another) {
                const int s = i % S::STAGES, v = i / S::STAGES;
                if (ok && !__all_sync(0xffffffffu, tc::mbar_wait(&sm.full[s], v & 1))) ok = false;
                uint8_t *sK = smem + s * (2 * S::KB), *sV = sK + S::KB;
#pragma unroll 1
                for (int k = k0; k < k0 + S::SL; k += S::SLICE) {
                    int valid = min(S::SLICE, len - w.tile * S::TILE - k);
                    if (!((sm.mask[s] >> (k / box)) & 1)) valid = 0;
                    if (ok && valid > 0) st.tile(sK, sV, k, valid, a.scale_log2, merge, lane, warp);
                }
                tc::fence_smem_to_async();  // zeroed rows before the next copy into this stage
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&sm.empty[s]);
                ++i;
                another = w.next(a, S::TILE);
            }
            // join the four warps' states: 1 into 0 and 3 into 2, then 2 into 0
            st.finish_sum();
            consumer_sync();  // (fp32: every warp is done with q)
            float *buf = (float *)merge + (warp >> 1) * (kPagedHeads * D);
            if (warp & 1) st.put(buf, sm.ml[warp >> 1], lane);
            consumer_sync();
            if (!(warp & 1)) st.join(buf, sm.ml[warp >> 1], lane);
            consumer_sync();
            if (warp == 2) st.put((float *)merge, sm.ml[0], lane);
            consumer_sync();
            if (warp == 0) {
                st.join((float *)merge, sm.ml[0], lane);
                if (whole) {
                    st.write_out(a, seg.row, h0, nh, lane);
                } else {
                    const int slot = 2 * blockIdx.x + (first_seg ? 0 : 1);
                    st.write_part(a.part_o + (size_t)slot * kPagedHeads * D, a.part_ml + (size_t)slot * kPagedHeads, nh,
                                  lane);
                }
            }
            consumer_sync();
            first_seg = false;
        }
    }
    if (!ok && lane == 0) record_error(a.counters, kDevErrTimeout);
}

// ---------------------------------------------------------------------------
// join of the parts: one block per (row, head); the runs' borders follow from the tile counts alone
// ---------------------------------------------------------------------------
constexpr int kJoinRows = 1024;  // up to so many rows a block counts the tiles before its own itself

template <typename T, int D>
__global__ void __launch_bounds__(128) k_paged_join(const Args a, int grid) {
    constexpr int DPL = D / 32, TILE = Shape<T, D>::TILE;
    __shared__ float s_o[4][D];
    __shared__ float s_l[4], s_m[4];
    __shared__ int s_n[4][2];
    const int row = blockIdx.x / a.Hq, h = blockIdx.x % a.Hq;
    const int kv = h / a.G, hc = (h % a.G) / kPagedHeads, hh = (h % a.G) % kPagedHeads;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    T *O = (T *)a.o + ((size_t)row * a.Hq + h) * D;
    const int HH = a.Hkv * a.HC;
    int pre, tiles, all;
    if (a.n <= kJoinRows) {  // from the lengths, while the attention still runs
        int before = 0, sum = 0;
        for (int r = threadIdx.x; r < a.n; r += 128) {
            const int t = (row_len(a, r) + TILE - 1) / TILE;
            sum += t;
            before += r < row ? t : 0;
        }
        before = __reduce_add_sync(0xffffffffu, before);
        sum = __reduce_add_sync(0xffffffffu, sum);
        if (lane == 0) {
            s_n[warp][0] = before;
            s_n[warp][1] = sum;
        }
        __syncthreads();
        pre = s_n[0][0] + s_n[1][0] + s_n[2][0] + s_n[3][0];
        all = s_n[0][1] + s_n[1][1] + s_n[2][1] + s_n[3][1];
        tiles = (row_len(a, row) + TILE - 1) / TILE;
        tc::grid_dep_wait();
    } else {
        tc::grid_dep_wait();
        pre = a.prefix[row];
        tiles = a.prefix[row + 1] - pre;
        all = a.prefix[a.n];
    }
    if (tiles <= 0) {  // an empty row
        for (int i = threadIdx.x; i < D; i += 128) O[i] = from_f<T>(0.f);
        return;
    }
    const long long total = (long long)all * HH;
    if (total <= 0) return;
    const int ctas = (int)min(total, (long long)grid);
    const long long u0 = (long long)pre * HH + (long long)(kv * a.HC + hc) * tiles, u1 = u0 + tiles;
    // the CTA of unit u is the last c with floor(c total / ctas) <= u
    const int c0 = (int)(((u0 + 1) * ctas - 1) / total), c1 = (int)((u1 * ctas - 1) / total);
    if (c0 == c1 || c0 < 0 || c1 >= ctas) return;  // one CTA had it whole and wrote the result
    const int first_slot = total * c0 / ctas == u0 ? 0 : 1;
    auto slot_of = [&](int c) { return 2 * c + (c == c0 ? first_slot : 0); };
    float m = -INFINITY, l = 0.f, o[DPL] = {};
    for (int b = c0 + warp; b <= c1; b += 4 * 32) {  // lane by lane the statistics of 32 parts, then their outputs
        const int c = b + 4 * lane;
        const float2 ml = c <= c1 ? a.part_ml[(size_t)slot_of(c) * kPagedHeads + hh] : make_float2(-INFINITY, 0.f);
        float mx = ml.x;
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
        const float mn = fmaxf(m, mx), ms = mn == -INFINITY ? 0.f : mn;
        const float f = exp2f(m - ms);
        m = mn;
        const float wgt = exp2f(ml.x - ms);
        float ls = ml.y * wgt;
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) ls += __shfl_xor_sync(0xffffffffu, ls, x);
        l = l * f + ls;
#pragma unroll
        for (int j = 0; j < DPL; ++j) o[j] *= f;
        const int nb = min(32, (c1 - b) / 4 + 1);
#pragma unroll 4
        for (int k = 0; k < nb; ++k) {
            const float wk = __shfl_sync(0xffffffffu, wgt, k);
            const float *po = a.part_o + ((size_t)slot_of(b + 4 * k) * kPagedHeads + hh) * D + lane * DPL;
#pragma unroll
            for (int j = 0; j < DPL; ++j) o[j] = fmaf(wk, po[j], o[j]);
        }
    }
    if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = l;
    }
#pragma unroll
    for (int j = 0; j < DPL; ++j) s_o[warp][lane * DPL + j] = o[j];
    __syncthreads();
    const float mm = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3])), ms = mm == -INFINITY ? 0.f : mm;
    float f[4], den = 0.f;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        f[x] = exp2f(s_m[x] - ms);
        den += s_l[x] * f[x];
    }
    const float inv = den > 0.f ? 1.f / den : 0.f;
    for (int i = threadIdx.x; i < D; i += 128) {
        float v = 0.f;
#pragma unroll
        for (int x = 0; x < 4; ++x) v = fmaf(s_o[x][i], f[x], v);
        O[i] = from_f<T>(v * inv);
    }
}

// the pool of a layer as [pages*Hkv*page, d], boxes of one 128-byte block x a page's (or tile's) rows
template <typename T>
bool pool_map(CUtensorMap *map, const void *ptr, int d, long long rows, int box_rows) {
    auto enc = (PFN_cuTensorMapEncodeTiled_v12000)tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)d * sizeof(T)};
    cuuint32_t box[2] = {(cuuint32_t)(128 / sizeof(T)), (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    return enc(map, sizeof(T) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2,
               const_cast<void *>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D, typename State>
cudaError_t launch_shape(const PagedPlan &p, const void *Kp, const void *Vp, const Args &a, cudaStream_t s) {
    using S = Shape<T, D>;
    Maps maps;
    const long long rows = (long long)a.pages * a.Hkv * a.page;
    const int box = std::min(a.page, S::TILE);
    if (!pool_map<T>(&maps.k, Kp, D, rows, box) || !pool_map<T>(&maps.v, Vp, D, rows, box)) return cudaErrorInvalidValue;
    cudaError_t e;
    int dev = 0, sms = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    auto kern = k_paged_attend<T, D, State>;
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::BYTES)) != cudaSuccess) return e;
    const int ctas = std::min(2 * sms, kPagedMaxCtas);
    if ((e = launch_after(kern, dim3(ctas), dim3(kThreads), S::BYTES, s, maps, a)) != cudaSuccess) return e;
    if ((e = launch_after(k_paged_join<T, D>, dim3((unsigned)a.n * a.Hq), dim3(128), 0, s, a, ctas)) != cudaSuccess)
        return e;
    count_launches(2);
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_paged_attend(const PagedPlan &p, int layer, int n, const void *Q, const int32_t *table,
                                const int32_t *lens, const void *Kp, const void *Vp, void *O, void *ws,
                                cudaStream_t s) {
    const mono_paged_config &c = p.cfg;
    const size_t off = (size_t)layer * c.pages * c.Hkv * c.page * c.d * p.es;
    const void *K = (const char *)Kp + off, *V = (const char *)Vp + off;
    Args a;
    a.q = Q;
    a.table = table;
    a.lens = lens;
    a.o = O;
    a.part_o = (float *)pg_ptr(p, ws, kPgPartO);
    a.part_ml = (float2 *)pg_ptr(p, ws, kPgPartML);
    a.prefix = (int32_t *)pg_ptr(p, ws, kPgPrefix);
    a.counters = (unsigned long long *)pg_ptr(p, ws, kPgCounters);
    a.n = n;
    a.Hq = c.Hq;
    a.Hkv = c.Hkv;
    a.G = c.Hq / c.Hkv;
    a.HC = (a.G + kPagedHeads - 1) / kPagedHeads;
    a.width = c.width;
    a.page = c.page;
    a.pages = c.pages;
    a.scale_log2 = p.scale_log2;
    if (c.dtype == MONO_BF16) {
        if (c.d == 64) return launch_shape<bf16, 64, StateBf16<64>>(p, K, V, a, s);
        return launch_shape<bf16, 128, StateBf16<128>>(p, K, V, a, s);
    }
    // fp32: registers for 1, 4 or 16 query heads (six rows of up to 4,099 tokens with one head each: 12.0 us, by the
    // code for four 13.2)
    if (c.d == 64) {
        if (a.G == 1) return launch_shape<float, 64, StateF32<64, 1>>(p, K, V, a, s);
        if (a.G <= 4) return launch_shape<float, 64, StateF32<64, 4>>(p, K, V, a, s);
        return launch_shape<float, 64, StateF32<64, 16>>(p, K, V, a, s);
    }
    if (a.G == 1) return launch_shape<float, 128, StateF32<128, 1>>(p, K, V, a, s);
    if (a.G <= 4) return launch_shape<float, 128, StateF32<128, 4>>(p, K, V, a, s);
    return launch_shape<float, 128, StateF32<128, 16>>(p, K, V, a, s);
}

}  // namespace mono
