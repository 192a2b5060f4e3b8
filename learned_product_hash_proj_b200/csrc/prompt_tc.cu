// prompt_tc.cu -- causal attention over packed prompts on the tensor cores
// (bf16 storage).
//
//   o_i = sum_{j <= i + lk - lq} softmax_j(scale <q_i, k_j>) v_j   per sequence and query head
//
// One CTA per 256 rows: two groups of 128 that share every K and V tile of 128
// keys.  The rows of a tile are 256/pack consecutive queries of a sequence for
// each of `pack` query heads that read the same key/value head (1, 2, 4, 8 or
// 16, whichever power of two divides the group): short sequences then fill the
// tiles (64 sequences of 300 tokens, 32 heads over 8: 187 us with a head per
// tile where four took 140).  A TMA warp streams K and V tiles through a ring of
// shared-memory stages; one thread issues the MMAs, S_g = Q_g K^T into tensor
// memory and O_g += P_g V with P_g read from tensor memory, alternating the
// groups; four warps per group, a thread per row, turn S into P in place.  So
// while one group's softmax runs, the tensor cores work for the other.  CTAs
// are persistent, one per SM, over a list of the call's query tiles, and the
// ring runs on from tile to tile; where one group needs a key tile more than the
// other, the other's next query tile begins meanwhile (16,384 tokens in two
// sequences, 16 heads of 64: 380 and 343 us).  Output goes through shared memory
// and from there by TMA while the next tile is worked on.
//
// The softmax keeps a reference maximum per row.  P is exp2(s - ref), and ref
// is only raised (and O and the sum rescaled by the row's own thread) when
// the running maximum has outgrown it by more than 2^8: any reference gives
// the same quotient O / sum, P stays below 2^8, and fp32 and bf16 have the
// range, so most tiles never touch O.  P is rounded to bf16 (the tensor cores
// take it in V's type; two terms would double the second product), the sum is that
// of the values before rounding: the result's relative error (2-norm, 16,384
// tokens) is 2.2e-3, of which its own rounding to bf16 makes 1.6e-3.
//
// Measured on one B200, in bursts of 3 ms after a pause, and at the power limit
// (sampled clocks of 1.51 to 1.7 GHz): 16,384 tokens, 16 heads of 128 over 4:
// 857 and 975 us, 1,283 and 1,128 TFLOP/s (76 and 67 % of the measured burst rate);
// 4,096 tokens 67 and 72 us, 16 x 1,024 87 and 98 us, 64 x 300 (32 heads over 8)
// 120 and 138 us; two sequences of 8,192, 16 heads of 64: 364 and 386 us.  What
// bounds it: a group's chain of softmax (about 1,650 cycles for 128 x 128 scores,
// 640 of them special-function exponentials) and its two products (1,024) takes
// 3,000 cycles, in which the tensor cores have 2,048 to do for both groups (half of
// it for heads of 64, with the same softmax); where query tiles have few key tiles,
// also the way from one to the next (about 3,000 cycles: the last product, the
// output, the first scores).  Tried and slower: two threads per row (16 softmax
// warps, 1,091 us where this takes 990), the maximum taken beside the
// exponentials with the reference a tile late (1,035), an MMA warp per group
// (844 and 829), P handed over in two parts (no gain).  (Figures of the tries are
// of the builds that they were compared in.)
#include <cooperative_groups.h>
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <type_traits>

#include "paged.cuh"

namespace cg = cooperative_groups;

namespace mono {

namespace {

using bf16 = __nv_bfloat16;

constexpr int kKeys = 128;      // keys per tile
constexpr int kThreads = 384;   // 2 groups of 4 softmax warps, the TMA, gate and MMA warps, one idle
// registers per thread: launched with 168 (64,512 of an SM's 65,536); the 8 softmax warps, which hold a row of 128
// scores per thread, draw on what the other four give back: 256 x 216 + 128 x 72 = 64,512
constexpr int kRegsSoftmax = 216, kRegsOther = 72;
constexpr float kGrow = 8.f;    // log2 of how far the maximum may outgrow the reference
// The exponents s scale - ref scale are one FMA each, with ref scale rounded beforehand.  Up to this size of it the
// rounding shifts a row's exponents together by at most 1, which the quotient does not see; beyond, as with a scale for
// hard attention, it could pass fp32's range, and ref is subtracted from the scores first, which is exact enough at any
// size.  (With the branch, and a maximum that keeps NaN, long calls take 0.4 to 1 % more, short ones and split keys up
// to 3 %: 16 x 1,024 tokens 96.2 and 98.6 us, 256 queries after 32,512 tokens 120.8 and 124.8.)
constexpr float kFar = 16777216.f;

template <int D>
struct Lay {
    static constexpr int QB = 128 * D * 2;          // bytes of a group's Q: [D/64][128 rows][128]
    static constexpr int TB = kKeys * D * 2;        // bytes of a K or V tile, the same layout
    static constexpr int NST = D == 128 ? 4 : 8;    // ring stages
    static constexpr int OUT = 2 * QB + NST * TB;   // 32 rows x 128 bytes per softmax warp, on the way out
    static constexpr int BAR = OUT + 8 * 32 * 128;
    static constexpr int BYTES = BAR + 512;
    static constexpr int O_COL = 256;               // tensor memory: S_0, S_1 (128 columns each), then O_0, O_1
};

// An item's first key tile lands on a barrier of its own, `first` in turn, not on its ring slot's `full`.  Only the MMA
// warp waits for it; the gate warp, which waits for all other tiles, would have to pass it either before it has landed
// (later tiles may land first) or after its slot has been used up and filled again, and take another phase's parity
// for the one that it waits for.  Eight: more first tiles than the ring can hold.
constexpr int kFirst = 8;
struct Bars {
    uint64_t q_full[2], q_empty[2], full[8], empty[8], first[kFirst], s_full[2], p_full[2], o_done[2], drain;
    uint32_t tmem;
    int abort;
    int scan[kThreads / 32 + 1], out[2];
};
static_assert(sizeof(Bars) <= 512, "behind the ring");

// A query tile: queries q .. q+rows-1, the sequence's keys from row k on; query r of the tile sees the keys up to
// min(keys, last + r + 1) - 1.
struct alignas(16) Tile {
    int q, rows, k, keys, last, pad[3];
    // key tiles that group g (queries g*half .. g*half + half - 1) needs
    __device__ __forceinline__ int tiles(int g, int half) const {
        const int n = min(rows, half * (g + 1));  // past the group's last query
        return half * g < rows ? max(0, min(keys, last + n) + kKeys - 1) / kKeys : 0;
    }
};
static_assert(sizeof(Tile) == 32, "two 16-byte loads");

__device__ __forceinline__ Tile make_tile(const int32_t *cu_q, const int32_t *cu_k, int seq, int row0, int qt,
                                          int total_q, int total_k, unsigned long long *counters) {
    const Span q = cu_span(cu_q, seq, total_q, counters), k = cu_span(cu_k, seq, total_k, counters);
    const int rows = row0 >= 0 ? max(0, min(qt, q.n - row0)) : 0;  // (row0 is inside wherever the lengths ascend)
    return {q.at + row0, rows, k.at, k.n, row0 + k.n - q.n, {}};
}

struct Maps {
    CUtensorMap q, k, v, o;
};

// tensor memory -> registers, 32 lanes x 128 columns, waited for
__device__ __forceinline__ void tmem_ld128(uint32_t taddr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x128.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
        "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
        "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63, "
        "%64, %65, %66, %67, %68, %69, %70, %71, %72, %73, %74, %75, %76, %77, %78, %79, "
        "%80, %81, %82, %83, %84, %85, %86, %87, %88, %89, %90, %91, %92, %93, %94, %95, "
        "%96, %97, %98, %99, %100, %101, %102, %103, %104, %105, %106, %107, %108, %109, %110, %111, "
        "%112, %113, %114, %115, %116, %117, %118, %119, %120, %121, %122, %123, %124, %125, %126, %127}, [%128];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
          "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
          "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
          "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
          "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63]),
          "=r"(r[64]), "=r"(r[65]), "=r"(r[66]), "=r"(r[67]), "=r"(r[68]), "=r"(r[69]), "=r"(r[70]), "=r"(r[71]),
          "=r"(r[72]), "=r"(r[73]), "=r"(r[74]), "=r"(r[75]), "=r"(r[76]), "=r"(r[77]), "=r"(r[78]), "=r"(r[79]),
          "=r"(r[80]), "=r"(r[81]), "=r"(r[82]), "=r"(r[83]), "=r"(r[84]), "=r"(r[85]), "=r"(r[86]), "=r"(r[87]),
          "=r"(r[88]), "=r"(r[89]), "=r"(r[90]), "=r"(r[91]), "=r"(r[92]), "=r"(r[93]), "=r"(r[94]), "=r"(r[95]),
          "=r"(r[96]), "=r"(r[97]), "=r"(r[98]), "=r"(r[99]), "=r"(r[100]), "=r"(r[101]), "=r"(r[102]), "=r"(r[103]),
          "=r"(r[104]), "=r"(r[105]), "=r"(r[106]), "=r"(r[107]), "=r"(r[108]), "=r"(r[109]), "=r"(r[110]), "=r"(r[111]),
          "=r"(r[112]), "=r"(r[113]), "=r"(r[114]), "=r"(r[115]), "=r"(r[116]), "=r"(r[117]), "=r"(r[118]), "=r"(r[119]),
          "=r"(r[120]), "=r"(r[121]), "=r"(r[122]), "=r"(r[123]), "=r"(r[124]), "=r"(r[125]), "=r"(r[126]), "=r"(r[127])
        : "r"(taddr)
        : "memory");
}
// 32 lanes x 16 columns, waited for
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
// true in one lane of the (converged) warp
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t"
        ".reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "}\n"
        : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// the largest of three, NaN if one of them is
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ tc::f2_t f2_add(tc::f2_t a, tc::f2_t b) {
    tc::f2_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// 2^x of two values on the FMA units, for x <= 127: x = n + r with n whole and |r| <= 1/2 (adding 1.5 * 2^23 leaves
// n in the low bits), 2^r by the cubic of least relative error on [-1/2, 1/2] (7.5e-5, a twentieth of the bf16
// rounding that P gets next), and n added to the exponent.  Below 2^-126 what is left of the bits is a denormal less
// than 2^-126; x is cut off a little above -127 (-inf, a masked key, among it), where the cubic gives just over 1 and
// the bits come to less than 2^-139, an exact zero in bf16.
constexpr float kLeast = -126.99985f;
__device__ __forceinline__ void exp2_pair(tc::f2_t x, float &a, float &b) {
    float lo, hi;
    tc::f2_split(x, lo, hi);
    x = tc::f2_pack(fmaxf(lo, kLeast), fmaxf(hi, kLeast));
    const tc::f2_t t = f2_add(x, tc::f2_dup(12582912.f));
    const tc::f2_t r = f2_add(x, tc::f2_fma(t, tc::f2_dup(-1.f), tc::f2_dup(12582912.f)));
    tc::f2_t p = tc::f2_fma(r, tc::f2_dup(0.0551716685f), tc::f2_dup(0.242611125f));
    p = tc::f2_fma(p, r, tc::f2_dup(0.693260968f));
    p = tc::f2_fma(p, r, tc::f2_dup(0.999928057f));
    float p0, p1, t0, t1;
    tc::f2_split(p, p0, p1);
    tc::f2_split(t, t0, t1);
    a = __int_as_float(__float_as_int(p0) + (__float_as_int(t0) << 23));
    b = __int_as_float(__float_as_int(p1) + (__float_as_int(t1) << 23));
}

// A row's scores into probabilities 2^(s scale - off), kept in s, and as bf16 over the scores in tensor memory.
// The special-function units make 4 exponentials a cycle and quarter SM, a tile's matrix products leave time for
// about as many as it has: with POLY, kPoly of 16 pairs go to the FMA units instead.  (Not where the other group has
// no rows, and these exponentials the units to themselves: 100 sequences of 100 tokens, 16 heads of 128 over 4, 35.4 us,
// with POLY 36.3.)
constexpr int kPoly = 6;
// With SHORT, 32 columns from `seen` on, which no row of the warp sees, are zeros without exponentials.
template <bool POLY, bool SHORT>
__device__ __forceinline__ void to_p(float (&s)[128], float scale, float off, uint32_t tS, int seen) {
    const tc::f2_t sc = tc::f2_dup(scale), no = tc::f2_dup(-off);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        uint32_t pk[16];
        if (SHORT && 32 * c >= seen) {
#pragma unroll
            for (int x = 0; x < 16; ++x) s[32 * c + 2 * x] = s[32 * c + 2 * x + 1] = 0.f, pk[x] = 0;
            tc::tmem_st16(tS + 16 * c, pk);
            continue;
        }
#pragma unroll
        for (int x = 0; x < 16; ++x) {
            float &a = s[32 * c + 2 * x], &b = s[32 * c + 2 * x + 1];
            const tc::f2_t e = tc::f2_fma(tc::f2_pack(a, b), sc, no);
            if (POLY && x * kPoly / 16 != (x + 1) * kPoly / 16) {
                exp2_pair(e, a, b);
            } else {
                tc::f2_split(e, a, b);
                a = tc::ex2_fast(a);
                b = tc::ex2_fast(b);
            }
            pk[x] = pack_bf16(a, b);
        }
        tc::tmem_st16(tS + 16 * c, pk);
    }
}

// ---------------------------------------------------------------------------
// the query tiles of all sequences, those with the most keys first.  One block.
// ---------------------------------------------------------------------------
constexpr int kBins = 256;
__device__ __forceinline__ int bin_of(const Tile &t, int qt) {  // 0: the longest
    const int n = max(t.tiles(0, qt / 2), t.tiles(1, qt / 2));
    return kBins - 1 - (n < 128 ? n : min(kBins - 1, 128 + (n - 128) / 16));
}

__global__ void __launch_bounds__(1024) k_prompt_list(const int32_t *cu_q, const int32_t *cu_k,
                                                      int n, int total_q, int total_k, int qt, int *prefix, Tile *list,
                                                      int *count, int most, unsigned long long *counters) {
    __shared__ int s_w[33], s_bin[kBins];
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    const int per = (n + 1023) / 1024, s0 = min(n, (int)threadIdx.x * per), s1 = min(n, s0 + per);
    auto tiles_of = [&](int s) { return (cu_span(cu_q, s, total_q, counters).n + qt - 1) / qt; };
    int mine = 0;
    for (int s = s0; s < s1; ++s) mine += tiles_of(s);
    int all;
    int pre = block_scan<1024>(mine, s_w, &all);
    for (int s = s0; s < s1; ++s) {
        prefix[s] = pre;
        pre += tiles_of(s);
    }
    if (threadIdx.x < kBins) s_bin[threadIdx.x] = 0;
    all = min(all, most);  // (cumulative lengths that do not ascend could ask for more)
    __syncthreads();
    auto tile_at = [&](int t) {
        int lo = 0, hi = n;  // the last sequence that starts at or before tile t
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (prefix[mid] <= t) lo = mid;
            else hi = mid;
        }
        return make_tile(cu_q, cu_k, lo, (t - prefix[lo]) * qt, qt, total_q, total_k, counters);
    };
    for (int t = threadIdx.x; t < all; t += 1024) atomicAdd(&s_bin[bin_of(tile_at(t), qt)], 1);
    __syncthreads();
    int total;
    const int before = block_scan<1024>(threadIdx.x < kBins ? s_bin[threadIdx.x] : 0, s_w, &total);
    __syncthreads();
    if (threadIdx.x < kBins) s_bin[threadIdx.x] = before;
    __syncthreads();
    for (int t = threadIdx.x; t < all; t += 1024) {
        const Tile x = tile_at(t);
        list[atomicAdd(&s_bin[bin_of(x, qt)], 1)] = x;  // the order within a bin does not show in any result
    }
    if (threadIdx.x == 0) *count = all;
}

// ---------------------------------------------------------------------------
// attention: persistent, one CTA per SM.  Without a list (few tiles) each CTA finds its one tile itself.  kSplit (and
// no list): the CTAs of a cluster share a tile, CTA r of R its key tiles r, r + R, ..., and join their outputs,
// maxima and sums through one another's shared memory.  kPair (short sequences): a tile is one group's 128 rows, and
// the two groups of a CTA work on two tiles, with key tiles of their own in one ring.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

enum PromptMode { kShared, kSplit, kPair };
template <int D, int MODE>
__global__ void __launch_bounds__(kThreads, 1) k_prompt_tc(const __grid_constant__ Maps maps,
                                                           const int32_t *cu_q,
                                                           const int32_t *cu_k, bf16 *__restrict__ O,
                                                           const Tile *list, const int *count, int n, int total_q,
                                                           int total_k, int Hq, int G, int pack, float scale_log2,
                                                           float grow_at,  // kGrow / scale_log2
                                                           unsigned long long *__restrict__ counters) {
    using L = Lay<D>;
    constexpr bool SPLIT = MODE == kSplit, PAIR = MODE == kPair;
    extern __shared__ __align__(1024) uint8_t smem[];
    Bars &b = *(Bars *)(smem + L::BAR);
    if (tc::smem_u32(smem) & 1023) {
        if (threadIdx.x == 0) record_error(counters, kDevErrSmemAlign);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == 8 && lane < 4)
        tc::prefetch_map(lane == 0 ? &maps.q : lane == 1 ? &maps.k : lane == 2 ? &maps.v : &maps.o);
    const int half = 128 >> pack;               // queries of a group; `pack` is the heads' log2
    const int qt = PAIR ? half : 2 * half;      // and of a tile
    const int chunks = Hq >> pack;              // of 2^pack heads: an item is a tile and one of them; PAIR: two such
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = SPLIT ? (int)cluster.block_rank() : 0, ranks = SPLIT ? (int)cluster.num_blocks() : 1;
    const int block = blockIdx.x / ranks;
    int seq = 0, row0 = 0;
    if (!list) tc::grid_dep_wait();
    if (!list && !find_tile<kThreads>(cu_q, n, total_q, qt, block / chunks, b.scan, b.out, &seq, &row0, counters))
        return;

    if (threadIdx.x == 0) {
        for (int s = 0; s < L::NST; ++s) {
            tc::mbar_init(&b.full[s], 1);
            tc::mbar_init(&b.empty[s], 1);
        }
        for (int i = 0; i < kFirst; ++i) tc::mbar_init(&b.first[i], 1);
        for (int g = 0; g < 2; ++g) {
            tc::mbar_init(&b.q_full[g], 1);
            tc::mbar_init(&b.q_empty[g], 1);
            tc::mbar_init(&b.s_full[g], 1);
            tc::mbar_init(&b.p_full[g], 5);
            tc::mbar_init(&b.o_done[g], 1);
        }
        tc::mbar_init(&b.drain, 1);
        b.abort = 0;
        tc::fence_mbar_init();
    }
    if (warp == 9) {
        tc::tmem_alloc(&b.tmem, 512);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = b.tmem;
    tc::grid_dep_wait();  // the list
    const int units = list ? *(volatile const int *)count * chunks : (int)gridDim.x / ranks;
    const int items = PAIR ? (units + 1) / 2 : units;
    // this CTA's j-th item (for group g): there and back over the list, so that no CTA always gets the longer ones
    auto item_at = [&](int j, int g, Tile *t, int *h) {
        int x = list ? j * gridDim.x + ((j & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x) : (j ? items : block);
        if (x >= items) return false;
        if (PAIR) {
            x = 2 * x + g;
            if (x >= units) {  // the last item's second group
                *t = {0, 0, 0, 0, -1, {}};
                *h = 0;
                return true;
            }
        }
        *h = x % chunks;
        if (list) {
            const int4 *p = (const int4 *)(list + x / chunks);
            ((int4 *)t)[0] = p[0];
            ((int4 *)t)[1] = p[1];
        } else {
            *t = make_tile(cu_q, cu_k, seq, row0, qt, total_q, total_k, counters);
        }
        return true;
    };
    volatile int *abort_flag = &b.abort;
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (!__all_sync(0xffffffffu, tc::mbar_wait_or_abort(bar, parity, abort_flag))) {
            ok = false;
            *abort_flag = 1;
        }
        return ok;
    };
    Tile t;
    int h;
    // this CTA's key tiles of group g, and the first key of its i-th
    auto tiles_in = [&](const Tile &x, int g) {
        const int m = x.tiles(PAIR ? 0 : g, half);
        return SPLIT ? (m > rank ? (m - 1 - rank) / ranks + 1 : 0) : m;
    };
    auto tiles_of = [&](int g) { return tiles_in(t, g); };
    auto key_of = [&](int i) { return (SPLIT ? i * ranks + rank : i) * kKeys; };
    // Counters that run on over the items: ring slots used, first key tiles, and per group the queries' and the key
    // tiles' turns.  A barrier's phase in turn x of its resource has parity x & 1; of the barriers `full`, whose slots
    // also hold first tiles, each warp keeps the next phase's parity in a bit per slot.

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
        if (warp == 8) {
            // ---------------- TMA producer: per item Q, K0 V0 K1 V1 ... ----------------
            int slot = 0, turn = 0;          // ring stage and how often the ring has gone round
            int qturn[2] = {0, 0}, firsts = 0;
            uint32_t phase = 0, used = 0;    // per slot: parity of the next phase of `full`; whether there was one
            auto load = [&](const void *map, int x, int y, bool first) {
                if (turn > 0 && !wait(&b.empty[slot], (turn - 1) & 1)) return false;
                uint64_t *bar = first ? &b.first[firsts % kFirst] : &b.full[slot];
                if (lane == 0) {
                    uint8_t *dst = smem + 2 * L::QB + slot * L::TB;
                    tc::mbar_expect_tx(bar, L::TB);
#pragma unroll
                    for (int a = 0; a < D / 64; ++a)
                        tc::tma_load_3d(dst + a * (kKeys * 128), map, 64 * a, x, y, bar);
                }
                if (first) {
                    ++firsts;
                } else {
                    phase ^= 1u << slot;
                    used |= 1u << slot;
                }
                if (++slot == L::NST) {
                    slot = 0;
                    ++turn;
                }
                return true;
            };
            auto load_q = [&](int g, int h, int q) {
                if (qturn[g] > 0 && !wait(&b.q_empty[g], (qturn[g] - 1) & 1)) return false;
                if (lane == 0) {
                    tc::mbar_expect_tx(&b.q_full[g], L::QB);
#pragma unroll
                    for (int a = 0; a < D / 64; ++a)
                        tc::tma_load_3d(smem + g * L::QB + a * (128 * 128), &maps.q, 64 * a, h << pack, q,
                                        &b.q_full[g]);
                }
                ++qturn[g];
                return true;
            };
            if constexpr (PAIR) {
                // Q and K0 of either group, then by turns V0 K1, V1 K2, ...
                for (int j = 0; ok; ++j) {
                    Tile tg[2];
                    int hg[2], nt[2], kv[2];
                    if (!item_at(j, 0, &tg[0], &hg[0])) break;
                    item_at(j, 1, &tg[1], &hg[1]);
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        nt[g] = tiles_in(tg[g], g);
                        kv[g] = (hg[g] << pack) / G;
                        if (nt[g] > 0 && load_q(g, hg[g], tg[g].q)) load(&maps.k, kv[g], tg[g].k, true);
                    }
                    for (int i = 0; ok && i < max(nt[0], nt[1]); ++i)
#pragma unroll
                        for (int g = 0; g < 2; ++g)
                            if (ok && i < nt[g] && load(&maps.v, kv[g], tg[g].k + i * kKeys, false) && i + 1 < nt[g])
                                load(&maps.k, kv[g], tg[g].k + (i + 1) * kKeys, false);
                }
            }
            for (int j = 0; !PAIR && ok && item_at(j, 0, &t, &h); ++j) {
                const int kv = (h << pack) / G, nt0 = tiles_of(0), nt1 = tiles_of(1), ntiles = max(nt0, nt1);
                if (nt0 > 0 && !load_q(0, h, t.q)) break;
                if (ntiles > 0 && !load(&maps.k, kv, t.k + key_of(0), true)) break;
                if (nt1 > 0 && !load_q(1, h, t.q + half)) break;
                for (int i = 0; i < ntiles; ++i) {
                    if (!load(&maps.v, kv, t.k + key_of(i), false)) break;
                    if (i + 1 < ntiles && !load(&maps.k, kv, t.k + key_of(i + 1), false)) break;
                }
            }
            // every copy issued has landed before the CTA may exit
            for (int g = 0; g < 2; ++g)
                if (qturn[g] > 0 && !tc::mbar_wait(&b.q_full[g], (qturn[g] - 1) & 1)) ok = false;
            for (int s = 0; s < L::NST; ++s)
                if (used >> s & 1 && !tc::mbar_wait(&b.full[s], phase >> s & 1 ^ 1)) ok = false;
            for (int i = 0; i < kFirst; ++i) {
                const int n = (firsts + kFirst - 1 - i) / kFirst;
                if (n > 0 && !tc::mbar_wait(&b.first[i], (n - 1) & 1)) ok = false;
            }
        } else if (warp == 10) {
            // ---------------- gate: an iteration's operands are there ----------------
            // The MMA warp waits once per product pair: this warp waits for V(i) and K(i+1) in its place and
            // counts as a fifth arrival on the group's P barrier.
            int slot = 0, pturn[2] = {0, 0};
            uint32_t phase = 0;
            auto advance = [&]() { slot = slot + 1 == L::NST ? 0 : slot + 1; };
            auto wait_full = [&]() {
                const bool r = wait(&b.full[slot], phase >> slot & 1);
                phase ^= 1u << slot;
                advance();
                return r;
            };
            // waits for V at the ring's next slot, whose last `have` < 128 rows are the sequence's
            auto wait_v = [&](int have) {
                uint8_t *v = smem + 2 * L::QB + slot * L::TB;
                if (!wait_full()) return false;
                if (have < kKeys) {
                    // V rows behind the sequence's end are another sequence's (or none): they must not meet a
                    // zero probability, whatever they hold
                    for (int x = lane; x < (kKeys - have) * (D / 64) * 8; x += 32) {
                        const int c = x & 7, a = (x >> 3) % (D / 64), r = have + (x >> 3) / (D / 64);
                        *(uint4 *)(v + a * (kKeys * 128) + r * 128 + 16 * c) = make_uint4(0, 0, 0, 0);
                    }
                    tc::fence_smem_to_async();
                    __syncwarp();
                }
                return true;
            };
            auto arrive = [&](int g) {
                // one arrival per phase: the one before is complete
                if (pturn[g] > 0 && !wait(&b.p_full[g], (pturn[g] - 1) & 1)) return;
                if (lane == 0) tc::mbar_arrive(&b.p_full[g]);
                ++pturn[g];
            };
            if constexpr (PAIR) {
                for (int j = 0; ok; ++j) {
                    Tile tg[2];
                    int hg[2], nt[2];
                    if (!item_at(j, 0, &tg[0], &hg[0])) break;
                    item_at(j, 1, &tg[1], &hg[1]);
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        nt[g] = tiles_in(tg[g], g);
                        if (nt[g] > 0) advance();  // (K0 is the MMA warp's own wait)
                    }
                    for (int i = 0; ok && i < max(nt[0], nt[1]); ++i)
#pragma unroll
                        for (int g = 0; g < 2; ++g)
                            if (ok && i < nt[g] && wait_v(tg[g].keys - i * kKeys) && (i + 1 == nt[g] || wait_full()))
                                arrive(g);
                }
            }
            for (int j = 0; !PAIR && ok && item_at(j, 0, &t, &h); ++j) {
                const int nt0 = tiles_of(0), nt1 = tiles_of(1), ntiles = max(nt0, nt1);
                if (ntiles > 0) advance();  // K0 is the MMA warp's own wait
                for (int i = 0; i < ntiles && ok; ++i) {
                    if (!wait_v(t.keys - key_of(i))) break;
                    if (i + 1 < ntiles && !wait_full()) break;
#pragma unroll
                    for (int g = 0; g < 2; ++g)
                        if (ok && i < (g ? nt1 : nt0)) arrive(g);
                }
            }
        } else if (warp == 9) {
            // ---------------- MMA issuer ----------------
            const uint32_t id_s = tc::idesc_bf16(128, kKeys), id_o = tc::idesc_bf16(128, D, true);
            const uint32_t sq = tc::smem_u32(smem), ring = sq + 2 * L::QB;
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            const bool one = elect_one();
            int slot = 0, qturn[2] = {0, 0}, pturn[2] = {0, 0}, firsts = 0;
            auto advance = [&]() {
                const int s = slot;
                slot = slot + 1 == L::NST ? 0 : slot + 1;
                return s;
            };
            auto mma_s = [&](int g, int s) {
                if (one) {
                    const uint64_t aq = tc::desc_sw128(sq + g * L::QB), bk = tc::desc_sw128(ring + s * L::TB);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const int step = ((kk >> 2) * (128 * 128) + (kk & 3) * 32) >> 4;
                        tc::mma_bf16(tm + g * 128, aq + step, bk + step, id_s, kk > 0);
                    }
                    tc::commit(&b.s_full[g]);
                }
            };
            auto mma_o = [&](int g, int s, bool add) {
                if (one) {
                    const uint64_t bv = tc::desc_sw128_mn(ring + s * L::TB, kKeys * 128);
#pragma unroll
                    for (int kk = 0; kk < kKeys / 16; ++kk)
                        tc::mma_bf16_ts(tm + L::O_COL + g * D, tm + g * 128 + 8 * kk, bv + ((2048 * kk) >> 4), id_o,
                                        add || kk > 0);
                }
            };
            // an item's first product of group g, which has `mine` key tiles
            auto first_s = [&](int g, int s, int mine) {
                ++qturn[g];
                tc::fence_after_sync();
                mma_s(g, s);
                if (mine == 1 && one) tc::commit(&b.q_empty[g]);
            };
            auto there = [&](uint64_t *bar, uint32_t parity) {
                return __all_sync(0xffffffffu, tc::mbar_test(bar, parity));
            };
            if constexpr (PAIR) {
                for (int j = 0; ok; ++j) {
                    Tile tg[2];
                    int hg[2], nt[2];
                    if (!item_at(j, 0, &tg[0], &hg[0])) break;
                    item_at(j, 1, &tg[1], &hg[1]);
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        nt[g] = tiles_in(tg[g], g);
                        if (!ok || nt[g] == 0 || !wait(&b.first[firsts % kFirst], firsts / kFirst & 1) ||
                            !wait(&b.q_full[g], qturn[g] & 1))
                            continue;
                        ++firsts;
                        const int s = advance();
                        first_s(g, s, nt[g]);
                        if (one) tc::commit(&b.empty[s]);
                    }
                    for (int i = 0; ok && i < max(nt[0], nt[1]); ++i)
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            if (!ok || i >= nt[g] || !wait(&b.p_full[g], pturn[g] & 1)) continue;
                            tc::fence_after_sync();
                            ++pturn[g];
                            const int sv = advance();
                            mma_o(g, sv, i > 0);
                            if (one) {
                                tc::commit(&b.o_done[g]);
                                tc::commit(&b.empty[sv]);
                            }
                            if (i + 1 < nt[g]) {
                                const int sk = advance();
                                mma_s(g, sk);
                                if (one) {
                                    if (i + 2 == nt[g]) tc::commit(&b.q_empty[g]);
                                    tc::commit(&b.empty[sk]);
                                }
                            }
                        }
                }
            }
            Tile tn;
            int hn;
            bool more = !PAIR && item_at(0, 0, &tn, &hn);
            bool ahead = false;  // group 0's first product of the item is under way already
            for (int j = 0; ok && more; ++j) {
                t = tn;
                h = hn;
                more = item_at(j + 1, 0, &tn, &hn);
                const int nt0 = tiles_of(0), nt1 = tiles_of(1), ntiles = max(nt0, nt1);
                const int next0 = more ? tiles_in(tn, 0) : 0;
                if (ntiles == 0) continue;
                if (!ahead && !wait(&b.first[firsts % kFirst], firsts / kFirst & 1)) break;
                ++firsts;
                {
                    const int s = advance();
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const int mine = g ? nt1 : nt0;
                        if (mine == 0 || (g == 0 && ahead)) continue;
                        if (!wait(&b.q_full[g], qturn[g] & 1)) break;
                        first_s(g, s, mine);
                    }
                    if (!ok) break;
                    if (one) tc::commit(&b.empty[s]);
                    ahead = false;
                }
                // P V of key tile i and Q K^T of the next, both groups
                auto pair = [&](int i, auto last) {
                    const int sv = advance(), sk = last ? 0 : advance();
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const int mine = g ? nt1 : nt0;
                        // group 0 is done with this item and group 1 is not: its next one begins, if it is there
                        if (last && g == 1 && i >= nt0 && next0 > 0 &&
                            there(&b.first[firsts % kFirst], firsts / kFirst & 1) &&
                            there(&b.q_full[0], qturn[0] & 1)) {
                            first_s(0, slot, next0);
                            ahead = true;
                        }
                        if (i < mine) {
                            if (!wait(&b.p_full[g], pturn[g] & 1)) return;
                            tc::fence_after_sync();
                            mma_o(g, sv, i > 0);
                            ++pturn[g];
                            if (one) tc::commit(&b.o_done[g]);
                        }
                        if (!last && i + 1 < mine) {
                            mma_s(g, sk);
                            if (i + 2 == mine && one) tc::commit(&b.q_empty[g]);
                        }
                    }
                    if (one) {
                        tc::commit(&b.empty[sv]);
                        if (!last) tc::commit(&b.empty[sk]);
                    }
                };
                for (int i = 0; i + 1 < ntiles && ok; ++i) pair(i, std::false_type{});
                if (ok) pair(ntiles - 1, std::true_type{});
            }
            // every MMA issued has completed before the CTA may exit
            if (one) tc::commit(&b.drain);
            if (!tc::mbar_wait(&b.drain, 0)) ok = false;
        }
        if (SPLIT) {
            cluster_sync();  // (the softmax warps' two)
            cluster_sync();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        // ---------------- softmax: thread = row: a query and a head ----------------
        const int g = warp >> 2, row = (PAIR ? 0 : 128 * g) + (warp & 3) * 32 + lane;  // of the tile
        const int query = row >> pack;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + g * 128 + lanes, tO = tmem + L::O_COL + g * D + lanes;
        int turn = 0;  // of the group's S, P and O
        Tile tn;
        int hn;
        bool more = item_at(0, g, &tn, &hn);  // (the next item's tile is read while this one is worked on)
        for (int j = 0; ok && more; ++j) {
            t = tn;
            h = hn;
            more = item_at(j + 1, g, &tn, &hn);
            const int last = min(t.keys - 1, t.last + query);  // the row's last key
            const bool live = (row - lane) >> pack < t.rows;   // the warp has queries
            float ref = -INFINITY, sum = 0.f;                // reference maximum (raw scores), sum of P
            bool far = false;                                // a row of the warp has its reference beyond kFar
            const int tiles = tiles_of(g);
            const bool alone = !PAIR && tiles_of(g ^ 1) == 0;  // the special-function units are this group's
            for (int i = 0; i < tiles; ++i, ++turn) {
                if (!wait(&b.s_full[g], turn & 1)) break;
                tc::fence_after_sync();
                if (PAIR && !live) {  // (what tensor memory holds for these rows no other row's result has)
                    if (lane == 0) tc::mbar_arrive(&b.p_full[g]);
                    continue;
                }
                float s[128];
                __syncwarp();
                tmem_ld128(tS, (uint32_t *)s);
                const int left = last - key_of(i);  // columns 0 .. left are seen
                const bool cut = !__all_sync(0xffffffffu, left >= kKeys - 1);
                if (cut) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int x = left - 32 * c;  // columns 0 .. x of the 32
                        const uint32_t seen = x >= 31 ? ~0u : x < 0 ? 0u : (2u << x) - 1;
#pragma unroll
                        for (int y = 0; y < 32; ++y) s[32 * c + y] = seen >> y & 1 ? s[32 * c + y] : -INFINITY;
                    }
                }
                float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int c = 4; c < 124; c += 8)
#pragma unroll
                    for (int x = 0; x < 4; ++x) mx[x] = max3_nan(mx[x], s[c + x], s[c + 4 + x]);
                mx[0] = max3_nan(mx[0], s[124], s[125]);
                mx[1] = max3_nan(mx[1], s[126], s[127]);
                const float m = max3_nan(max3_nan(mx[0], mx[1], mx[2]), mx[3], mx[3]);
                // (the exponentials on the FMA units and the reference would lose a score that is NaN or infinite: the
                // sum keeps it, and the row is NaN, whichever key it was)
                if (!(m < INFINITY)) sum = NAN;
                // (before the first finite maximum ref is -inf and nothing has been summed; compared unscaled, the first
                // raise does not depend on the scale, however small: grow_at may be infinite)
                const bool grow = m - ref >= grow_at;
                if (__any_sync(0xffffffffu, grow)) {
                    const float to = grow ? m : ref;
                    const float f = grow ? (ref == -INFINITY ? 0.f : tc::ex2_fast((ref - m) * scale_log2)) : 1.f;
                    sum *= f;
                    ref = to;
                    far = __any_sync(0xffffffffu, fabsf(ref) < INFINITY && fabsf(ref * scale_log2) > kFar);
                    if (i > 0) {
                        if (!wait(&b.o_done[g], (turn - 1) & 1)) break;
                        tc::fence_after_sync();
#pragma unroll
                        for (int c = 0; c < D; c += 16) {
                            uint32_t o[16];
                            __syncwarp();
                            tmem_ld16(tO + c, o);
#pragma unroll
                            for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
                            __syncwarp();
                            tc::tmem_st16(tO + c, o);
                        }
                    }
                }
                float off = ref == -INFINITY ? 0.f : ref * scale_log2;
                if (__builtin_expect(far, false)) {
                    const float from = ref == -INFINITY ? 0.f : ref;
#pragma unroll
                    for (int c = 0; c < 128; ++c) s[c] -= from;
                    off = 0.f;
                }
                if (PAIR) to_p<true, true>(s, scale_log2, off, tS, __reduce_max_sync(0xffffffffu, left) + 1);
                else if (alone) to_p<false, false>(s, scale_log2, off, tS, 0);
                else to_p<true, false>(s, scale_log2, off, tS, 0);
                tc::tmem_st_wait();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&b.p_full[g]);
                // the sum, while the tensor cores work
                tc::f2_t add[4] = {};
#pragma unroll
                for (int c = 0; c < 128; c += 8)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        add[x] = f2_add(add[x], tc::f2_pack(s[c + 2 * x], s[c + 2 * x + 1]));
                float lo, hi;
                tc::f2_split(f2_add(f2_add(add[0], add[1]), f2_add(add[2], add[3])), lo, hi);
                sum += lo + hi;
            }
            // (a row that saw no key has no reference; its sum may hold the denormals of masked keys)
            if (ref == -INFINITY && sum == sum) sum = 0.f;
            const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
            if (tiles > 0 && ok) {
                wait(&b.o_done[g], (turn - 1) & 1);
                tc::fence_after_sync();
            }
            if constexpr (SPLIT) {
                // (reached by every softmax warp, also after a wait that ran out: nobody waits here alone)
                asm volatile("bar.sync 1, 256;" ::: "memory");  // both groups are done with the ring and with Q
                float *part = (float *)smem + row * D;
                float2 *ml = (float2 *)(smem + 256 * D * 4);
#pragma unroll
                for (int c = 0; c < D; c += 32) {
                    float o[32];
                    if (tiles > 0) {
                        __syncwarp();
                        tc::tmem_ld32(tO + c, o);
                    } else {
#pragma unroll
                        for (int y = 0; y < 32; ++y) o[y] = 0.f;
                    }
#pragma unroll
                    for (int y = 0; y < 8; ++y)
                        *(float4 *)(part + ((((c >> 2) + y) ^ (row & 7)) << 2)) =
                            make_float4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
                }
                ml[row] = make_float2(ref, sum);
                cluster_sync();
                const int share = 256 / ranks;
                for (int x = threadIdx.x; x < share * (D / 8); x += 256) {
                    const int r = rank * share + x / (D / 8), c = 2 * (x % (D / 8));
                    if ((r >> pack) >= t.rows) continue;
                    float top = -INFINITY, den = 0.f;
                    for (int w = 0; w < ranks; ++w) top = fmaxf(top, cluster.map_shared_rank(ml + r, w)->x);
                    if (top == -INFINITY) top = 0.f;
                    float acc[8] = {};
                    for (int w = 0; w < ranks; ++w) {
                        const float2 m = *cluster.map_shared_rank(ml + r, w);
                        const float f = tc::ex2_fast((m.x - top) * scale_log2);
                        den = fmaf(m.y, f, den);
                        float4 *from = (float4 *)((float *)smem + r * D);
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const float4 v = *cluster.map_shared_rank(from + ((c + y) ^ (r & 7)), w);
                            acc[4 * y] = fmaf(v.x, f, acc[4 * y]);
                            acc[4 * y + 1] = fmaf(v.y, f, acc[4 * y + 1]);
                            acc[4 * y + 2] = fmaf(v.z, f, acc[4 * y + 2]);
                            acc[4 * y + 3] = fmaf(v.w, f, acc[4 * y + 3]);
                        }
                    }
                    const float id = den > 0.f ? 1.f / den : (den == 0.f ? 0.f : den);
                    const size_t to = ((size_t)(t.q + (r >> pack)) * Hq + (h << pack) + (r & ((1 << pack) - 1))) * D + 4 * c;
                    *(uint4 *)(O + to) =
                        make_uint4(pack_bf16(acc[0] * id, acc[1] * id), pack_bf16(acc[2] * id, acc[3] * id),
                                   pack_bf16(acc[4] * id, acc[5] * id), pack_bf16(acc[6] * id, acc[7] * id));
                }
                cluster_sync();  // the parts stay readable until every CTA has joined its rows
                break;
            }
            if (!ok) break;
            // 64 columns at a time through this warp's piece of shared memory (16-byte pieces XORed with the row, as
            // the 128-byte swizzle has them), from where TMA stores the warp's rows; if some of them lie behind the
            // sequence's end, the others are stored by eight lanes per 128 bytes
            uint8_t *stage = smem + L::OUT + warp * (32 * 128);
            const int first = (row - lane) >> pack;  // the warp's first query
            const bool all = t.rows - first >= 32 >> pack;
#pragma unroll
            for (int c = 0; c < D; c += 64) {
                if (PAIR && !live) break;
                uint4 w[8];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float o[32];
                    if (tiles > 0) {
                        __syncwarp();
                        tc::tmem_ld32(tO + c + 32 * x, o);
                    } else {
#pragma unroll
                        for (int y = 0; y < 32; ++y) o[y] = 0.f;
                    }
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        w[4 * x + y] = make_uint4(pack_bf16(o[8 * y] * inv, o[8 * y + 1] * inv),
                                                  pack_bf16(o[8 * y + 2] * inv, o[8 * y + 3] * inv),
                                                  pack_bf16(o[8 * y + 4] * inv, o[8 * y + 5] * inv),
                                                  pack_bf16(o[8 * y + 6] * inv, o[8 * y + 7] * inv));
                }
                if (lane == 0) tc::bulk_wait_read();
                __syncwarp();
#pragma unroll
                for (int y = 0; y < 8; ++y) *(uint4 *)(stage + lane * 128 + ((y ^ (lane & 7)) << 4)) = w[y];
                if (all) tc::fence_smem_to_async();
                __syncwarp();
                if (all) {
                    if (lane == 0) {
                        tc::tma_store_3d(&maps.o, stage, c, h << pack, t.q + first);
                        tc::bulk_commit();
                    }
                    continue;
                }
#pragma unroll
                for (int y = 0; y < 8; ++y) {
                    const int l = 4 * y + (lane >> 3), r = row - lane + l;  // that lane's row
                    const uint4 v = *(const uint4 *)(stage + l * 128 + (((lane & 7) ^ (l & 7)) << 4));
                    const int ry = r >> pack, rh = r & ((1 << pack) - 1);
                    if (ry < t.rows)
                        *(uint4 *)(O + ((size_t)(t.q + ry) * Hq + (h << pack) + rh) * D + c + 8 * (lane & 7)) = v;
                }
            }
            // (the next item's first product into O follows this group's next arrival on p_full)
            tc::fence_before_sync();
        }
        if (lane == 0) tc::bulk_wait();
    }
    if (!ok && lane == 0) record_error(counters, kDevErrTimeout);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 9) {
        __syncwarp();
        tc::tmem_dealloc(tmem, 512);
    }
}

// [rows, heads, D] bf16, boxes of 64 elements x 2^pack heads x box_rows/2^pack rows, 128-byte swizzle
bool rows_map(CUtensorMap *map, const void *ptr, int d, int heads, int rows, int pack, int box_rows = 128) {
    auto enc = (PFN_cuTensorMapEncodeTiled_v12000)tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows};
    cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)heads * d * 2};
    cuuint32_t box[3] = {64, 1u << pack, (cuuint32_t)box_rows >> pack};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch_d(const PagedPlan &p, int n, int total_q, int total_k, const void *Q, const void *K, const void *V,
                     const int32_t *cu_q, const int32_t *cu_k, void *O, void *ws, cudaStream_t s) {
    const mono_paged_config &c = p.cfg;
    Maps maps;
    // without keys the maps of K and V are never used: any valid one will do
    const int pack = prompt_pack_log2(c), chunks = c.Hq >> pack;
    if (!rows_map(&maps.q, Q, D, c.Hq, total_q, pack) || !rows_map(&maps.o, O, D, c.Hq, total_q, pack, 32) ||
        !rows_map(&maps.k, total_k ? K : Q, D, total_k ? c.Hkv : c.Hq, total_k ? total_k : total_q, 0) ||
        !rows_map(&maps.v, total_k ? V : Q, D, total_k ? c.Hkv : c.Hq, total_k ? total_k : total_q, 0))
        return cudaErrorInvalidValue;
    cudaError_t e;
    int dev = 0, sms = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    // Sequences that on average fit into one group, and enough of them: the groups take an item each, with keys of
    // their own; one group of a shared item would have no rows.  (500 sequences of 30 tokens, 16 heads of 64: 171 us shared,
    // 136 so; 64 of 100 tokens, 8 heads of 128: 22.6 and 18.0.  100 of 100 tokens, 16 heads over 4, which the rule
    // leaves shared, 35 us.)
    const int group_rows = 128 >> pack;
    const bool pair = total_q / n < group_rows && ((long long)total_q / group_rows + n) * chunks > sms;
    const int qt = (pair ? 128 : 256) >> pack, most = total_q / qt + n;  // query tiles
    const int items = most * chunks;
    unsigned long long *counters = (unsigned long long *)pg_ptr(p, ws, kPgCounters);
    const int group = c.Hq / c.Hkv;
    const float grow_at = kGrow / p.scale_log2;
    const Tile *no_list = nullptr;
    const int *no_count = nullptr;
    // Few items over many keys: clusters split the keys, as far as every CTA finds an SM and, on average, four key
    // tiles (256 queries after 32,512 tokens, 16 heads over 4: 392 us without, 123 with 8 CTAs; the joins cost about
    // 5 us, 512 tokens alone 14 and 20 us).
    int ranks = 8;
    while (ranks > 1 && (pair || ranks * items > sms || ranks * 4 * kKeys > total_k / n)) ranks /= 2;
    if (ranks > 1) {
        auto kern = k_prompt_tc<D, kSplit>;
        if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<D>::BYTES)) != cudaSuccess)
            return e;
        e = launch_after_cluster(kern, dim3(items * ranks), dim3(kThreads), Lay<D>::BYTES, s, ranks, maps, cu_q, cu_k,
                                 (bf16 *)O, no_list, no_count, n, total_q, total_k, c.Hq, group, pack, p.scale_log2,
                                 grow_at, counters);
        count_launches(1);
        return e;
    }
    auto kern = pair ? k_prompt_tc<D, kPair> : k_prompt_tc<D, kShared>;
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<D>::BYTES)) != cudaSuccess)
        return e;
    if (!pair && items <= sms) {  // a CTA per item: no list
        e = launch_after(kern, dim3(items), dim3(kThreads), Lay<D>::BYTES, s, maps, cu_q, cu_k, (bf16 *)O, no_list,
                         no_count, n, total_q, total_k, c.Hq, group, pack, p.scale_log2, grow_at, counters);
        count_launches(1);
        return e;
    }
    Tile *list = (Tile *)pg_ptr(p, ws, kPgWork);
    int *count = (int *)(counters + kPagedTiles);
    if ((e = launch_after(k_prompt_list, dim3(1), dim3(1024), 0, s, cu_q, cu_k, n, total_q, total_k, qt,
                          (int *)pg_ptr(p, ws, kPgPrefix), list, count, most, counters)) != cudaSuccess)
        return e;
    if ((e = launch_after(kern, dim3(sms), dim3(kThreads), Lay<D>::BYTES, s, maps, cu_q, cu_k, (bf16 *)O, list,
                          count, n, total_q, total_k, c.Hq, group, pack, p.scale_log2, grow_at, counters)) != cudaSuccess)
        return e;
    count_launches(2);
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_prompt_tc(const PagedPlan &p, int n, int total_q, int total_k, const void *Q, const void *K,
                             const void *V, const int32_t *cu_q, const int32_t *cu_k, void *O, void *ws,
                             cudaStream_t s) {
    if (p.cfg.d == 64) return launch_d<64>(p, n, total_q, total_k, Q, K, V, cu_q, cu_k, O, ws, s);
    return launch_d<128>(p, n, total_q, total_k, Q, K, V, cu_q, cu_k, O, ws, s);
}

}  // namespace mono
