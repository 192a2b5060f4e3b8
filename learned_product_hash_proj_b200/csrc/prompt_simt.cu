// prompt_simt.cu -- causal attention over packed prompts with fp32 FMAs.
//
//   o_i = sum_{j <= i + lk - lq} softmax_j(scale <q_i, k_j>) v_j   per sequence and query head
//
// A cluster of 1, 2 or 4 CTAs per (64 query rows of a sequence, query head),
// those with the most keys first over all heads.  The CTAs, and the groups of
// 8 x TX threads in each, take the key tiles in turn, with a running maximum
// and sum of their own; at the end each CTA joins its share of the rows out of
// all the groups' shared memory.  A thread holds 8 rows x 64/TX keys of a
// 64-key tile's scores and 8 rows x d/TX columns of the output, all in fp32.
// The next tile's K is fetched (cp.async) while the scores are turned into the
// output, its V while the next scores are made.  Rows in shared memory are
// padded by 16 bytes: eight consecutive rows' pieces then lie in different
// banks.
//
// Measured on one B200: 2,048 tokens, 16 heads of 64 over 8, 242 us (half of
// the FMA rate); of 128, 462 us.  It is bound by shared-memory reads (a
// 16-byte read of a warp takes two to four cycles however many lanes share
// the address) and, with the 8 x 8 tiles that need fewer of them, by the
// latency that 8 warps per SM leave open.  At d = 64: 4 x 4 tiles in 16 warps
// 262 us, 8 x 4 in 16 warps 271, 8 x 8 in 8 warps 254 without and 242 with the
// fetch ahead.  Every CTA finds its tile by a scan of all cumulative lengths, which
// tells with thousands of short sequences (2,000 of 2 tokens, 16 heads of 64:
// 2.87 ms).
#include <cooperative_groups.h>

#include "paged.cuh"

namespace cg = cooperative_groups;

namespace mono {

namespace {

constexpr int QT = 64, KT = 64;
template <int D>
struct Simt {
    static constexpr int TX = D == 64 ? 8 : 16;     // threads along the keys and the output's columns
    static constexpr int CS = KT / TX;              // keys per thread
    static constexpr int CO = D / TX / 4;           // output columns per thread, in fours
    static constexpr int GT = 8 * TX;               // threads of a group
    static constexpr int NG = D == 64 ? 4 : 2, NT = NG * GT;
    static constexpr int P = D / 4;                 // 16-byte pieces of a row
    static constexpr int PD = P + 1;                // of a padded row of q or k
    static constexpr int PP = KT / 4 + 1;           // of p
    static constexpr int GROUP = KT * PD + KT * P + QT * PP;  // K, V and P of a group
    static constexpr int BYTES = (QT * PD + NG * GROUP) * 16;
};

struct alignas(16) F4 {
    tc::f2_t xy, zw;
};

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all but this thread's latest group of copies have landed
__device__ __forceinline__ void cp_async_wait_but_one() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }

template <int D>
__global__ void __launch_bounds__(Simt<D>::NT, 1)
    k_prompt_simt(const float *__restrict__ Q, const float *__restrict__ K, const float *__restrict__ V,
                  const int32_t *__restrict__ cu_q, const int32_t *__restrict__ cu_k, float *__restrict__ O, int n,
                  int total_q, int total_k, int Hq, int Hkv, float scale_log2, unsigned long long *counters) {
    using S = Simt<D>;
    constexpr int P = S::P, PD = S::PD, PP = S::PP, TX = S::TX, CS = S::CS, CO = S::CO, GT = S::GT, NG = S::NG,
                  NT = S::NT;
    extern __shared__ __align__(16) float4 smem4[];
    const int group = threadIdx.x / GT, tid = threadIdx.x % GT, tx = tid % TX, ty = tid / TX;
    float4 *sQ = smem4, *sK = sQ + QT * PD + group * S::GROUP, *sV = sK + KT * PD, *sP = sV + KT * P;
    __shared__ int s_w[NT / 32 + 1], s_out[2];
    __shared__ float2 s_ml[NG][QT];
    auto group_sync = [&]() { asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(GT) : "memory"); };
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    const int item = blockIdx.x / ranks;
    int seq, row0;
    if (!find_tile<NT>(cu_q, n, total_q, QT, item / Hq, s_w, s_out, &seq, &row0, counters)) return;
    const int h = item % Hq, kv = h / (Hq / Hkv);
    const Span sq = cu_span(cu_q, seq, total_q, counters), sk = cu_span(cu_k, seq, total_k, counters);
    const int q0 = sq.at, lq = sq.n, k0 = sk.at, lk = sk.n;
    const int shift = lk - lq;  // row i sees keys j <= i + shift
    const int keys = min(lk, min(lq, row0 + QT) + shift);

    // rows j0 .. j0+63 of K (padded) or V into shared memory, zeros behind the sequence's end
    const float *k = K + ((size_t)k0 * Hkv + kv) * D, *v = V + ((size_t)k0 * Hkv + kv) * D;
    auto fetch = [&](float4 *dst, int pitch, const float *src, int j0) {
        if (j0 < keys) {
#pragma unroll 4
            for (int i = tid; i < KT * P; i += GT) {
                const int r = i / P, c = i % P;
                const bool in = j0 + r < lk;
                tc::cp_async16(dst + r * pitch + c, (const float4 *)src + (in ? (size_t)(j0 + r) * Hkv * P + c : 0), in);
            }
        }
        cp_async_commit();
    };
    const int step = ranks * NG * KT, first = (group * ranks + rank) * KT;
    fetch(sK, PD, k, first);
    fetch(sV, P, v, first);
    const float *q = Q + ((size_t)(q0 + row0) * Hq + h) * D;
    for (int i = threadIdx.x; i < QT * P; i += NT) {
        const int r = i / P, c = i % P;
        sQ[r * PD + c] = row0 + r < lq ? __ldg((const float4 *)(q + (size_t)r * Hq * D) + c)
                                       : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    tc::f2_t o[8][2 * CO] = {};
    float m[8], l[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
    }
    __syncthreads();
    for (int j0 = first; j0 < keys; j0 += step) {
        cp_async_wait_but_one();  // K
        group_sync();
        float s[8][CS] = {};
        {
            const float4 *pa = sQ + ty * PD, *pb = sK + tx * PD;
#pragma unroll 2
            for (int c = 0; c < P; ++c) {
                float4 b[CS];
#pragma unroll
                for (int j = 0; j < CS; ++j) b[j] = pb[TX * j * PD + c];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float4 a = pa[8 * i * PD + c];
#pragma unroll
                    for (int j = 0; j < CS; ++j) {
                        s[i][j] = fmaf(a.x, b[j].x, s[i][j]);
                        s[i][j] = fmaf(a.y, b[j].y, s[i][j]);
                        s[i][j] = fmaf(a.z, b[j].z, s[i][j]);
                        s[i][j] = fmaf(a.w, b[j].w, s[i][j]);
                    }
                }
            }
        }
        group_sync();  // K is done with
        fetch(sK, PD, k, j0 + step);
#pragma unroll
        for (int i = 0; i < 8; ++i)  // (rounded here: a row's largest weight is exactly 1)
#pragma unroll
            for (int j = 0; j < CS; ++j) s[i][j] = __fmul_rn(s[i][j], scale_log2);
        if (j0 + KT > min(lk, row0 + shift + 1)) {  // some row does not see some key of the tile
            asm volatile("");                       // (a branch, not a select per score of every tile)
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int j = 0; j < CS; ++j) {
                    const int key = j0 + tx + TX * j;
                    s[i][j] = key <= row0 + ty + 8 * i + shift && key < lk ? s[i][j] : -INFINITY;
                }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float mx = s[i][0];
#pragma unroll
            for (int j = 1; j < CS; ++j) mx = fmaxf(mx, s[i][j]);
#pragma unroll
            for (int x = 1; x < TX; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
            const float mn = fmaxf(m[i], mx), ms = mn == -INFINITY ? 0.f : mn;
            const float f = tc::ex2_fast(m[i] - ms);
            m[i] = mn;
            l[i] *= f;
            const tc::f2_t ff = tc::f2_dup(f);
#pragma unroll
            for (int e = 0; e < 2 * CO; ++e) o[i][e] = tc::f2_fma(o[i][e], ff, 0);
#pragma unroll
            for (int j = 0; j < CS; ++j) {
                const float p = tc::ex2_fast(s[i][j] - ms);
                l[i] += p;
                ((float *)(sP + (ty + 8 * i) * PP))[tx + TX * j] = p;
            }
        }
        cp_async_wait_but_one();  // V
        group_sync();             // (and P, although a row's threads are in one warp)
        const float4 *pp = sP + ty * PP;
        const F4 *pv = (const F4 *)sV + tx;
#pragma unroll 2
        for (int c = 0; c < KT / 4; ++c) {
            F4 b[4][CO];
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int e = 0; e < CO; ++e) b[x][e] = pv[(4 * c + x) * P + TX * e];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float4 a = pp[8 * i * PP + c];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const tc::f2_t p = tc::f2_dup(x == 0 ? a.x : x == 1 ? a.y : x == 2 ? a.z : a.w);
#pragma unroll
                    for (int e = 0; e < CO; ++e) {
                        o[i][2 * e] = tc::f2_fma(p, b[x][e].xy, o[i][2 * e]);
                        o[i][2 * e + 1] = tc::f2_fma(p, b[x][e].zw, o[i][2 * e + 1]);
                    }
                }
            }
        }
        group_sync();  // V and P are done with
        fetch(sV, P, v, j0 + step);
    }
    tc::cp_async_wait_all();
    // join: every group leaves its output (where its V was), maxima and sums; each CTA finishes its share of the rows
    group_sync();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int x = 1; x < TX; x <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], x);
        if (tx == 0) s_ml[group][ty + 8 * i] = make_float2(m[i], l[i]);
#pragma unroll
        for (int e = 0; e < CO; ++e) ((F4 *)sV)[(ty + 8 * i) * P + tx + TX * e] = {o[i][2 * e], o[i][2 * e + 1]};
    }
    cluster.sync();
    const float4 *so = smem4 + QT * PD + KT * PD;  // group 0's output
    const int share = QT / ranks;
    for (int x = threadIdx.x; x < share * P; x += NT) {
        const int r = rank * share + x / P, c = x % P;
        if (row0 + r >= lq) break;
        float mx = -INFINITY, sum = 0.f;
        for (int w = 0; w < ranks; ++w)
#pragma unroll
            for (int g = 0; g < NG; ++g) mx = fmaxf(mx, cluster.map_shared_rank(&s_ml[g][r], w)->x);
        const float ms = mx == -INFINITY ? 0.f : mx;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = 0; w < ranks; ++w)
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const float2 part = *cluster.map_shared_rank(&s_ml[g][r], w);
                const float f = exp2f(part.x - ms);
                const float4 y = *cluster.map_shared_rank(so + g * S::GROUP + r * P + c, w);
                sum = fmaf(part.y, f, sum);
                acc.x = fmaf(y.x, f, acc.x);
                acc.y = fmaf(y.y, f, acc.y);
                acc.z = fmaf(y.z, f, acc.z);
                acc.w = fmaf(y.w, f, acc.w);
            }
        const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
        ((float4 *)(O + ((size_t)(q0 + row0 + r) * Hq + h) * D))[c] =
            make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    }
    cluster.sync();  // the parts stay readable until every CTA has joined its rows
}

template <int D>
cudaError_t launch_d(const PagedPlan &p, int n, int total_q, int total_k, const void *Q, const void *K, const void *V,
                     const int32_t *cu_q, const int32_t *cu_k, void *O, void *ws, cudaStream_t s) {
    cudaError_t e =
        cudaFuncSetAttribute(k_prompt_simt<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Simt<D>::BYTES);
    if (e != cudaSuccess) return e;
    int dev = 0, sms = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    const int items = (int)prompt_items(p.cfg, n, total_q);
    // Few items: their keys are split, or SMs stay idle (64 items of 2,000 keys, d = 128: 244 us with one CTA each, 130
    // with two, 87 with four; 136 of 1,024, d = 64: 66, 52, 78).  With more of them the CTAs' fixed cost, about a key
    // tile's work, tells (198 items of 2,048 keys, d = 128: 248, 204, 250; 264 of them, d = 64: 124, 144, 206).
    int ranks = 2ll * items <= sms ? 4 : 2ll * items <= 3 * sms ? 2 : 1;
    while (ranks > 1 && ranks * KT > total_k) ranks /= 2;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(items * ranks);
    lc.blockDim = dim3(Simt<D>::NT);
    lc.dynamicSmemBytes = Simt<D>::BYTES;
    lc.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ranks;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    lc.attrs = at;
    lc.numAttrs = 1;
    e = cudaLaunchKernelEx(&lc, k_prompt_simt<D>, (const float *)Q, (const float *)K, (const float *)V, cu_q, cu_k,
                           (float *)O, n, total_q, total_k, p.cfg.Hq, p.cfg.Hkv, p.scale_log2,
                           (unsigned long long *)pg_ptr(p, ws, kPgCounters));
    count_launches(1);
    return e;
}

}  // namespace

cudaError_t launch_prompt_simt(const PagedPlan &p, int n, int total_q, int total_k, const void *Q, const void *K,
                               const void *V, const int32_t *cu_q, const int32_t *cu_k, void *O, void *ws,
                               cudaStream_t s) {
    if (p.cfg.d == 64) return launch_d<64>(p, n, total_q, total_k, Q, K, V, cu_q, cu_k, O, ws, s);
    return launch_d<128>(p, n, total_q, total_k, Q, K, V, cu_q, cu_k, O, ws, s);
}

}  // namespace mono
