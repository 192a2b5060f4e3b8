// prompt_simt.cu -- causal attention over packed prompts with fp32 FMAs.
//
//   o_i = sum_{j <= i + lk - lq} softmax_j(scale <q_i, k_j>) v_j   per sequence and query head
//
// A cluster of 1, 2 or 4 CTAs per (64 query rows of a sequence, query head),
// those with the most keys first over all heads.  The CTAs, and two groups of
// 256 threads in each, take the key tiles in turn, with a running maximum and
// sum of their own; at the end each CTA joins its share of the rows out of all
// the groups' shared memory.  A group is a 16 x 16 grid: a thread holds 4 x 4
// scores of a 64-key tile and 4 x d/16 of the output, all in fp32.  Products
// go two at a time (fma.rn.f32x2), so that the loads and address steps between
// them find issue slots.  Rows in shared memory are padded by 16 bytes: eight
// consecutive rows' pieces then lie in different banks.  P takes K's place.
#include <cooperative_groups.h>
#include <limits.h>

#include "paged.cuh"

namespace cg = cooperative_groups;

namespace mono {

namespace {

constexpr int QT = 64, KT = 64;
constexpr int kGroups = 2, kGroupThreads = 256, kThreads = kGroups * kGroupThreads;

template <int D>
struct Simt {
    static constexpr int P = D / 4;        // 16-byte pieces of a row
    static constexpr int PD = P + 1;       // of a padded row of q or k
    static constexpr int PP = KT / 4 + 1;  // of p
    static constexpr int GROUP = KT * PD + KT * P;  // K (then P) and V of a group
    static constexpr int BYTES = (QT * PD + kGroups * GROUP) * 16;
};

struct alignas(16) F4 {
    tc::f2_t xy, zw;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    k_prompt_simt(const float *__restrict__ Q, const float *__restrict__ K, const float *__restrict__ V,
                  const int32_t *__restrict__ cu_q, const int32_t *__restrict__ cu_k, float *__restrict__ O, int n,
                  int total_q, int total_k, int Hq, int Hkv, float scale_log2) {
    using S = Simt<D>;
    constexpr int P = S::P, PD = S::PD, PP = S::PP;
    extern __shared__ __align__(16) float4 smem4[];
    const int group = threadIdx.x / kGroupThreads, tid = threadIdx.x % kGroupThreads, tx = tid & 15, ty = tid >> 4;
    float4 *sQ = smem4, *sK = sQ + QT * PD + group * S::GROUP, *sV = sK + KT * PD, *sP = sK;
    __shared__ int s_w[kThreads / 32 + 1], s_out[2];
    __shared__ float2 s_ml[kGroups][QT];
    auto group_sync = [&]() { asm volatile("bar.sync %0, 256;" ::"r"(1 + group) : "memory"); };
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    const int item = blockIdx.x / ranks;
    int seq, row0;
    if (!find_tile<kThreads>(cu_q, n, total_q, QT, item / Hq, s_w, s_out, &seq, &row0)) return;
    const int h = item % Hq, kv = h / (Hq / Hkv);
    const int q0 = cu_at(cu_q, seq, total_q), lq = cu_at(cu_q, seq + 1, total_q) - q0;
    const int k0 = cu_at(cu_k, seq, total_k), lk = max(0, cu_at(cu_k, seq + 1, total_k) - k0);
    const int shift = lk - lq;  // row i sees keys j <= i + shift
    const int keys = min(lk, min(lq, row0 + QT) + shift);

    const float *q = Q + ((size_t)(q0 + row0) * Hq + h) * D;
    for (int i = threadIdx.x; i < QT * P; i += kThreads) {
        const int r = i / P, c = i % P;
        sQ[r * PD + c] = row0 + r < lq ? __ldg((const float4 *)(q + (size_t)r * Hq * D) + c)
                                       : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    tc::f2_t o[4][D / 32] = {};
    float m[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
    }
    const float *k = K + ((size_t)k0 * Hkv + kv) * D, *v = V + ((size_t)k0 * Hkv + kv) * D;
    __syncthreads();
    for (int j0 = (rank * kGroups + group) * KT; j0 < keys; j0 += ranks * kGroups * KT) {
        group_sync();
        for (int i = tid; i < KT * P; i += kGroupThreads) {
            const int r = i / P, c = i % P;
            const bool in = j0 + r < lk;
            const size_t g = (size_t)(j0 + r) * Hkv * P + c;
            sK[r * PD + c] = in ? __ldg((const float4 *)k + g) : make_float4(0.f, 0.f, 0.f, 0.f);
            sV[r * P + c] = in ? __ldg((const float4 *)v + g) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        group_sync();
        float s[4][4];
        {
            tc::f2_t acc[4][4] = {};
            const F4 *pa = (const F4 *)(sQ + ty * 4 * PD), *pb = (const F4 *)(sK + tx * PD);
#pragma unroll 8
            for (int c = 0; c < P; ++c) {
                F4 a[4], b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) a[i] = pa[i * PD + c];
#pragma unroll
                for (int j = 0; j < 4; ++j) b[j] = pb[16 * j * PD + c];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        acc[i][j] = tc::f2_fma(a[i].xy, b[j].xy, acc[i][j]);
                        acc[i][j] = tc::f2_fma(a[i].zw, b[j].zw, acc[i][j]);
                    }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float lo, hi;
                    tc::f2_split(acc[i][j], lo, hi);
                    s[i][j] = lo + hi;
                }
        }
        group_sync();  // K is done with: P takes its place
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int last = row0 + ty * 4 + i + shift;  // the row's last key
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int key = j0 + tx + 16 * j;
                s[i][j] = key <= last && key < lk ? s[i][j] * scale_log2 : -INFINITY;
                mx = fmaxf(mx, s[i][j]);
            }
#pragma unroll
            for (int x = 1; x < 16; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
            const float mn = fmaxf(m[i], mx), ms = mn == -INFINITY ? 0.f : mn;
            const float f = exp2f(m[i] - ms);
            m[i] = mn;
            l[i] *= f;
            const tc::f2_t ff = tc::f2_dup(f);
#pragma unroll
            for (int e = 0; e < D / 32; ++e) o[i][e] = tc::f2_fma(o[i][e], ff, 0);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = exp2f(s[i][j] - ms);
                l[i] += p;
                ((float *)(sP + (ty * 4 + i) * PP))[tx + 16 * j] = p;
            }
        }
        __syncwarp();  // a row's 16 threads are one half of a warp
        const float4 *pp = sP + ty * 4 * PP;
        const F4 *pv = (const F4 *)sV + tx;
#pragma unroll 2
        for (int c = 0; c < KT / 4; ++c) {
            float4 a[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = pp[i * PP + c];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                tc::f2_t p[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    p[i] = tc::f2_dup(x == 0 ? a[i].x : x == 1 ? a[i].y : x == 2 ? a[i].z : a[i].w);
#pragma unroll
                for (int e = 0; e < D / 64; ++e) {
                    const F4 b = pv[(4 * c + x) * P + 16 * e];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        o[i][2 * e] = tc::f2_fma(p[i], b.xy, o[i][2 * e]);
                        o[i][2 * e + 1] = tc::f2_fma(p[i], b.zw, o[i][2 * e + 1]);
                    }
                }
            }
        }
    }
    // join: every group leaves its output (where its V was), maxima and sums; each CTA finishes its share of the rows
    group_sync();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int x = 1; x < 16; x <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], x);
        if (tx == 0) s_ml[group][ty * 4 + i] = make_float2(m[i], l[i]);
#pragma unroll
        for (int e = 0; e < D / 64; ++e) ((F4 *)sV)[(ty * 4 + i) * P + tx + 16 * e] = {o[i][2 * e], o[i][2 * e + 1]};
    }
    cluster.sync();
    const float4 *so = smem4 + QT * PD + KT * PD;  // group 0's output
    const int share = QT / ranks;
    for (int x = threadIdx.x; x < share * P; x += kThreads) {
        const int r = rank * share + x / P, c = x % P;
        if (row0 + r >= lq) break;
        float mx = -INFINITY, sum = 0.f;
        for (int w = 0; w < ranks; ++w)
#pragma unroll
            for (int g = 0; g < kGroups; ++g) mx = fmaxf(mx, cluster.map_shared_rank(&s_ml[g][r], w)->x);
        const float ms = mx == -INFINITY ? 0.f : mx;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = 0; w < ranks; ++w)
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
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
                     const int32_t *cu_q, const int32_t *cu_k, void *O, cudaStream_t s) {
    cudaError_t e =
        cudaFuncSetAttribute(k_prompt_simt<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Simt<D>::BYTES);
    if (e != cudaSuccess) return e;
    int dev = 0, sms = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    const long long items = ((long long)total_q / QT + n) * p.cfg.Hq;
    // Few items: their keys are split, or SMs stay idle (64 items of 2,000 keys, d = 128: 246 us with one CTA each, 130
    // with two, 93 with four; 136 of 1,024, d = 64: 74, 52, 74).  With more of them the CTAs' fixed cost, about a key
    // tile's work, tells (198 items of 2,048 keys, d = 128: 249, 203, 264; 264 of them, d = 64: 139, 153, 207).
    int ranks = 2 * items <= sms ? 4 : 2 * items <= 3 * sms ? 2 : 1;
    while (ranks > 1 && ranks * kGroups * KT > total_k) ranks /= 2;
    if (items * ranks > INT_MAX) return cudaErrorInvalidValue;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((unsigned)(items * ranks));
    lc.blockDim = dim3(kThreads);
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
                           (float *)O, n, total_q, total_k, p.cfg.Hq, p.cfg.Hkv, p.scale_log2);
    count_launches(1);
    return e;
}

}  // namespace

cudaError_t launch_prompt_simt(const PagedPlan &p, int n, int total_q, int total_k, const void *Q, const void *K,
                               const void *V, const int32_t *cu_q, const int32_t *cu_k, void *O, void *,
                               cudaStream_t s) {
    if (p.cfg.d == 64) return launch_d<64>(p, n, total_q, total_k, Q, K, V, cu_q, cu_k, O, s);
    return launch_d<128>(p, n, total_q, total_k, Q, K, V, cu_q, cu_k, O, s);
}

}  // namespace mono
