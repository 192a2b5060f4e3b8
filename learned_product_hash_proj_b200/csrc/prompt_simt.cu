// prompt_simt.cu -- causal attention over packed prompts with fp32 FMAs.
//
//   o_i = sum_{j <= i + lk - lq} softmax_j(scale <q_i, k_j>) v_j   per sequence and query head
//
// One CTA per (64 query rows of a sequence, query head), 256 threads as a
// 16 x 16 grid: a thread holds 4 x 4 scores of a 64-key tile and 4 x d/16 of
// the output, a running maximum and sum per row, all in fp32.  Rows of q, k, v
// and p lie in shared memory as 16-byte pieces XORed with the row, so that the
// reads of 8 consecutive rows and of 8 consecutive pieces are both free of
// bank conflicts.
#include "paged.cuh"

namespace mono {

namespace {

constexpr int QT = 64, KT = 64;

template <int D>
struct Simt {
    static constexpr int BYTES = (QT + 2 * KT) * D * 4 + QT * KT * 4;
};

// piece c (16 bytes) of row r in a tile of rows of `pieces` pieces
__device__ __forceinline__ int at16(int r, int c, int pieces) { return r * pieces + (c ^ (r & 7)); }

template <typename T>
__device__ __forceinline__ float4 load4(const T *p);
template <>
__device__ __forceinline__ float4 load4<float>(const float *p) {
    return __ldg((const float4 *)p);
}

template <typename T, int D>
__global__ void __launch_bounds__(256, 2) k_prompt_simt(const T *__restrict__ Q, const T *__restrict__ K,
                                                        const T *__restrict__ V, const int32_t *__restrict__ cu_q,
                                                        const int32_t *__restrict__ cu_k, T *__restrict__ O, int n,
                                                        int total_q, int total_k, int Hq, int Hkv, float scale_log2,
                                                        unsigned long long *__restrict__ counters) {
    constexpr int P = D / 4;  // pieces of a row
    extern __shared__ __align__(16) float4 smem4[];
    float4 *sQ = smem4, *sK = sQ + QT * P, *sV = sK + KT * P, *sP = sV + KT * P;
    __shared__ int s_w[9], s_out[2];
    int seq, row0;
    if (!find_tile<256>(cu_q, n, total_q, QT, blockIdx.x, s_w, s_out, &seq, &row0)) return;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int h = blockIdx.y, kv = h / (Hq / Hkv);
    const int q0 = cu_at(cu_q, seq, total_q), lq = cu_at(cu_q, seq + 1, total_q) - q0;
    const int k0 = cu_at(cu_k, seq, total_k), lk = max(0, cu_at(cu_k, seq + 1, total_k) - k0);
    const int shift = lk - lq;  // row i sees keys j <= i + shift
    const int keys = min(lk, min(lq, row0 + QT) + shift);

    const T *q = Q + ((size_t)(q0 + row0) * Hq + h) * D;
    for (int i = tid; i < QT * P; i += 256) {
        const int r = i / P, c = i % P;
        sQ[at16(r, c, P)] = row0 + r < lq ? load4(q + (size_t)r * Hq * D + 4 * c) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float o[4][D / 16] = {}, m[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
    }
    const T *k = K + ((size_t)k0 * Hkv + kv) * D, *v = V + ((size_t)k0 * Hkv + kv) * D;
    for (int j0 = 0; j0 < keys; j0 += KT) {
        __syncthreads();
        for (int i = tid; i < KT * P; i += 256) {
            const int r = i / P, c = i % P;
            const bool in = j0 + r < lk;
            const size_t g = (size_t)(j0 + r) * Hkv * D + 4 * c;
            sK[at16(r, c, P)] = in ? load4(k + g) : make_float4(0.f, 0.f, 0.f, 0.f);
            sV[at16(r, c, P)] = in ? load4(v + g) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        __syncthreads();
        float s[4][4] = {};
#pragma unroll 4
        for (int c = 0; c < P; ++c) {
            float4 a[4], b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = sQ[at16(ty * 4 + i, c, P)];
#pragma unroll
            for (int j = 0; j < 4; ++j) b[j] = sK[at16(tx + 16 * j, c, P)];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][j] = fmaf(a[i].x, b[j].x, s[i][j]);
                    s[i][j] = fmaf(a[i].y, b[j].y, s[i][j]);
                    s[i][j] = fmaf(a[i].z, b[j].z, s[i][j]);
                    s[i][j] = fmaf(a[i].w, b[j].w, s[i][j]);
                }
        }
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
#pragma unroll
            for (int e = 0; e < D / 16; ++e) o[i][e] *= f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = exp2f(s[i][j] - ms);
                l[i] += p;
                const int r = ty * 4 + i, key = tx + 16 * j;
                ((float *)sP)[at16(r, key >> 2, KT / 4) * 4 + (key & 3)] = p;
            }
        }
        __syncwarp();  // a row's 16 threads are one half of a warp
#pragma unroll 4
        for (int c = 0; c < KT / 4; ++c) {
            float4 a[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = sP[at16(ty * 4 + i, c, KT / 4)];
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int e = 0; e < D / 64; ++e) {
                    const float4 b = sV[at16(4 * c + x, tx + 16 * e, P)];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float p = x == 0 ? a[i].x : x == 1 ? a[i].y : x == 2 ? a[i].z : a[i].w;
                        o[i][4 * e] = fmaf(p, b.x, o[i][4 * e]);
                        o[i][4 * e + 1] = fmaf(p, b.y, o[i][4 * e + 1]);
                        o[i][4 * e + 2] = fmaf(p, b.z, o[i][4 * e + 2]);
                        o[i][4 * e + 3] = fmaf(p, b.w, o[i][4 * e + 3]);
                    }
                }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float sum = l[i];
#pragma unroll
        for (int x = 1; x < 16; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        const int r = row0 + ty * 4 + i;
        if (r >= lq) continue;
        const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
        T *out = O + ((size_t)(q0 + r) * Hq + h) * D;
#pragma unroll
        for (int e = 0; e < D / 64; ++e)
            *(float4 *)(out + 4 * (tx + 16 * e)) = make_float4(o[i][4 * e] * inv, o[i][4 * e + 1] * inv,
                                                               o[i][4 * e + 2] * inv, o[i][4 * e + 3] * inv);
    }
}

template <typename T, int D>
cudaError_t launch_d(const PagedPlan &p, int n, int total_q, int total_k, const void *Q, const void *K, const void *V,
                     const int32_t *cu_q, const int32_t *cu_k, void *O, void *ws, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(k_prompt_simt<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         Simt<D>::BYTES);
    if (e != cudaSuccess) return e;
    dim3 grid(total_q / QT + n, p.cfg.Hq);
    k_prompt_simt<T, D><<<grid, 256, Simt<D>::BYTES, s>>>(
        (const T *)Q, (const T *)K, (const T *)V, cu_q, cu_k, (T *)O, n, total_q, total_k, p.cfg.Hq, p.cfg.Hkv,
        p.scale_log2, (unsigned long long *)pg_ptr(p, ws, kPgCounters));
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prompt_simt(const PagedPlan &p, int n, int total_q, int total_k, const void *Q, const void *K,
                               const void *V, const int32_t *cu_q, const int32_t *cu_k, void *O, void *ws,
                               cudaStream_t s) {
    if (p.cfg.d == 64) return launch_d<float, 64>(p, n, total_q, total_k, Q, K, V, cu_q, cu_k, O, ws, s);
    return launch_d<float, 128>(p, n, total_q, total_k, Q, K, V, cu_q, cu_k, O, ws, s);
}

}  // namespace mono
