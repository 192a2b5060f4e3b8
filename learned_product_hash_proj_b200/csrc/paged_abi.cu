// paged_abi.cu -- the C-ABI of the dense operators (packed prompts and the
// paged key/value cache): validation, workspace layout, entry points.
// Host code only.
#include <float.h>
#include <limits.h>
#include <math.h>
#include <stdlib.h>
#include <string.h>

#include <algorithm>
#include <initializer_list>

#include "paged.cuh"

using namespace mono;

namespace {

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

int cuda_status(cudaError_t e) { return e == cudaSuccess ? MONO_OK : MONO_ERR_CUDA; }

int validate(const mono_paged_config *c) {
    if (c->Hq < 1 || c->Hkv < 1 || c->Hq % c->Hkv != 0 || c->d < 1 || c->page < 1) return MONO_ERR_INVALID;
    if (c->pages < 1 || c->layers < 1 || c->rows < 0 || c->width < 0 || c->tokens < 0) return MONO_ERR_INVALID;
    if (c->dtype != MONO_F32 && c->dtype != MONO_BF16) return MONO_ERR_INVALID;
    if (!isfinite(c->scale) || c->scale < 0.0) return MONO_ERR_INVALID;
    // what this build implements
    if (c->scale > 1e30) return MONO_ERR_UNSUPPORTED;  // the kernels scale in fp32
    if (c->d != 64 && c->d != 128) return MONO_ERR_UNSUPPORTED;
    if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128) return MONO_ERR_UNSUPPORTED;
    if (c->Hq > 65535 || c->rows > kPagedMaxRows) return MONO_ERR_UNSUPPORTED;
    if ((long long)c->pages * c->Hkv > INT_MAX / c->page) return MONO_ERR_UNSUPPORTED;
    if ((long long)c->width * c->page > INT_MAX - 256) return MONO_ERR_UNSUPPORTED;
    if ((long long)c->Hkv * c->page * c->d * 4 > INT_MAX) return MONO_ERR_UNSUPPORTED;
    // key tiles of one call, counted in 32 bits
    if ((long long)c->rows * (((long long)c->width * c->page + 31) / 32) > INT_MAX) return MONO_ERR_UNSUPPORTED;
    if ((long long)c->tokens + 256ll * c->rows > INT_MAX) return MONO_ERR_UNSUPPORTED;
    return MONO_OK;
}

void layout(PagedPlan *p) {
    const mono_paged_config &c = p->cfg;
    const size_t rows = c.rows, pages = c.pages;
    size_t bytes[kPgN] = {};
    bytes[kPgCounters] = kCntN * 8;
    bytes[kPgMarks] = marks_bytes(c.pages);
    bytes[kPgFree] = pages * 4;
    bytes[kPgFresh] = rows * 4;
    bytes[kPgPairs] = std::max(rows, pages) * 8;
    bytes[kPgPrefix] = (rows + 1) * 4;
    bytes[kPgPartO] = (size_t)2 * kPagedMaxCtas * kPagedHeads * c.d * 4;
    bytes[kPgPartML] = (size_t)2 * kPagedMaxCtas * kPagedHeads * 8;
    bytes[kPgWork] = (((size_t)c.tokens << prompt_pack_log2(c)) / 128 + rows + 1) * 32;
    size_t off = 0;
    for (int r = 0; r < kPgN; ++r) {
        p->off[r] = off;
        off = (off + bytes[r] + 255) / 256 * 256;
    }
    p->ws_bytes = off;
}

int check_common(const mono_paged_plan_t *plan, const void *ws) {
    if (!plan) return MONO_ERR_NULL;
    if (!ws) return MONO_ERR_WORKSPACE;
    if (!aligned(ws, 256)) return MONO_ERR_ALIGN;
    return MONO_OK;
}

int check_ptrs(std::initializer_list<const void *> ptrs) {
    for (const void *q : ptrs) {
        if (!q) return MONO_ERR_NULL;
        if (!aligned(q, 16)) return MONO_ERR_ALIGN;
    }
    return MONO_OK;
}

// int32 arrays of lengths and ids: their own alignment is enough
int check_ints(std::initializer_list<const void *> ptrs) {
    for (const void *q : ptrs) {
        if (!q) return MONO_ERR_NULL;
        if (!aligned(q, 4)) return MONO_ERR_ALIGN;
    }
    return MONO_OK;
}

struct Range {
    const void *at;
    size_t bytes;
};
bool overlap(const Range &a, const Range &b) {
    const uintptr_t x = (uintptr_t)a.at, y = (uintptr_t)b.at;
    return a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes;
}
// whether something that a call writes overlaps something that it reads, or something else that it writes
bool overlap(std::initializer_list<Range> written, std::initializer_list<Range> read) {
    for (auto w = written.begin(); w != written.end(); ++w) {
        for (const Range &r : read)
            if (overlap(*w, r)) return true;
        for (auto x = w + 1; x != written.end(); ++x)
            if (overlap(*w, *x)) return true;
    }
    return false;
}

size_t pool_bytes(const PagedPlan &p) {
    const mono_paged_config &c = p.cfg;
    return (size_t)c.layers * c.pages * c.Hkv * c.page * c.d * p.es;
}

}  // namespace

extern "C" {

int mono_paged_plan(const mono_paged_config *cfg, mono_paged_plan_t **plan, size_t *workspace_bytes) {
    if (!cfg || !plan) return MONO_ERR_NULL;
    *plan = nullptr;
    const int v = validate(cfg);
    if (v != MONO_OK) return v;
    mono_paged_plan_s *ps = (mono_paged_plan_s *)calloc(1, sizeof(mono_paged_plan_s));
    if (!ps) return MONO_ERR_INVALID;
    PagedPlan &p = ps->p;
    p.cfg = *cfg;
    p.es = cfg->dtype == MONO_BF16 ? 2 : 4;
    const double scale = cfg->scale > 0.0 ? cfg->scale : 1.0 / sqrt((double)cfg->d);
    // (a scale that fp32 would round to 0 stays above it, so that a masked key's -inf times it is -inf; scores that fit
    // fp32 are then still all but equal)
    p.scale_log2 = std::max((float)(scale * 1.4426950408889634), FLT_TRUE_MIN);
    layout(&p);
    *plan = ps;
    if (workspace_bytes) *workspace_bytes = p.ws_bytes;
    return MONO_OK;
}

void mono_paged_plan_destroy(mono_paged_plan_t *plan) { free(plan); }

int mono_prompt_attend(const mono_paged_plan_t *plan, int n, int total_q, int total_k, const void *Q, const void *K,
                       const void *V, const int32_t *cu_q, const int32_t *cu_k, void *O, void *workspace,
                       void *stream) {
    int st = check_common(plan, workspace);
    if (st) return st;
    const PagedPlan &p = plan->p;
    if (n < 0 || n > p.cfg.rows || total_q < 0 || total_q > p.cfg.tokens || total_k < 0) return MONO_ERR_INVALID;
    if (n == 0 || total_q == 0) return MONO_OK;
    if ((st = check_ptrs({Q, O}))) return st;
    if (total_k > 0 && (st = check_ptrs({K, V}))) return st;
    if ((st = check_ints({cu_q, cu_k}))) return st;
    if (prompt_items(p.cfg, n, total_q) > INT_MAX / 16) return MONO_ERR_UNSUPPORTED;  // counted in 32 bits
    const size_t row = (size_t)p.cfg.d * p.es, out = total_q * (p.cfg.Hq * row), in = total_k * (p.cfg.Hkv * row);
    const size_t cu = ((size_t)n + 1) * 4;
    if (overlap({{O, out}, {workspace, p.ws_bytes}}, {{Q, out}, {K, in}, {V, in}, {cu_q, cu}, {cu_k, cu}}))
        return MONO_ERR_INVALID;
    const auto launch = p.cfg.dtype == MONO_BF16 ? launch_prompt_tc : launch_prompt_simt;
    return cuda_status(launch(p, n, total_q, total_k, Q, K, V, cu_q, cu_k, O, workspace,
                                          (cudaStream_t)stream));
}

int mono_paged_append(const mono_paged_plan_t *plan, int layer, int n, int total, const void *K, const void *V,
                      const int32_t *cu, const int32_t *table, const int32_t *lens, void *Kp, void *Vp,
                      void *workspace, void *stream) {
    int st = check_common(plan, workspace);
    if (st) return st;
    const PagedPlan &p = plan->p;
    if (layer < 0 || layer >= p.cfg.layers || n < 0 || n > p.cfg.rows || total < 0) return MONO_ERR_INVALID;
    if (n == 0 || total == 0) return MONO_OK;
    if ((st = check_ptrs({K, V, Kp, Vp}))) return st;
    if ((st = check_ints({cu, lens}))) return st;
    if (p.cfg.width > 0 && (st = check_ints({table}))) return st;
    const size_t pool = pool_bytes(p), in = total * ((size_t)p.cfg.Hkv * p.cfg.d * p.es);
    if (overlap({{Kp, pool}, {Vp, pool}, {workspace, p.ws_bytes}},
                {{K, in}, {V, in}, {cu, ((size_t)n + 1) * 4}, {table, (size_t)n * p.cfg.width * 4}, {lens, (size_t)n * 4}}))
        return MONO_ERR_INVALID;
    return cuda_status(launch_paged_append(p, layer, n, total, K, V, cu, table, lens, Kp, Vp, workspace,
                                           (cudaStream_t)stream));
}

int mono_paged_attend(const mono_paged_plan_t *plan, int layer, int n, const void *Q, const int32_t *table,
                      const int32_t *lens, const void *Kp, const void *Vp, void *O, void *workspace, void *stream) {
    int st = check_common(plan, workspace);
    if (st) return st;
    const PagedPlan &p = plan->p;
    if (layer < 0 || layer >= p.cfg.layers || n < 0 || n > p.cfg.rows) return MONO_ERR_INVALID;
    if (n == 0) return MONO_OK;
    if ((st = check_ptrs({Q, Kp, Vp, O}))) return st;
    if ((st = check_ints({lens}))) return st;
    if (p.cfg.width > 0 && (st = check_ints({table}))) return st;
    const size_t pool = pool_bytes(p), out = (size_t)n * p.cfg.Hq * p.cfg.d * p.es;
    if (overlap({{O, out}, {workspace, p.ws_bytes}},
                {{Q, out}, {Kp, pool}, {Vp, pool}, {table, (size_t)n * p.cfg.width * 4}, {lens, (size_t)n * 4}}))
        return MONO_ERR_INVALID;
    return cuda_status(launch_paged_attend(p, layer, n, Q, table, lens, Kp, Vp, O, workspace, (cudaStream_t)stream));
}

int mono_paged_update(const mono_paged_plan_t *plan, int n_in, const int32_t *table, const int32_t *lens, int n_out,
                      const int32_t *parents, const int32_t *grow, int32_t *table_out, int32_t *lens_out, void *Kp,
                      void *Vp, void *workspace, void *stream) {
    int st = check_common(plan, workspace);
    if (st) return st;
    const PagedPlan &p = plan->p;
    const mono_paged_config &c = p.cfg;
    if (n_in < 0 || n_in > c.rows || n_out < 0 || n_out > c.rows) return MONO_ERR_INVALID;
    if (n_out == 0) return MONO_OK;
    if ((st = check_ptrs({Kp, Vp}))) return st;
    if ((st = check_ints({parents, grow, lens_out}))) return st;
    if (n_in > 0 && (st = check_ints({lens}))) return st;
    if (c.width > 0 && (st = check_ints({table_out}))) return st;
    if (c.width > 0 && n_in > 0 && (st = check_ints({table}))) return st;
    const size_t row = (size_t)c.width * 4, in = n_in, out = n_out, pool = pool_bytes(p);
    if (overlap({{table_out, out * row}, {lens_out, out * 4}, {Kp, pool}, {Vp, pool}, {workspace, p.ws_bytes}},
                {{table, in * row}, {lens, in * 4}, {parents, out * 4}, {grow, out * 4}}))
        return MONO_ERR_INVALID;
    return cuda_status(launch_paged_update(p, n_in, table, lens, n_out, parents, grow, table_out, lens_out, Kp, Vp,
                                           workspace, (cudaStream_t)stream));
}

int mono_paged_compact(const mono_paged_plan_t *plan, int n, const int32_t *table, const int32_t *lens,
                       int32_t *table_out, void *Kp, void *Vp, void *workspace, void *stream) {
    int st = check_common(plan, workspace);
    if (st) return st;
    const PagedPlan &p = plan->p;
    if (n < 0 || n > p.cfg.rows) return MONO_ERR_INVALID;
    if (n == 0 || p.cfg.width == 0) return MONO_OK;
    if ((st = check_ptrs({Kp, Vp}))) return st;
    if ((st = check_ints({table, lens, table_out}))) return st;
    const size_t bytes = (size_t)n * p.cfg.width * 4, pool = pool_bytes(p);
    if (overlap({{table_out, bytes}, {Kp, pool}, {Vp, pool}, {workspace, p.ws_bytes}},
                {{table, bytes}, {lens, (size_t)n * 4}}))
        return MONO_ERR_INVALID;
    return cuda_status(launch_paged_compact(p, n, table, lens, table_out, Kp, Vp, workspace, (cudaStream_t)stream));
}

int mono_paged_stats(const mono_paged_plan_t *plan, void *workspace, void *stream, mono_paged_stats_t *out) {
    if (!out) return MONO_ERR_NULL;
    memset(out, 0, sizeof(*out));
    const int st = check_common(plan, workspace);
    if (st) return st;
    cudaStream_t s = (cudaStream_t)stream;
    unsigned long long cnt[kCntN];
    char *at = pg_ptr(plan->p, workspace, kPgCounters);
    if (cudaMemcpyAsync(cnt, at, sizeof(cnt), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaMemsetAsync(at + 8 * kPagedErr, 0, 8, s) != cudaSuccess || cudaStreamSynchronize(s) != cudaSuccess)
        return MONO_ERR_CUDA;
    out->device_error = (int32_t)cnt[kPagedErr];
    out->pages_held = (int32_t)cnt[kPagedHeld];
    out->pages_copied = (int32_t)cnt[kPagedCopied];
    out->pages_short = (int32_t)cnt[kPagedShort];
    return out->device_error ? MONO_ERR_DEVICE : MONO_OK;
}

}  // extern "C"
