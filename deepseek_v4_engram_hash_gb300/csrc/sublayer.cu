// sublayer.cu -- entry points of the attention sub-layer (engram_residual_norm,
// engram_kv_append, engram_attention): host-side validation before anything is
// enqueued, and the attention's workspace.
#include "sublayer.cuh"

#include <cmath>
#include <new>

using namespace engram;

struct engram_attn {
    AttnWorkspace ws;
    int device, sms;
};

namespace {

inline cudaStream_t S(uintptr_t s) { return reinterpret_cast<cudaStream_t>(s); }
inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline int cuda_rc(cudaError_t e) { return e == cudaSuccess ? ENGRAM_OK : ENGRAM_E_CUDA; }

// SMs of the current device, 0 if they cannot be had.
inline int sm_count() {
    static int known[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    if (!known[dev]) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        known[dev] = n;
    }
    return known[dev];
}

// A stride of 0 means dense; others must keep every row 16-byte aligned.
inline int check_stride(int64_t *stride, int64_t dense) {
    if (*stride == 0) *stride = dense;
    return *stride < dense || *stride % 8 || *stride > (int64_t(1) << 40) ? ENGRAM_E_INVALID : ENGRAM_OK;
}

int check_kv(const engram_kv_cache *c, const engram_kv_batch *b, KvView *v) {
    if (!c || !b) return ENGRAM_E_NULL;
    if (c->head_dim != 64 && c->head_dim != 128) return ENGRAM_E_UNSUPPORTED;
    if (c->page_tokens != 16 && c->page_tokens != 32 && c->page_tokens != 64 && c->page_tokens != 128)
        return ENGRAM_E_UNSUPPORTED;
    if (c->n_kv_heads < 1 || c->n_kv_heads > 1024 || c->n_pages < 1 || c->n_pages > 0x7FFFFFFE) return ENGRAM_E_INVALID;
    const int64_t page = (int64_t)c->n_kv_heads * c->page_tokens * c->head_dim;
    v->page_stride = c->page_stride ? c->page_stride : page;
    if (v->page_stride < page || v->page_stride % 16 || v->page_stride >= (int64_t(1) << 40)) return ENGRAM_E_INVALID;
    if (b->batch < 1 || b->batch > 8192 || b->max_pages < 1 || b->rows < 0 || b->max_rows < 0) return ENGRAM_E_INVALID;
    if ((int64_t)b->max_pages * c->page_tokens > (int64_t(1) << 30) || b->rows > 1 << 30) return ENGRAM_E_INVALID;
    v->table_stride = b->table_stride ? b->table_stride : b->max_pages;
    if (v->table_stride < b->max_pages) return ENGRAM_E_INVALID;
    if (!b->row_start && (b->rows % b->batch || (b->max_rows && b->max_rows < b->rows / b->batch))) return ENGRAM_E_INVALID;
    if (b->row_start && b->rows && !b->max_rows) return ENGRAM_E_INVALID;
    if (b->rows == 0) return ENGRAM_OK;              // nothing to read or write
    if (!c->k || !c->v || !c->k_scales || !c->v_scales || !b->page_table || !b->kv_len) return ENGRAM_E_NULL;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(b->page_table, 4) || !aligned(b->kv_len, 4) ||
        !aligned(b->row_start, 4))
        return ENGRAM_E_ALIGN;
    v->k = c->k;
    v->v = c->v;
    v->k_scales = c->k_scales;
    v->v_scales = c->v_scales;
    v->page_table = b->page_table;
    v->kv_len = b->kv_len;
    v->row_start = b->row_start;
    v->n_pages = (int32_t)c->n_pages;
    v->KH = c->n_kv_heads;
    v->pt = c->page_tokens;
    v->pt_log2 = c->page_tokens == 16 ? 4 : c->page_tokens == 32 ? 5 : c->page_tokens == 64 ? 6 : 7;
    v->D = c->head_dim;
    v->batch = b->batch;
    v->max_pages = b->max_pages;
    v->rows = b->rows;
    v->max_rows = b->row_start ? (b->max_rows < b->rows ? b->max_rows : b->rows) : b->rows / b->batch;
    return ENGRAM_OK;
}

}  // namespace

extern "C" {

int engram_residual_norm(const void *d_x, int32_t x_type, int64_t x_stride, const void *d_res, int32_t res_type,
                         int64_t res_stride, void *d_res_out, const float *d_weight, int32_t rows, int32_t dim,
                         float eps, int32_t out_fmt, int32_t scale_block, void *d_out, void *d_scales,
                         uintptr_t stream) {
    if (x_type < ENGRAM_T_BF16 || x_type > ENGRAM_T_F32 || (res_type != ENGRAM_T_F32 && res_type != ENGRAM_T_BF16))
        return ENGRAM_E_INVALID;
    if (out_fmt != ENGRAM_FMT_BF16 && out_fmt != ENGRAM_FMT_FP8 && out_fmt != ENGRAM_FMT_FP8_E8M0) return ENGRAM_E_INVALID;
    if (rows < 0 || dim < 8 || dim % 8 || dim > 16384 || !(eps >= 0.f) || !std::isfinite(eps)) return ENGRAM_E_INVALID;
    const bool fp8 = out_fmt != ENGRAM_FMT_BF16;
    if (fp8 && (scale_block < 16 || scale_block % 16 || dim % scale_block)) return ENGRAM_E_INVALID;
    if (check_stride(&x_stride, dim) || check_stride(&res_stride, dim)) return ENGRAM_E_INVALID;
    if (rows == 0) return ENGRAM_OK;
    if (!d_res || !d_out || (fp8 && !d_scales)) return ENGRAM_E_NULL;
    if (!aligned(d_x, 16) || !aligned(d_res, 16) || !aligned(d_res_out, 16) || !aligned(d_weight, 16) ||
        !aligned(d_out, 16) || (out_fmt == ENGRAM_FMT_FP8 && !aligned(d_scales, 4)))
        return ENGRAM_E_ALIGN;
    NormArgs a;
    a.x = d_x;
    a.res = d_res;
    a.res_out = d_res_out;
    a.w = d_weight;
    a.x_stride = x_stride;
    a.res_stride = res_stride;
    a.x_type = x_type;
    a.res_type = res_type;
    a.rows = rows;
    a.dim = dim;
    a.fmt = out_fmt;
    a.block = fp8 ? scale_block : 16;
    a.eps = eps;
    a.out = d_out;
    a.scales = d_scales;
    if (!(a.sms = sm_count())) return ENGRAM_E_CUDA;
    return cuda_rc(launch_residual_norm(a, S(stream)));
}

int engram_kv_append(const engram_kv_cache *cache, const engram_kv_batch *batch, int32_t type, const void *d_k,
                     int64_t k_stride, const void *d_v, int64_t v_stride, const void *d_q, int64_t q_stride,
                     void *d_q_out, int64_t q_out_stride, int32_t n_heads, const engram_rope *rope,
                     uintptr_t stream) {
    AppendArgs a = {};
    const int rc = check_kv(cache, batch, &a.c);
    if (rc) return rc;
    if (type < ENGRAM_T_BF16 || type > ENGRAM_T_F32) return ENGRAM_E_INVALID;
    const int64_t kv_row = (int64_t)cache->n_kv_heads * cache->head_dim;
    if (check_stride(&k_stride, kv_row) || check_stride(&v_stride, kv_row)) return ENGRAM_E_INVALID;
    if (d_q) {
        if (n_heads < 1 || n_heads > 65536) return ENGRAM_E_INVALID;
        const int64_t q_row = (int64_t)n_heads * cache->head_dim;
        if (check_stride(&q_stride, q_row) || check_stride(&q_out_stride, q_row)) return ENGRAM_E_INVALID;
        if (d_q_out == d_q && q_out_stride != q_stride) return ENGRAM_E_INVALID;
    }
    const bool turn = rope && rope->dim > 0;
    if (rope && (rope->dim < 0 || rope->dim % 16 || rope->dim > cache->head_dim || rope->positions < 0))
        return ENGRAM_E_INVALID;
    if (batch->rows == 0) return ENGRAM_OK;
    if (!d_k || !d_v || (d_q && !d_q_out) || (turn && !rope->table)) return ENGRAM_E_NULL;
    if (!aligned(d_k, 16) || !aligned(d_v, 16) || !aligned(d_q, 16) || !aligned(d_q_out, 16) ||
        (turn && !aligned(rope->table, 16)))
        return ENGRAM_E_ALIGN;
    if (!(a.c.err = error_word())) return ENGRAM_E_CUDA;
    a.k = d_k;
    a.v = d_v;
    a.q = d_q;
    a.q_out = d_q_out;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_stride = q_stride;
    a.q_out_stride = q_out_stride;
    a.type = type;
    a.H = n_heads;
    a.rope = turn ? rope->table : nullptr;
    a.rope_positions = turn ? rope->positions : 0;
    a.rot = turn ? rope->dim : 0;
    a.interleaved = turn && rope->interleaved;
    const cudaError_t e = launch_kv_append(a, S(stream));
    return e == cudaErrorInvalidConfiguration ? ENGRAM_E_UNSUPPORTED : cuda_rc(e);
}

int engram_attn_create(engram_attn **out) {
    if (!out) return ENGRAM_E_NULL;
    *out = nullptr;
    engram_attn *h = new (std::nothrow) engram_attn();
    if (!h) return ENGRAM_E_CUDA;
    h->sms = sm_count();
    if (h->sms > kMaxSms) {
        delete h;
        return ENGRAM_E_UNSUPPORTED;
    }
    if (!h->sms || cudaGetDevice(&h->device) != cudaSuccess ||
        cudaMalloc(&h->ws.part, attn_part_floats(h->sms) * sizeof(float)) != cudaSuccess ||
        cudaMalloc(&h->ws.arrived, attn_counters(h->sms) * sizeof(int)) != cudaSuccess ||
        zero_now(h->ws.arrived, attn_counters(h->sms) * sizeof(int)) != cudaSuccess || !error_word()) {
        engram_attn_destroy(h);
        return ENGRAM_E_CUDA;
    }
    *out = h;
    return ENGRAM_OK;
}

int engram_attn_reset(engram_attn *a, uintptr_t stream) {
    if (!a) return ENGRAM_E_NULL;
    return cuda_rc(cudaMemsetAsync(a->ws.arrived, 0, attn_counters(a->sms) * sizeof(int), S(stream)));
}

void engram_attn_destroy(engram_attn *a) {
    if (!a) return;
    cudaFree(a->ws.part);
    cudaFree(a->ws.arrived);
    delete a;
}

int engram_attention(engram_attn *attn, const engram_kv_cache *cache, const engram_kv_batch *batch, int32_t type,
                     const void *d_q, int64_t q_stride, int32_t n_heads, float scale, int32_t window, void *d_out,
                     int64_t out_stride, float *d_lse, uintptr_t stream) {
    if (!attn) return ENGRAM_E_NULL;
    AttnArgs a = {};
    const int rc = check_kv(cache, batch, &a.c);
    if (rc) return rc;
    if ((type != ENGRAM_T_BF16 && type != ENGRAM_T_F16) || window < 0 || !std::isfinite(scale)) return ENGRAM_E_INVALID;
    if (n_heads < 1 || n_heads > 65536 || n_heads % cache->n_kv_heads) return ENGRAM_E_INVALID;
    const int64_t row = (int64_t)n_heads * cache->head_dim;
    if (check_stride(&q_stride, row) || check_stride(&out_stride, row)) return ENGRAM_E_INVALID;
    if ((int64_t)batch->rows * n_heads > 0x7FFFFFFF) return ENGRAM_E_UNSUPPORTED;
    if (batch->rows == 0) return ENGRAM_OK;
    if (!d_q || !d_out) return ENGRAM_E_NULL;
    if (!aligned(d_q, 16) || !aligned(d_out, 16) || !aligned(d_lse, 4)) return ENGRAM_E_ALIGN;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || !(a.c.err = error_word())) return ENGRAM_E_CUDA;
    if (dev != attn->device) return ENGRAM_E_INVALID;
    a.ws = attn->ws;
    a.q = d_q;
    a.out = d_out;
    a.lse = d_lse;
    a.q_stride = q_stride;
    a.out_stride = out_stride;
    a.type = type;
    a.H = n_heads;
    a.group = n_heads / cache->n_kv_heads;
    a.group_log2 = (a.group & (a.group - 1)) ? -1 : __builtin_ctz(a.group);
    a.window = window >= 1 << 30 ? 0 : window;          // no sequence is longer
    a.scale_log2 = (float)((double)scale * 1.4426950408889634);
    a.sms = attn->sms;
    return cuda_rc(launch_attention(a, S(stream)));
}

}  // extern "C"
