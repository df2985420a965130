// experts.cu -- entry points of the experts' sub-layer (engram_route,
// engram_project_fp8, engram_glu_fp8, engram_combine): host-side validation
// before anything is enqueued.
#include "experts.cuh"

#include <cmath>

using namespace engram;

namespace {

inline cudaStream_t S(uintptr_t s) { return reinterpret_cast<cudaStream_t>(s); }
inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline int cuda_rc(cudaError_t e) {
    return e == cudaSuccess ? ENGRAM_OK : e == cudaErrorInvalidConfiguration ? ENGRAM_E_UNSUPPORTED : ENGRAM_E_CUDA;
}
inline bool is_type(int t) { return t >= ENGRAM_T_BF16 && t <= ENGRAM_T_F32; }
inline bool is_fp8(int f) { return f == ENGRAM_FMT_FP8 || f == ENGRAM_FMT_FP8_E8M0; }
inline size_t type_bytes(int t) { return t == ENGRAM_T_F32 ? 4 : 2; }
constexpr int64_t kMostStride = int64_t(1) << 39;

// A stride of 0 means dense; others must be a multiple of `unit`.
inline bool bad_stride(int64_t *stride, int64_t dense, int64_t unit) {
    if (*stride == 0) *stride = dense;
    return *stride < dense || *stride % unit || *stride >= kMostStride;
}

// Lists of a call; their pointers only where they are used.
int check_lists(const engram_expert_lists *l, int n_experts) {
    if (l->n_experts != n_experts || l->top_k < 1 || l->top_k > kMaxTopK || l->tokens < 0) return ENGRAM_E_INVALID;
    return (int64_t)l->tokens * l->top_k > 1 << 30 ? ENGRAM_E_INVALID : ENGRAM_OK;
}
int check_list_pointers(const engram_expert_lists *l, bool pairs) {
    if (!l->offsets || (pairs && !l->pairs)) return ENGRAM_E_NULL;
    return aligned(l->offsets, 4) && aligned(l->pairs, 4) ? ENGRAM_OK : ENGRAM_E_ALIGN;
}

// What the two products have in common; *none: nothing to do.
int check_product(const uint8_t *d_x, int64_t x_stride, const void *d_x_scales, int32_t x_fmt, int32_t rows,
                  const engram_fp8_weight *w, const engram_expert_lists *lists, bool glu, ProductArgs *a, bool *none) {
    *none = false;
    if (!w) return ENGRAM_E_NULL;
    if (!is_fp8(x_fmt) || !is_fp8(w->fmt) || (w->gated != 0) != glu) return ENGRAM_E_INVALID;
    if (w->n_experts < 1 || w->n_experts > kMaxExperts || w->n < 1 || w->n > 1 << 24 || w->k < 16 || w->k % 16 || w->k > 65536)
        return ENGRAM_E_INVALID;
    if ((int64_t)w->n * w->k * 2 >= kMostStride || rows < 0 || rows > 1 << 30) return ENGRAM_E_INVALID;
    if (bad_stride(&x_stride, w->k, 16)) return ENGRAM_E_INVALID;
    a->n_pairs = rows;
    a->top_k = 1;
    if (lists) {
        const int rc = check_lists(lists, w->n_experts);
        if (rc) return rc;
        a->top_k = lists->top_k;
        a->n_pairs = lists->tokens * lists->top_k;
        if (rows != (glu ? lists->tokens : a->n_pairs)) return ENGRAM_E_INVALID;
    } else if (w->n_experts != 1) {
        return ENGRAM_E_INVALID;
    }
    if (rows == 0) {
        *none = true;
        return ENGRAM_OK;
    }
    if (!d_x || !d_x_scales || !w->codes || !w->scales) return ENGRAM_E_NULL;
    if (!aligned(d_x, 16) || !aligned(w->codes, 16) || (x_fmt == ENGRAM_FMT_FP8 && !aligned(d_x_scales, 4)) ||
        (w->fmt == ENGRAM_FMT_FP8 && !aligned(w->scales, 4)))
        return ENGRAM_E_ALIGN;
    if (lists && glu && (int64_t)rows * (x_stride / 16) >= int64_t(1) << 32) return ENGRAM_E_UNSUPPORTED;   // gathered rows
    if (lists) {
        const int rc = check_list_pointers(lists, true);
        if (rc) return rc;
        a->offsets = lists->offsets;
        a->pairs = lists->pairs;
    }
    a->x = d_x;
    a->x_scales = d_x_scales;
    a->x_stride = x_stride;
    a->x_fmt = x_fmt;
    a->rows = rows;
    a->w = w->codes;
    a->w_scales = w->scales;
    a->w_fmt = w->fmt;
    a->E = w->n_experts;
    a->N = w->n;
    a->K = w->k;
    a->glu = glu;
    return ENGRAM_OK;
}

int device_of(ProductArgs *a) {
    if (!(a->sms = sm_count()) || !(a->err = error_word())) return ENGRAM_E_CUDA;
    return ENGRAM_OK;
}

}  // namespace

extern "C" {

size_t engram_route_workspace_bytes(int32_t n_experts, int32_t tokens) {
    return n_experts < 1 || n_experts > kMaxExperts || tokens < 0 ? 0 : route_workspace_ints(n_experts, tokens) * sizeof(int);
}

int engram_route(const engram_router *router, int32_t type, const void *d_logits, int64_t stride, const float *d_bias,
                 int32_t tokens, int32_t *d_ids, float *d_weights, const engram_expert_lists *lists, void *d_ws,
                 size_t ws_bytes, uintptr_t stream) {
    if (!router) return ENGRAM_E_NULL;
    const engram_router &r = *router;
    if (r.n_experts < 1 || r.n_experts > kMaxExperts || r.n_groups < 1 || r.n_groups > 32 || r.n_experts % r.n_groups ||
        r.top_groups < 1 || r.top_groups > r.n_groups || (r.group_best != 1 && r.group_best != 2))
        return ENGRAM_E_INVALID;
    if (r.top_k < 1 || r.top_k > kMaxTopK || r.top_k > r.top_groups * (r.n_experts / r.n_groups)) return ENGRAM_E_INVALID;
    if ((r.score != ENGRAM_SCORE_SIGMOID && r.score != ENGRAM_SCORE_SOFTMAX) || !std::isfinite(r.scale)) return ENGRAM_E_INVALID;
    if (!is_type(type) || tokens < 0 || (int64_t)tokens * r.top_k > 1 << 30 || bad_stride(&stride, r.n_experts, 1))
        return ENGRAM_E_INVALID;
    if (lists) {
        const int rc = check_lists(lists, r.n_experts);
        if (rc) return rc;
        if (lists->top_k != r.top_k || lists->tokens != tokens) return ENGRAM_E_INVALID;
    } else if (tokens == 0) {
        return ENGRAM_OK;
    }
    if (tokens && (!d_logits || !d_ids || !d_weights)) return ENGRAM_E_NULL;
    if (!aligned(d_logits, type_bytes(type)) || !aligned(d_bias, 4) || !aligned(d_ids, 4) || !aligned(d_weights, 4))
        return ENGRAM_E_ALIGN;
    RouteArgs a = {};
    if (lists) {
        const int rc = check_list_pointers(lists, tokens > 0);
        if (rc) return rc;
        const size_t need = engram_route_workspace_bytes(r.n_experts, tokens);
        if (need && !d_ws) return ENGRAM_E_NULL;
        if (ws_bytes < need) return ENGRAM_E_WORKSPACE;
        if (!aligned(d_ws, 4)) return ENGRAM_E_ALIGN;
        a.offsets = lists->offsets;
        a.pairs = lists->pairs;
        a.ws = static_cast<int32_t *>(d_ws);
    }
    a.r = r;
    a.type = type;
    a.tokens = tokens;
    a.logits = d_logits;
    a.stride = stride;
    a.bias = d_bias;
    a.ids = d_ids;
    a.weights = d_weights;
    return cuda_rc(launch_route(a, S(stream)));
}

int engram_project_fp8(const uint8_t *d_x, int64_t x_stride, const void *d_x_scales, int32_t x_fmt, int32_t rows,
                       const engram_fp8_weight *w, const engram_expert_lists *lists, int32_t out_type, void *d_out,
                       int64_t out_stride, uintptr_t stream) {
    ProductArgs a = {};
    bool none;
    if (!is_type(out_type)) return ENGRAM_E_INVALID;
    int rc = check_product(d_x, x_stride, d_x_scales, x_fmt, rows, w, lists, false, &a, &none);
    if (rc) return rc;
    if (bad_stride(&out_stride, w->n, 1)) return ENGRAM_E_INVALID;
    if (none) return ENGRAM_OK;
    if (!d_out) return ENGRAM_E_NULL;
    if (!aligned(d_out, type_bytes(out_type))) return ENGRAM_E_ALIGN;
    if ((rc = device_of(&a))) return rc;
    a.out_type = out_type;
    a.out = d_out;
    a.out_stride = out_stride;
    return cuda_rc(launch_product(a, S(stream)));
}

int engram_glu_fp8(const uint8_t *d_x, int64_t x_stride, const void *d_x_scales, int32_t x_fmt, int32_t rows,
                   const engram_fp8_weight *w, const engram_expert_lists *lists, float limit, int32_t out_fmt,
                   uint8_t *d_out, void *d_out_scales, uintptr_t stream) {
    ProductArgs a = {};
    bool none;
    if (!is_fp8(out_fmt) || !(limit >= 0.f) || !std::isfinite(limit)) return ENGRAM_E_INVALID;
    int rc = check_product(d_x, x_stride, d_x_scales, x_fmt, rows, w, lists, true, &a, &none);
    if (rc) return rc;
    if (w->n % 16) return ENGRAM_E_INVALID;
    if (none) return ENGRAM_OK;
    if (!d_out || !d_out_scales) return ENGRAM_E_NULL;
    if (!aligned(d_out, 16) || (out_fmt == ENGRAM_FMT_FP8 && !aligned(d_out_scales, 4))) return ENGRAM_E_ALIGN;
    if ((rc = device_of(&a))) return rc;
    a.limit = limit;
    a.out_type = out_fmt;
    a.out = d_out;
    a.out_scales = d_out_scales;
    a.out_stride = w->n;
    return cuda_rc(launch_product(a, S(stream)));
}

int engram_combine(const void *d_y, int32_t y_type, int64_t y_stride, const float *d_weights, int32_t tokens,
                   int32_t top_k, int32_t dim, const void *d_add, int32_t add_type, int64_t add_stride,
                   int32_t out_type, void *d_out, int64_t out_stride, uintptr_t stream) {
    if (!is_type(y_type) || !is_type(out_type) || (d_add && !is_type(add_type))) return ENGRAM_E_INVALID;
    if (tokens < 0 || top_k < 1 || top_k > kMaxTopK || dim < 8 || dim % 8 || dim > 65536 || (int64_t)tokens * top_k > 1 << 30)
        return ENGRAM_E_INVALID;
    if (bad_stride(&y_stride, dim, 8) || bad_stride(&out_stride, dim, 8) || (d_add && bad_stride(&add_stride, dim, 8)))
        return ENGRAM_E_INVALID;
    if (d_add && d_add == d_out && (add_type != out_type || add_stride != out_stride)) return ENGRAM_E_INVALID;
    if (tokens == 0) return ENGRAM_OK;
    if (!d_y || !d_weights || !d_out) return ENGRAM_E_NULL;
    if (!aligned(d_y, 16) || !aligned(d_add, 16) || !aligned(d_out, 16) || !aligned(d_weights, 4)) return ENGRAM_E_ALIGN;
    CombineArgs a;
    a.y = d_y;
    a.add = d_add;
    a.w = d_weights;
    a.out = d_out;
    a.y_stride = y_stride;
    a.add_stride = add_stride;
    a.out_stride = out_stride;
    a.y_type = y_type;
    a.add_type = add_type;
    a.out_type = out_type;
    a.tokens = tokens;
    a.top_k = top_k;
    a.dim = dim;
    return cuda_rc(launch_combine(a, S(stream)));
}

}  // extern "C"
