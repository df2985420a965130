// experts.cuh -- what the experts' sub-layer shares (route.cu, product.cu,
// combine.cu): the launchers behind the entry points of experts.cu.
#pragma once

#include "sublayer.cuh"

namespace engram {

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 32;
constexpr int kScaleBlock = 128;        // values of a row, and rows of a weight, that share a scale

struct RouteArgs {
    engram_router r;
    int32_t type, tokens;
    const void *logits;
    int64_t stride;
    const float *bias;
    int32_t *ids;
    float *weights;
    int32_t *offsets, *pairs;           // null: no lists
    int32_t *ws;                        // [blocks][n_experts] counts
    int32_t sms;
};
size_t route_workspace_ints(int n_experts, int tokens);
cudaError_t launch_route(const RouteArgs &a, cudaStream_t s);

struct ProductArgs {
    const uint8_t *x;
    const void *x_scales;
    int64_t x_stride;
    int32_t x_fmt, rows;                // rows of x
    const uint8_t *w;
    const void *w_scales;
    int32_t w_fmt, E, N, K;
    const int32_t *offsets, *pairs;     // null: one matrix for all rows
    int32_t top_k, n_pairs;             // rows of the output
    bool glu;
    float limit;
    int32_t out_type;                   // element type, or the format of glu's scales
    void *out, *out_scales;
    int64_t out_stride;                 // elements
    int32_t sms;
    int *err;
};
cudaError_t launch_product(const ProductArgs &a, cudaStream_t s);

struct CombineArgs {
    const void *y, *add;
    const float *w;
    void *out;
    int64_t y_stride, add_stride, out_stride;
    int32_t y_type, add_type, out_type, tokens, top_k, dim;
    uint32_t blocks;                    // set by the launcher
};
cudaError_t launch_combine(CombineArgs a, cudaStream_t s);

}  // namespace engram
