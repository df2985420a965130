// combine.cu -- out[t] = sum_j w[t, j] y[t k + j] (+ add[t]), the experts' outputs
// back to their tokens (engram_combine).
//
// Memory bound: a thread takes 8 consecutive elements of a token and asks for
// the rows of up to 8 choices before it adds the first.
#include "experts.cuh"

namespace engram {

namespace {

constexpr int kThreads = 256;

template <int YT>
__global__ void __launch_bounds__(kThreads) combine_kernel(const CombineArgs a) {
    const int chunks = a.dim >> 3;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= (int64_t)a.tokens * chunks) return;
    const int64_t t = i / chunks;
    const int c = (int)(i - t * chunks) * 8;
    const float *w = a.w + t * a.top_k;
    float s[8] = {};
    for (int j0 = 0; j0 < a.top_k; j0 += 8) {
        Raw8<YT> raw[8];
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            f[j] = j0 + j < a.top_k ? w[j0 + j] : 0.f;
            if (f[j] != 0.f) raw[j].load(a.y, (t * a.top_k + j0 + j) * a.y_stride + c);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (f[j] == 0.f) continue;
            float y[8];
            raw[j].get(y);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] = fmaf(f[j], y[e], s[e]);
        }
    }
    if (a.add) {
        float y[8];
        const int64_t at = t * a.add_stride + c;
        if (a.add_type == ENGRAM_T_BF16)
            load8<ENGRAM_T_BF16>(a.add, at, y);
        else if (a.add_type == ENGRAM_T_F16)
            load8<ENGRAM_T_F16>(a.add, at, y);
        else
            load8<ENGRAM_T_F32>(a.add, at, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] += y[e];
    }
    const int64_t at = t * a.out_stride + c;
    if (a.out_type == ENGRAM_T_BF16)
        store8<ENGRAM_T_BF16>(a.out, at, s);
    else if (a.out_type == ENGRAM_T_F16)
        store8<ENGRAM_T_F16>(a.out, at, s);
    else
        store8<ENGRAM_T_F32>(a.out, at, s);
}

}  // namespace

cudaError_t launch_combine(const CombineArgs &a, cudaStream_t s) {
    const int64_t blocks = ((int64_t)a.tokens * (a.dim >> 3) + kThreads - 1) / kThreads;
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    switch (a.y_type) {
        case ENGRAM_T_BF16: combine_kernel<ENGRAM_T_BF16><<<(unsigned)blocks, kThreads, 0, s>>>(a); break;
        case ENGRAM_T_F16: combine_kernel<ENGRAM_T_F16><<<(unsigned)blocks, kThreads, 0, s>>>(a); break;
        default: combine_kernel<ENGRAM_T_F32><<<(unsigned)blocks, kThreads, 0, s>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace engram
