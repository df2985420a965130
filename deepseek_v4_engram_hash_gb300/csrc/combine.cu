// combine.cu -- out[t] = sum_j w[t, j] y[t k + j] (+ add[t]), the experts' outputs
// back to their tokens (engram_combine).
//
// Memory bound: a thread takes 8 consecutive elements of a token and asks for
// the rows of 8 choices (4 of 32-bit ones) before it adds the first.  What counts is the bytes in flight: 4096 x 8 rows of
// 4096 in bf16, 302 MB, take 45.1 us (0.98 of the measured copy rate) with 8 blocks of 128 threads an SM at 64 registers, 49.3
// with 6, 51.9 with what 80 registers allow, 47.6 with 10 blocks, which spill.
#include "experts.cuh"

namespace engram {

namespace {

constexpr int kThreads = 128, kBlocks = 8;             // blocks an SM at least

// Waits for the kernel before it (a programmatic dependent launch) where it first reads.
template <int YT>
__global__ void __launch_bounds__(kThreads, kBlocks) combine_kernel(const CombineArgs a) {
    const unsigned token = blockIdx.x / a.blocks;    // blocks: of a token
    const int64_t t = token;
    const int c = (int)((blockIdx.x - token * a.blocks) * blockDim.x + threadIdx.x) * 8;
    if (c >= a.dim) return;
    const float *w = a.w + t * a.top_k;
    float s[8] = {};
    griddep_wait();
    constexpr int kRows = YT == ENGRAM_T_F32 ? 4 : 8;
    for (int j0 = 0; j0 < a.top_k; j0 += kRows) {
        Raw8<YT> raw[kRows];
        float f[kRows];
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
            f[j] = j0 + j < a.top_k ? w[j0 + j] : 0.f;
            if (f[j] != 0.f) raw[j].load(a.y, (t * a.top_k + j0 + j) * a.y_stride + c);
        }
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
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

cudaError_t launch_combine(CombineArgs a, cudaStream_t s) {
    const int chunks = a.dim >> 3, threads = chunks < kThreads ? (chunks + 31) / 32 * 32 : kThreads;
    a.blocks = (chunks + threads - 1) / threads;
    const int64_t blocks = (int64_t)a.tokens * a.blocks;
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = s;
    cudaLaunchAttribute la[1];
    la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    la[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = la;
    cfg.numAttrs = 1;
    switch (a.y_type) {
        case ENGRAM_T_BF16: return cudaLaunchKernelEx(&cfg, combine_kernel<ENGRAM_T_BF16>, a);
        case ENGRAM_T_F16: return cudaLaunchKernelEx(&cfg, combine_kernel<ENGRAM_T_F16>, a);
        default: return cudaLaunchKernelEx(&cfg, combine_kernel<ENGRAM_T_F32>, a);
    }
}

}  // namespace engram
