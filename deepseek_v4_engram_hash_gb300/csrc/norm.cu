// norm.cu -- residual addition, root-mean-square norm and the 8-bit output in
// one pass: r = res + x, y = r rsqrt(mean r^2 + eps) w, y as bf16 or as e4m3
// codes with one power-of-two scale a block (engram_residual_norm).
//
// Memory bound (about 6 flop an element against 7 to 17 bytes): each element is
// read once and stays in registers between the two uses.  One CTA a row,
// thread t holding the 8-element chunks t, t + THREADS, ...; the sum of squares
// goes through shuffles and one shared-memory exchange, a block's largest |y|
// through shuffles where the block is a power-of-two number of chunks that fits
// a warp, through shared-memory maxima otherwise.
#include "sublayer.cuh"

namespace engram {

namespace {

constexpr int kMaxDim = 16384;

template <int XT, int RT, int THREADS, int NV>
__global__ void __launch_bounds__(THREADS) residual_norm_kernel(const NormArgs a) {
    __shared__ float part[THREADS / 32];
    __shared__ uint32_t amax[kMaxDim / 16];
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int chunks = a.dim >> 3;

    float r[NV][8];
    float ss = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = tid + v * THREADS;
        if (c < chunks) {
            load8<RT>(a.res, row * a.res_stride + 8 * c, r[v]);
            if (a.x) {
                float x[8];
                load8<XT>(a.x, row * a.x_stride + 8 * c, x);
#pragma unroll
                for (int e = 0; e < 8; ++e) r[v][e] += x[e];
            }
            if (a.res_out) store8<RT>(a.res_out, row * a.res_stride + 8 * c, r[v]);
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(r[v][e], r[v][e], ss);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) r[v][e] = 0.f;
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
    if (lane == 0) part[warp] = ss;
    const int bc = a.block >> 3;                                  // chunks a block
    const bool in_warp = a.fmt != ENGRAM_FMT_BF16 && bc <= 32 && (bc & (bc - 1)) == 0;
    if (a.fmt != ENGRAM_FMT_BF16 && !in_warp)
        for (int i = tid; i < a.dim / a.block; i += THREADS) amax[i] = 0u;
    __syncthreads();
    ss = part[0];
#pragma unroll
    for (int w = 1; w < THREADS / 32; ++w) ss += part[w];
    const float inv = 1.f / sqrtf(ss / (float)a.dim + a.eps);

#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = tid + v * THREADS;
        float w[8];
        if (a.w && c < chunks) {
            load8<ENGRAM_T_F32>(a.w, 8 * c, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) r[v][e] = r[v][e] * inv * w[e];
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) r[v][e] *= inv;
        }
    }
    if (a.fmt == ENGRAM_FMT_BF16) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = tid + v * THREADS;
            if (c < chunks) store8<ENGRAM_T_BF16>(a.out, row * a.dim + 8 * c, r[v]);
        }
        return;
    }
    uint32_t m[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        m[v] = 0u;
#pragma unroll
        for (int e = 0; e < 8; ++e) m[v] = max(m[v], __float_as_uint(r[v][e]) & 0x7FFFFFFFu);
    }
    if (in_warp) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
            for (int o = 1; o < bc; o <<= 1) m[v] = max(m[v], __shfl_xor_sync(0xFFFFFFFFu, m[v], o));
    } else {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = tid + v * THREADS;
            if (c < chunks) atomicMax(&amax[c / bc], m[v]);
        }
        __syncthreads();
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = tid + v * THREADS;
            if (c < chunks) m[v] = amax[c / bc];
        }
    }
    const int64_t blocks = a.dim / a.block;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = tid + v * THREADS;
        if (c >= chunks) continue;
        const uint32_t byte = block_scale_byte(m[v]);
        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.out) + row * a.dim + 8 * c) = encode8(r[v], byte);
        if (c % bc == 0) {
            const int64_t i = row * blocks + c / bc;
            if (a.fmt == ENGRAM_FMT_FP8_E8M0)
                static_cast<uint8_t *>(a.scales)[i] = (uint8_t)byte;
            else
                static_cast<float *>(a.scales)[i] = e8m0_to_f32(byte);
        }
    }
}

template <int XT, int RT>
cudaError_t launch_typed(const NormArgs &a, cudaStream_t s) {
    const int chunks = a.dim >> 3;
    if (chunks <= 128)
        residual_norm_kernel<XT, RT, 128, 1><<<a.rows, 128, 0, s>>>(a);
    else if (chunks <= 256)
        residual_norm_kernel<XT, RT, 256, 1><<<a.rows, 256, 0, s>>>(a);
    else if (chunks <= 512)
        residual_norm_kernel<XT, RT, 256, 2><<<a.rows, 256, 0, s>>>(a);
    else if (chunks <= 1024)
        residual_norm_kernel<XT, RT, 256, 4><<<a.rows, 256, 0, s>>>(a);
    else
        residual_norm_kernel<XT, RT, 512, 4><<<a.rows, 512, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_residual_norm(const NormArgs &a, cudaStream_t s) {
    const bool f32 = a.res_type == ENGRAM_T_F32;
    switch (a.x_type) {
        case ENGRAM_T_BF16:
            return f32 ? launch_typed<ENGRAM_T_BF16, ENGRAM_T_F32>(a, s) : launch_typed<ENGRAM_T_BF16, ENGRAM_T_BF16>(a, s);
        case ENGRAM_T_F16:
            return f32 ? launch_typed<ENGRAM_T_F16, ENGRAM_T_F32>(a, s) : launch_typed<ENGRAM_T_F16, ENGRAM_T_BF16>(a, s);
        default:
            return f32 ? launch_typed<ENGRAM_T_F32, ENGRAM_T_F32>(a, s) : launch_typed<ENGRAM_T_F32, ENGRAM_T_BF16>(a, s);
    }
}

}  // namespace engram
