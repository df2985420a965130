// norm.cu -- residual addition, root-mean-square norm and the 8-bit output in
// one pass: r = res + x, y = r rsqrt(mean r^2 + eps) w, y as bf16 or as e4m3
// codes with one power-of-two scale a block (engram_residual_norm).
//
// Memory bound (about 6 flop an element against 7 to 17 bytes): each element is
// read once and stays in registers between the two uses.  A block takes a row, thread t
// the 8-element chunks t, t + blockDim.x of it; other blocks' loads run beside a
// block's exchanges and stores.  (Blocks that go through several rows and ask for the
// next one ahead measured 118 against 115 us for 16384 x 4096, f32 residual: 109 us of bytes.)
// The sum of squares goes through shuffles and one shared-memory exchange, a block's
// largest |y| through shuffles where the block is a power-of-two number of
// chunks that fits a warp, through shared-memory maxima otherwise.
#include "sublayer.cuh"

namespace engram {

namespace {

constexpr int kMaxDim = 16384;

template <int XT, int RT, int NV>
__global__ void __launch_bounds__(1024, 2) residual_norm_kernel(const NormArgs a) {
    __shared__ float part[32];
    __shared__ uint32_t amax[kMaxDim / 16];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, threads = blockDim.x;
    const int chunks = a.dim >> 3;
    const int bc = a.block >> 3;                                  // chunks a block
    const bool codes = a.fmt != ENGRAM_FMT_BF16, in_warp = bc <= 32 && (bc & (bc - 1)) == 0;

    const int64_t row = blockIdx.x;
    float r[NV][8];
    float ss = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = tid + v * threads;
        if (c < chunks) {
            load8<RT>(a.res, row * a.res_stride + 8 * c, r[v]);
            if (a.x) {
                float x[8];
                load8<XT>(a.x, row * a.x_stride + 8 * c, x);
#pragma unroll
                for (int e = 0; e < 8; ++e) r[v][e] += x[e];
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) r[v][e] = 0.f;
        }
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = tid + v * threads;
        if (a.res_out && c < chunks) store8<RT>(a.res_out, row * a.res_stride + 8 * c, r[v]);
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(r[v][e], r[v][e], ss);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
    if (lane == 0) part[warp] = ss;
    if (codes && !in_warp)
        for (int i = tid; i < a.dim / a.block; i += threads) amax[i] = 0u;
    __syncthreads();
    ss = lane < threads >> 5 ? part[lane] : 0.f;
#pragma unroll
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
    const float inv = 1.f / sqrtf(ss / (float)a.dim + a.eps);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = tid + v * threads;
        if (a.w && c < chunks) {
            float w[8];
            load8<ENGRAM_T_F32>(a.w, 8 * c, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) r[v][e] = r[v][e] * inv * w[e];
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) r[v][e] *= inv;
        }
    }
    if (!codes) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = tid + v * threads;
            if (c < chunks) store8<ENGRAM_T_BF16>(a.out, row * a.dim + 8 * c, r[v]);
        }
    } else {
        uint32_t m[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float big = 0.f;
#pragma unroll
            for (int e = 0; e < 8; e += 2) big = amax3(big, r[v][e], r[v][e + 1]);
            m[v] = __float_as_uint(big);                          // ordered: numbers, infinity, NaN
        }
        if (in_warp) {
#pragma unroll
            for (int v = 0; v < NV; ++v)
                for (int o = 1; o < bc; o <<= 1) m[v] = max(m[v], __shfl_xor_sync(0xFFFFFFFFu, m[v], o));
        } else {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c = tid + v * threads;
                if (c < chunks) atomicMax(&amax[c / bc], m[v]);
            }
            __syncthreads();
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c = tid + v * threads;
                if (c < chunks) m[v] = amax[c / bc];
            }
        }
        const int64_t blocks = a.dim / a.block;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = tid + v * threads;
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
}

template <int XT, int RT>
cudaError_t launch_typed(const NormArgs &a, cudaStream_t s) {
    // Two chunks a thread keep more bytes in flight on an SM (16384 rows of 4096, 32-bit residual: 115 against 147
    // us; 1537 rows of 5120, 16-bit: 16.0 against 17.1); one a thread shortens the time of a row, which counts while
    // the rows do not fill the SMs (one row: 2.6 against 3.1 us).
    const int chunks = a.dim >> 3;
    const bool one = chunks <= 256 || (chunks <= 1024 && a.rows <= a.sms);
    const int threads = ((one ? chunks : (chunks + 1) / 2) + 31) / 32 * 32;
    if (one)
        residual_norm_kernel<XT, RT, 1><<<a.rows, threads, 0, s>>>(a);
    else
        residual_norm_kernel<XT, RT, 2><<<a.rows, threads, 0, s>>>(a);
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
