// sublayer.cuh -- what the attention sub-layer's kernels share (norm.cu,
// append.cu, attention.cu): element loads, the 8-bit block scale, the
// sequences of a call, and the launchers behind sublayer.cu's entry points.
#pragma once

#include "common.cuh"

namespace engram {

int *error_word();                  // the device error word (api.cu), null if it cannot be had
// Zeroes device memory that nothing uses yet (or any more) and waits for that alone (api.cu).  cudaMemset would queue it on the legacy stream: behind
// whatever that holds, and unordered with the non-blocking streams that use the memory next.
cudaError_t zero_now(void *p, size_t bytes);
int sm_count();                     // SMs of the current device (sublayer.cu), 0 if they cannot be had

// ---------------------------------------------------------------------------
// Eight consecutive elements (16-byte aligned) to f32 and back.
// ---------------------------------------------------------------------------
template <int TYPE>
__device__ __forceinline__ void load8(const void *p, int64_t i, float (&x)[8]) {
    if (TYPE == ENGRAM_T_F32) {
        const float4 *f = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
        const float4 a = f[0], b = f[1];
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    } else {
        const uint4 w = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (TYPE == ENGRAM_T_BF16) {
                x[2 * j] = bf16_lo(u[j]), x[2 * j + 1] = bf16_hi(u[j]);
            } else {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u[j]));
                x[2 * j] = f.x, x[2 * j + 1] = f.y;
            }
        }
    }
}

// Eight elements as they lie in memory.
template <int TYPE>
struct Raw8 {
    uint4 v[TYPE == ENGRAM_T_F32 ? 2 : 1];
    __device__ __forceinline__ void load(const void *p, int64_t i) {
        const uint4 *s = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p) + i * (TYPE == ENGRAM_T_F32 ? 4 : 2));
        v[0] = s[0];
        if (TYPE == ENGRAM_T_F32) v[sizeof(v) / 16 - 1] = s[1];
    }
    __device__ __forceinline__ void get(float (&x)[8]) const { load8<TYPE>(v, 0, x); }
};

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

template <int TYPE>
__device__ __forceinline__ void store8(void *p, int64_t i, const float (&x)[8]) {
    if (TYPE == ENGRAM_T_F32) {
        float4 *f = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
        f[0] = make_float4(x[0], x[1], x[2], x[3]);
        f[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        uint32_t u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            u[j] = TYPE == ENGRAM_T_BF16 ? pack_bf16x2(x[2 * j], x[2 * j + 1]) : pack_f16x2(x[2 * j], x[2 * j + 1]);
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + i) = make_uint4(u[0], u[1], u[2], u[3]);
    }
}

// ---------------------------------------------------------------------------
// 8-bit blocks
// ---------------------------------------------------------------------------
// The larger of m and |x|, |y|; a NaN among them stays.
__device__ __forceinline__ float amax3(float m, float x, float y) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(fabsf(x)), "f"(fabsf(y)));
    return r;
}
// The e8m0 byte of a block whose largest |value| has the f32 bits `amax`: the
// smallest 2^e with amax <= 448 2^e.  With amax = m 2^x, 1 <= m < 2, and 448 =
// 1.75 x 2^8, that is e = x - 8, one more when m > 1.75.  Infinities and NaN
// (their bits order above every number's) give 255; the least byte is 1.
__device__ __forceinline__ uint32_t block_scale_byte(uint32_t amax) {
    if (amax >= 0x7F800000u) return 255u;
    const int b = (int)(amax >> 23) - 8 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return b < 1 ? 1u : (uint32_t)b;
}
// 1 / 2^(byte - 127) for the bytes 1..254 (block_scale_byte gives up to 247, a caller's cache may hold more), exact: 2^-127,
// for 254, is subnormal.  0 for 255 (codes of a NaN block).
__device__ __forceinline__ float inv_scale(uint32_t byte) {
    return __uint_as_float(byte < 254u ? (254u - byte) << 23 : byte == 254u ? 0x00400000u : 0u);
}
// Four values times `inv` as e4m3 codes, nearest even.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}
// The codes of eight values of a block; zero for a NaN block.
__device__ __forceinline__ uint2 encode8(const float (&x)[8], uint32_t byte) {
    if (byte == 255u) return make_uint2(0u, 0u);
    const float s = inv_scale(byte);
    return make_uint2(e4m3x4(x[0] * s, x[1] * s, x[2] * s, x[3] * s), e4m3x4(x[4] * s, x[5] * s, x[6] * s, x[7] * s));
}
__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t codes) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(codes & 0xFFFFu), __NV_E4M3);
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// ---------------------------------------------------------------------------
// The sequences of a call
// ---------------------------------------------------------------------------
struct KvView {
    uint8_t *k, *v, *k_scales, *v_scales;
    int64_t page_stride;                // bytes between pages
    const int32_t *page_table, *kv_len, *row_start;
    int64_t table_stride;
    int32_t n_pages, KH, pt, pt_log2, D;
    int32_t batch, max_pages, rows, max_rows;
    int *err;
};

struct Seq {
    int row0, n, kv;                    // first row, rows, tokens
};

// Sequence b, checked (see engram_kv_batch): without rows or tokens where the arrays do not fit the call.
__device__ __forceinline__ Seq sequence(const KvView &c, int b) {
    Seq s;
    s.kv = c.kv_len[b];
    if (s.kv < 0 || (int64_t)s.kv > (int64_t)c.max_pages << c.pt_log2) {
        set_err(c.err, ENGRAM_E_LENGTH);
        s.kv = 0;
    }
    if (c.row_start) {
        s.row0 = c.row_start[b];
        const int end = c.row_start[b + 1];
        s.n = end - s.row0;
        if (s.row0 < 0 || end < s.row0 || end > c.rows || s.n > c.max_rows) {
            set_err(c.err, ENGRAM_E_LENGTH);
            s.row0 = s.n = 0;
        }
    } else {
        s.n = c.max_rows;
        s.row0 = b * s.n;
    }
    return s;
}

// The page of token p of sequence b, or -1 (and ENGRAM_E_PAGE) where its id is outside the cache.
__device__ __forceinline__ int page_of(const KvView &c, int b, int page) {
    const int id = c.page_table[(int64_t)b * c.table_stride + page];
    if ((uint32_t)id < (uint32_t)c.n_pages) return id;
    set_err(c.err, ENGRAM_E_PAGE);
    return -1;
}

// ---------------------------------------------------------------------------
// Launchers
// ---------------------------------------------------------------------------
struct NormArgs {
    const void *x, *res;
    void *res_out;
    const float *w;
    int64_t x_stride, res_stride;
    int32_t x_type, res_type, rows, dim, fmt, block;
    int32_t sms;
    float eps;
    void *out, *scales;
};
cudaError_t launch_residual_norm(const NormArgs &a, cudaStream_t s);

struct AppendArgs {
    KvView c;
    const void *k, *v, *q;
    void *q_out;
    int64_t k_stride, v_stride, q_stride, q_out_stride;
    int32_t type, H;
    const float *rope;
    int64_t rope_positions;
    int32_t rot, interleaved;
    int32_t span, slots, rows_per_block;    // set by the launcher
};
cudaError_t launch_kv_append(AppendArgs a, cudaStream_t s);

constexpr int kMaxSms = 160;            // what the joins' shared memory is sized for (GB300: 152)
// Workspace of the attention: two partial results a CTA and its arrival counters (one, on row tiles one a half).
struct AttnWorkspace {
    float *part;
    int *arrived;
};
size_t attn_part_floats(int sms);
size_t attn_counters(int sms);
struct AttnArgs {
    KvView c;
    AttnWorkspace ws;
    const void *q;
    void *out;
    float *lse;
    int64_t q_stride, out_stride;
    int32_t type, H, group, group_log2, window;     // group_log2 < 0: not a power of two
    float scale_log2;                   // scale x log2(e)
    int32_t sms;
};
cudaError_t launch_attention(const AttnArgs &a, cudaStream_t s);
// The same on tensor-core tiles (attn_tile.cu), and what it takes of the workspace.
cudaError_t launch_attn_tile(const AttnArgs &a, cudaStream_t s);
size_t attn_tile_part_floats(int sms);
size_t attn_tile_counters(int sms);

}  // namespace engram
