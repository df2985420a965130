// attn.cuh -- what the attention kernels share: the tensor maps of the cache,
// its reads as mma operands, the softmax in log2 units and the joining of
// partial results.
#pragma once

#include "sublayer.cuh"
#include "tcgen05.cuh"

namespace engram {
namespace attn {

// Value blocks with smaller scales (2^-66) count as zeros: the least exponent that
// joins the scores, so that a block of zeros (scale 2^-126) beside ordinary ones
// keeps its weight in the row's sum.
constexpr int kLeastValueByte = 61;

// 2^x by the hardware's ex2 (subnormal results are zero).
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The exponent that a value block's scale adds to the scores; NaN for a NaN block.
__device__ __forceinline__ float value_exp(uint32_t byte) {
    return byte == 255u ? __uint_as_float(0x7FC00000u) : (float)(max((int)byte, kLeastValueByte) - 127);
}

// 2^-value_exp(byte): takes the value scale out of the row's sum again.
__device__ __forceinline__ float value_unscale(uint32_t byte) {
    return inv_scale(max(byte, (uint32_t)kLeastValueByte));
}

// A query row of largest |element| bits m goes to f16 times the power of two
// `down` that brings it to [1, 2): exact but for elements under 2^-13 of the
// largest.  kf takes the scale back: scores in log2 units = kf 2^ek <q16, kc>.
__device__ __forceinline__ void q_scale(uint32_t m, float scale_log2, float &down, float &kf) {
    const int e = m == 0u || m >= 0x7F800000u ? 127 : (int)(m >> 23);
    down = e == 254 ? 5.877471754111438e-39f : __uint_as_float((uint32_t)(254 - e) << 23);   // 2^(127 - e)
    kf = scale_log2 * (e == 0 ? 5.877471754111438e-39f : __uint_as_float((uint32_t)e << 23));
}

// x / y of non-negative numbers, in 32 bits where both fit (several times faster).
__device__ __forceinline__ int64_t divide(int64_t x, int64_t y) {
    return ((x | y) >> 32) == 0 ? (int64_t)((uint32_t)x / (uint32_t)y) : x / y;
}

// The low / high two codes of a word as f16x2 (exact).
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t w) {
    uint32_t h;
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(h) : "r"(w));
    return h;
}
__device__ __forceinline__ uint32_t e4m3_hi(uint32_t w) {
    uint32_t h;
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, u;\n\t}" : "=r"(h) : "r"(w));
    return h;
}

// Shared-memory rows as the tensor maps place them: rows of 128 bytes with the
// 128-byte swizzle (16-byte chunk c of row r at c ^ (r & 7)), rows of 64 bytes
// with the 64-byte swizzle (chunk c at c ^ (r >> 1 & 3)).
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
    return D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}
__device__ __forceinline__ uint4 lds_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds_v2(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}
// Codes D/4 q .. D/4 q + D/4 - 1 of row r (conflict-free over a warp's (r = g, q)).
template <int D>
__device__ __forceinline__ void load_k_row(uint32_t ks, int r, int q, uint32_t (&w)[D / 16]) {
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
        const uint4 x = lds_v4(ks + chunk_at<D>(r, D / 64 * q + i));
        w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
    }
}
// Codes D/8 g .. D/8 g + D/8 - 1 of row r.
template <int D>
__device__ __forceinline__ void load_v_row(uint32_t vs, int r, int g, uint32_t (&w)[D / 32]) {
    if (D == 128) {
        const uint4 x = lds_v4(vs + chunk_at<D>(r, g));
        w[0] = x.x, w[1] = x.y, w[D / 32 - 2] = x.z, w[D / 32 - 1] = x.w;
    } else {
        const uint2 x = lds_v2(vs + chunk_at<D>(r, g >> 1) + 8 * (g & 1));
        w[0] = x.x, w[1] = x.y;
    }
}

// Bounded wait whose tests sleep until the phase completes or 20 us pass: many
// warps wait here at a time, and those that test in a loop slow the others down.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int *abort_flag, int *err) {
    return mbar_try(bar, parity) || mbar_wait(bar, parity, abort_flag, err, kWaitNs, 20000u);
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int w, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}

// Where float4 i of row r lies in a warp's sums (spreads the rows over the banks).
__device__ __forceinline__ int swz(int r, int i) { return i ^ (r >> 1 & 3); }

// Two query elements to f32.
template <int TYPE>
__device__ __forceinline__ float2 q_pair(uint32_t u) {
    return TYPE == ENGRAM_T_BF16 ? make_float2(bf16_lo(u), bf16_hi(u)) : __half22float2(*reinterpret_cast<const __half2 *>(&u));
}

// One more arrival at a counter: how many came before.  Releases what the block wrote before its last
// barrier and acquires what the others released.
__device__ __forceinline__ int arrive(int *counter) {
    int before;
    asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
    return before;
}

// Four output values of tile row rr (token rr / group, head rr % group) and, with the first, its lse.
template <int TYPE, int D>
__device__ __forceinline__ void store_row4(const AttnArgs &a, int row0, int head, int rr, int d4, const float4 &acc, float m,
                                           float l) {
    const int64_t row = row0 + rr / a.group;
    const int h = head * a.group + rr % a.group;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint2 w;
    if (TYPE == ENGRAM_T_BF16)
        w = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    else
        w = make_uint2(pack_f16x2(acc.x * inv, acc.y * inv), pack_f16x2(acc.z * inv, acc.w * inv));
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + row * a.out_stride + (int64_t)h * D + 4 * d4) = w;
    if (d4 == 0 && a.lse) a.lse[row * a.H + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// The cache's codes as a 4D map {head_dim, page_tokens, heads, pages}, boxes of `tokens` rows of one head.
inline bool make_cache_map(CUtensorMap *map, const KvView &c, const uint8_t *codes, int tokens) {
    const uint64_t dims[4] = {(uint64_t)c.D, (uint64_t)c.pt, (uint64_t)c.KH, (uint64_t)c.n_pages};
    const uint64_t strides[3] = {(uint64_t)c.D, (uint64_t)c.pt * c.D, (uint64_t)c.page_stride};
    return tcg::make_map_u8_4d(map, codes, dims, strides, (uint32_t)tokens);
}

}  // namespace attn
}  // namespace engram
