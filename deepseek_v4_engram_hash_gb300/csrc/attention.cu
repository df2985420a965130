// attention.cu -- causal attention over the paged 8-bit cache (engram_attention)
// for up to 16 query rows a key/value head and tile (rows = new tokens x query
// heads that share the head): single tokens and short chunks.
//
// Mathematics.  With a power-of-two scale 2^ek, 2^ev a (page, head) block and
// codes kc, vc, the scores in log2 units are s_j = <q, kc_j> 2^ek scale log2(e),
// and  out = sum_j 2^(s_j) 2^ev vc_j / sum_j 2^(s_j).  The value scale goes into
// the exponent: t_j = s_j + ev, p_j = 2^(t_j - M) with M a running bound of the
// row's t, out = sum p_j vc_j / L, L = sum p_j 2^-ev, so the f16 probabilities
// always hold the row's largest contributions with full precision, whatever
// the scales.  M moves (and the sums are rescaled) only when a t exceeds it by more
// than 8: until then p <= 2^8, which f16 and the f32 sums hold.
//
// Bound by the cache's bytes.  A CTA takes a contiguous range of the call's
// (sequence, head, row tile, 64-token tile) list, cut evenly over the grid, so any
// mix of lengths keeps every SM busy; ranges that cut a list entry leave partial results,
// which the last CTA to arrive joins in a fixed order.  Inside a CTA each warp
// streams its own 16-token units through a private ring of TMA copies (one
// thread issues, the warp itself consumes: no barrier between warps), turns codes
// into f16 mma operands in registers (e4m3 to f16 is exact) and keeps its own
// softmax state; four warps join through shared memory at the end of an entry.
#include "attn.cuh"

namespace engram {

namespace {

using namespace attn;

constexpr int kWarps = 4;
constexpr int kUnit = 16;                            // tokens a copy
constexpr int kTile = kUnit * kWarps;                // tokens a CTA step
constexpr int kRows = 16;
constexpr int kCtasPerSm = 3;
constexpr uint32_t kNever = 0x7FFFFFFF;

struct FewParams {
    AttnArgs a;
    CUtensorMap mk, mv;
};

template <int D>
struct Few {
    static constexpr int kStages = 512 / D;          // 16 KB a warp
    static constexpr int kHalf = kUnit * D;          // bytes of a unit's keys (or values)
    static constexpr int kRing = kStages * 2 * kHalf;
    static constexpr int kRegion = kWarps * kRing;
    static constexpr size_t kSmem = 1024 + kRegion + 1024;
    static constexpr int kPart = kRows * (D + 2);    // floats of a partial result
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// List entries of a sequence: row tiles x heads, each of `tiles` 64-token tiles from token lo.
struct Plan {
    Seq s;
    int lo, tiles, row_tiles;
};
__device__ __forceinline__ Plan plan_of(const AttnArgs &a, int b) {
    Plan p;
    p.s = sequence(a.c, b);
    p.row_tiles = (p.s.n * a.group + kRows - 1) / kRows;
    p.lo = a.window ? max(0, p.s.kv - p.s.n - a.window + 1) / kTile * kTile : 0;
    p.tiles = max(1, (p.s.kv - p.lo + kTile - 1) / kTile);
    return p;
}
__device__ __forceinline__ int64_t tiles_of(const AttnArgs &a, int b) {
    const Plan p = plan_of(a, b);
    return (int64_t)p.row_tiles * a.c.KH * p.tiles;
}

template <int TYPE, int D>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm) attn_few_kernel(const __grid_constant__ FewParams p) {
    using F = Few<D>;
    constexpr int KS = D / 16;                       // mma k steps of q k, and n tiles of p v over 2
    extern __shared__ uint8_t smem_raw[];
    const AttnArgs &a = p.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q4 = lane & 3;
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw);
    const uint32_t ring = base + warp * F::kRing;
    float *stat = reinterpret_cast<float *>(smem + F::kRegion);          // [2][kWarps][kRows]
    const uint32_t bars = smem_u32(smem + F::kRegion + 512) + warp * F::kStages * 8;
    int *flags = reinterpret_cast<int *>(smem + F::kRegion + 512 + kWarps * F::kStages * 8);
    volatile int *abort_flag = flags;
    if (tid == 0) flags[0] = 0;
    if (lane == 0) {
        for (int i = 0; i < F::kStages; ++i) mbar_init(bars + 8 * i, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncthreads();

    // this CTA's range of the list
    const int lanes_per = (a.c.batch + 31) / 32;
    int64_t mine = 0;
    for (int j = 0; j < lanes_per; ++j) {
        const int b = lane * lanes_per + j;
        if (b < a.c.batch) mine += tiles_of(a, b);
    }
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o) upto += x;
    }
    const int64_t total = __shfl_sync(0xFFFFFFFFu, upto, 31);
    const int64_t per = max((int64_t)1, (total + gridDim.x - 1) / gridDim.x);
    int64_t t = blockIdx.x * per;
    const int64_t end = min(total, t + per);
    if (t >= end) return;
    const int owner = __ffs(__ballot_sync(0xFFFFFFFFu, t < upto)) - 1;
    int b = owner * lanes_per;
    int64_t before = __shfl_sync(0xFFFFFFFFu, upto - mine, owner);
    Plan pl = plan_of(a, b);
    int64_t mine_b = (int64_t)pl.row_tiles * a.c.KH * pl.tiles;

    uint32_t phase = 0;                              // parity of each stage's next wait
    int stage = 0;
    while (t < end) {
        while (t >= before + mine_b && b + 1 < a.c.batch) {
            before += mine_b;
            pl = plan_of(a, ++b);
            mine_b = (int64_t)pl.row_tiles * a.c.KH * pl.tiles;
        }
        const int64_t rel = t - before;
        const int entry = (int)(rel / pl.tiles), tile0 = (int)(rel % pl.tiles);
        const int count = (int)min((int64_t)(pl.tiles - tile0), end - t);
        const int head = entry / pl.row_tiles, r0 = entry % pl.row_tiles * kRows;
        const int64_t entry_t0 = t - tile0;
        t += count;

        const int tok0 = pl.lo + tile0 * kTile + warp * kUnit, tok1 = min(pl.s.kv, pl.lo + (tile0 + count) * kTile);
        const int units = tok0 < tok1 ? (tok1 - tok0 + kTile - 1) / kTile : 0;
        const int n_rows = min(kRows, pl.s.n * a.group - r0);

        // pages and scales of 32 units at a time, one a lane: id, key byte | value byte << 8
        auto load_id = [&](int k) {
            const int u = 32 * k + lane, tok = tok0 + u * kTile;
            return u < units ? page_of(a.c, b, tok >> a.c.pt_log2) : -1;
        };
        auto load_scales = [&](int id) {
            if (id < 0) return 0u;
            const int64_t i = (int64_t)id * a.c.KH + head;
            return (uint32_t)a.c.k_scales[i] | (uint32_t)a.c.v_scales[i] << 8;
        };
        int id_cur = load_id(0), id_next = load_id(1);
        auto issue = [&](int u, int cur_block) {
            const int mine_id = (u >> 5) == cur_block ? id_cur : id_next;
            const int id = __shfl_sync(0xFFFFFFFFu, mine_id, u & 31);
            if (lane == 0) {
                const int st = (stage + u) % F::kStages;
                const int tok = tok0 + u * kTile, at = tok & (a.c.pt - 1), page = id < 0 ? a.c.n_pages : id;
                const uint32_t dst = ring + st * 2 * F::kHalf, bar = bars + 8 * st;
                mbar_expect_tx(bar, 2 * F::kHalf);
                tma_load_4d(dst, &p.mk, 0, at, head, page, bar);       // a page outside the cache reads as zeros
                tma_load_4d(dst + F::kHalf, &p.mv, 0, at, head, page, bar);
            }
        };
        for (int u = 0; u < min(units, F::kStages); ++u) issue(u, 0);
        uint32_t sc_cur = load_scales(id_cur), sc_next = 0;

        // queries of rows g and g + 8, the thread's D / 4 dims, as f16 of about 1
        uint32_t qa[KS][4];
        float kf[2];
        int lim[2], low[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = r0 + g + 8 * h;
            const bool live = g + 8 * h < n_rows;
            const int i = r / a.group, pos = pl.s.kv - pl.s.n + i;
            lim[h] = live ? pos + 1 : (int)kNever;
            low[h] = live && a.window ? pos - a.window + 1 : 0;
            const int64_t at = (int64_t)(pl.s.row0 + i) * a.q_stride + (int64_t)(head * a.group + r % a.group) * D + q4 * (D / 4);
            float x[D / 4];
            uint32_t m = 0;
#pragma unroll
            for (int e = 0; e < D / 4; e += 8) {
                float y[8] = {};
                if (live) load8<TYPE>(a.q, at + e, y);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    x[e + k] = y[k];
                    m = max(m, __float_as_uint(y[k]) & 0x7FFFFFFFu);
                }
            }
            m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
            m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
            float down;
            q_scale(m, a.scale_log2, down, kf[h]);
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                qa[k][h] = pack_f16x2(x[4 * k] * down, x[4 * k + 1] * down);
                qa[k][2 + h] = pack_f16x2(x[4 * k + 2] * down, x[4 * k + 3] * down);
            }
        }
        // tokens that every row of the tile sees
        const int first_pos = pl.s.kv - pl.s.n + r0 / a.group, last_pos = pl.s.kv - pl.s.n + (r0 + n_rows - 1) / a.group;
        const int all_lo = a.window ? last_pos - a.window + 1 : 0, all_hi = first_pos + 1;

        float o[2 * KS][4] = {};
        float M[2] = {-INFINITY, -INFINITY}, L[2] = {};
#pragma unroll 1
        for (int u = 0; u < units; ++u) {
            const int tb = tok0 + u * kTile;
            if ((u & 31) == 0 && u) {
                id_cur = id_next;
                sc_cur = sc_next;
                id_next = load_id((u >> 5) + 1);
            }
            if ((u & 31) == 16) sc_next = load_scales(id_next);
            const int st = (stage + u) % F::kStages;
            const bool here = wait_bar(bars + 8 * st, (phase >> st) & 1, abort_flag, a.c.err);
            phase ^= 1u << st;
            if (!__all_sync(0xFFFFFFFFu, here)) break;
            const uint32_t ks = ring + st * 2 * F::kHalf, vs = ks + F::kHalf;
            const uint32_t sc = __shfl_sync(0xFFFFFFFFu, sc_cur, u & 31);
            const int id = __shfl_sync(0xFFFFFFFFu, id_cur, u & 31);

            // scores: token n of the mma is row g of the unit's half; its dims go to the k slots in the order of qa
            float s[2][4] = {};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint32_t w[KS];
                load_k_row<D>(ks, 8 * j + g, q4, w);
#pragma unroll
                for (int k = 0; k < KS; ++k)
                    mma16816(s[j], qa[k][0], qa[k][1], qa[k][2], qa[k][3], e4m3_lo(w[k]), e4m3_hi(w[k]));
            }
            const float ek = e8m0_to_f32(sc & 255u), ev = value_exp(sc >> 8);
            const float c0 = kf[0] * ek, c1 = kf[1] * ek;
            float tmax0 = -INFINITY, tmax1 = -INFINITY;
            const bool whole = tb >= all_lo && tb + kUnit <= all_hi && id >= 0;
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float t0 = fmaf(s[j][e], c0, ev), t1 = fmaf(s[j][2 + e], c1, ev);
                    if (!whole) {
                        const int tok = tb + 8 * j + 2 * q4 + e;
                        if (tok >= lim[0] || tok < low[0] || id < 0) t0 = -INFINITY;
                        if (tok >= lim[1] || tok < low[1] || id < 0) t1 = -INFINITY;
                    }
                    s[j][e] = t0, s[j][2 + e] = t1;
                    tmax0 = fmaxf(tmax0, t0), tmax1 = fmaxf(tmax1, t1);
                }
            if (__any_sync(0xFFFFFFFFu, tmax0 > M[0] + kLazy || tmax1 > M[1] + kLazy)) {
                tmax0 = fmaxf(tmax0, __shfl_xor_sync(0xFFFFFFFFu, tmax0, 1));
                tmax1 = fmaxf(tmax1, __shfl_xor_sync(0xFFFFFFFFu, tmax1, 1));
                tmax0 = fmaxf(tmax0, __shfl_xor_sync(0xFFFFFFFFu, tmax0, 2));
                tmax1 = fmaxf(tmax1, __shfl_xor_sync(0xFFFFFFFFu, tmax1, 2));
                const float n0 = fmaxf(M[0], tmax0), n1 = fmaxf(M[1], tmax1);
                const float f0 = M[0] == n0 ? 1.f : exp2_approx(M[0] - n0), f1 = M[1] == n1 ? 1.f : exp2_approx(M[1] - n1);
                M[0] = n0, M[1] = n1;
                L[0] *= f0, L[1] *= f1;
#pragma unroll
                for (int k = 0; k < 2 * KS; ++k) {
                    o[k][0] *= f0, o[k][1] *= f0;
                    o[k][2] *= f1, o[k][3] *= f1;
                }
            }
            const float m0 = M[0] == -INFINITY ? 0.f : M[0], m1 = M[1] == -INFINITY ? 0.f : M[1];
            const float back = value_unscale(sc >> 8);
            uint32_t pa[4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float x0 = exp2_approx(s[j][0] - m0), x1 = exp2_approx(s[j][1] - m0);
                const float y0 = exp2_approx(s[j][2] - m1), y1 = exp2_approx(s[j][3] - m1);
                L[0] = fmaf(x0 + x1, back, L[0]);
                L[1] = fmaf(y0 + y1, back, L[1]);
                pa[2 * j] = pack_f16x2(x0, x1);
                pa[2 * j + 1] = pack_f16x2(y0, y1);
            }
            // out: k slots are the unit's tokens 2q, 2q + 1 (and + 8), n = g the dims D / 8 g + j of n tile j
            {
                constexpr int VW = D / 32;                             // 32-bit words of a thread's dims
                uint32_t v[4][VW];
                const bool zero = (int)((sc >> 8) & 255u) < kLeastValueByte;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int tok = 2 * q4 + (r & 1) + 8 * (r >> 1);
                    load_v_row<D>(vs, tok, g, v[r]);
                    if (zero || tb + tok >= pl.s.kv)                   // nothing is written there, or it does not count
#pragma unroll
                        for (int i = 0; i < VW; ++i) v[r][i] = 0u;
                }
#pragma unroll
                for (int i = 0; i < VW; ++i) {
                    const uint32_t a01 = __byte_perm(v[0][i], v[1][i], 0x5140), a23 = __byte_perm(v[0][i], v[1][i], 0x7362);
                    const uint32_t b01 = __byte_perm(v[2][i], v[3][i], 0x5140), b23 = __byte_perm(v[2][i], v[3][i], 0x7362);
                    mma16816(o[4 * i + 0], pa[0], pa[1], pa[2], pa[3], e4m3_lo(a01), e4m3_lo(b01));
                    mma16816(o[4 * i + 1], pa[0], pa[1], pa[2], pa[3], e4m3_hi(a01), e4m3_hi(b01));
                    mma16816(o[4 * i + 2], pa[0], pa[1], pa[2], pa[3], e4m3_lo(a23), e4m3_lo(b23));
                    mma16816(o[4 * i + 3], pa[0], pa[1], pa[2], pa[3], e4m3_hi(a23), e4m3_hi(b23));
                }
            }
            __syncwarp();                                              // the stage is read
            if (u + F::kStages < units) issue(u + F::kStages, u >> 5);
        }
        stage = (stage + units) % F::kStages;
        if (__syncthreads_or(*abort_flag)) break;                      // copies in flight are waited for below

        // join the four warps: each leaves its sums in its own ring
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            L[h] += __shfl_xor_sync(0xFFFFFFFFu, L[h], 1);
            L[h] += __shfl_xor_sync(0xFFFFFFFFu, L[h], 2);
            const int r = g + 8 * h;
            if (r >= n_rows) continue;
            if (q4 == 0) stat[warp * kRows + r] = M[h], stat[(kWarps + warp) * kRows + r] = L[h];
            float4 *dst = reinterpret_cast<float4 *>(smem + warp * F::kRing) + r * (D / 4);
#pragma unroll
            for (int c = 0; c < 2; ++c)                               // dims D/4 q + D/8 c + 0 .. D/8 - 1
#pragma unroll
                for (int i = 0; i < D / 32; ++i)
                    dst[swz(r, 2 * q4 * (D / 32) + c * (D / 32) + i)] =
                        make_float4(o[4 * i][2 * h + c], o[4 * i + 1][2 * h + c], o[4 * i + 2][2 * h + c], o[4 * i + 3][2 * h + c]);
        }
        __syncthreads();
        const int64_t first_cta = entry_t0 / per, last_cta = (entry_t0 + pl.tiles - 1) / per;
        const bool alone = first_cta == last_cta;
        float *part = a.ws.part + ((int64_t)blockIdx.x * 2 + (blockIdx.x == first_cta ? 1 : 0)) * F::kPart;
        for (int i = tid; i < n_rows * (D / 4); i += kWarps * 32) {
            const int r = i / (D / 4), d4 = i % (D / 4);
            float m = stat[r], l = 0.f;
#pragma unroll
            for (int w = 1; w < kWarps; ++w) m = fmaxf(m, stat[w * kRows + r]);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float mw = stat[w * kRows + r], f = mw == -INFINITY ? 0.f : exp2_approx(mw - m);
                if (mw == -INFINITY && stat[(kWarps + w) * kRows + r] == 0.f) continue;
                const float4 x = reinterpret_cast<const float4 *>(smem + w * F::kRing)[r * (D / 4) + swz(r, d4)];
                l = fmaf(stat[(kWarps + w) * kRows + r], f, l);
                acc.x = fmaf(x.x, f, acc.x), acc.y = fmaf(x.y, f, acc.y), acc.z = fmaf(x.z, f, acc.z), acc.w = fmaf(x.w, f, acc.w);
            }
            if (alone) {
                store_row4<TYPE, D>(a, pl.s.row0, head, r0 + r, d4, acc, m, l);
            } else {
                reinterpret_cast<float4 *>(part)[i] = acc;
                if (d4 == 0) part[kRows * D + r] = m, part[kRows * D + kRows + r] = l;
            }
        }
        if (!alone) {
            // the last CTA of the entry to arrive joins the partial results, in CTA order
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const int n = (int)(last_cta - first_cta);
                const bool last = atomicAdd(&a.ws.arrived[first_cta], 1) == n;
                if (last) a.ws.arrived[first_cta] = 0;
                flags[1] = last;
                __threadfence();
            }
            __syncthreads();
            if (flags[1]) {
                for (int i = tid; i < n_rows * (D / 4); i += kWarps * 32) {
                    const int r = i / (D / 4);
                    float m = -INFINITY, l = 0.f;
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int64_t c = first_cta; c <= last_cta; ++c) {
                        const float *pc = a.ws.part + (c * 2 + (c == first_cta ? 1 : 0)) * F::kPart;
                        const float4 x = __ldcg(reinterpret_cast<const float4 *>(pc) + i);
                        join(m, l, acc, __ldcg(pc + kRows * D + r), __ldcg(pc + kRows * D + kRows + r), x);
                    }
                    store_row4<TYPE, D>(a, pl.s.row0, head, r0 + r, i % (D / 4), acc, m, l);
                }
            }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the rings go back to the copies
        __syncthreads();
    }
    if (*abort_flag) {                                                 // leave no copy in flight behind
        const uint64_t t0 = now_ns();
        for (int i = 0; i < F::kStages; ++i)
            while (!mbar_try(bars + 8 * i, (phase >> i) & 1) && now_ns() - t0 < 10000000ull) {
            }
    }
}

template <int TYPE, int D>
cudaError_t launch_few(const AttnArgs &a, cudaStream_t s) {
    FewParams p;
    p.a = a;
    if (!make_cache_map(&p.mk, a.c, a.c.k, kUnit) || !make_cache_map(&p.mv, a.c, a.c.v, kUnit)) return cudaErrorInvalidValue;
    int dev = 0;
    cudaGetDevice(&dev);
    static bool attr[64] = {};
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(attn_few_kernel<TYPE, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)Few<D>::kSmem);
        if (e != cudaSuccess) return e;
        attr[dev] = true;
    }
    attn_few_kernel<TYPE, D><<<a.sms * kCtasPerSm, kWarps * 32, Few<D>::kSmem, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

size_t attn_part_floats(int sms) {
    const size_t few = (size_t)sms * kCtasPerSm * 2 * Few<128>::kPart, tile = attn_tile_part_floats(sms);
    return few > tile ? few : tile;
}
size_t attn_counters(int sms) {
    const size_t few = (size_t)sms * kCtasPerSm, tile = attn_tile_counters(sms);
    return few > tile ? few : tile;
}

cudaError_t launch_attention(const AttnArgs &a, cudaStream_t s) {
    // rows of one key/value head and sequence: up to one 16-row mma tile, or the tensor cores' 128-row tiles
    if ((int64_t)a.c.max_rows * a.group > kRows) return launch_attn_tile(a, s);
    const bool bf = a.type == ENGRAM_T_BF16;
    if (a.c.D == 128) return bf ? launch_few<ENGRAM_T_BF16, 128>(a, s) : launch_few<ENGRAM_T_F16, 128>(a, s);
    return bf ? launch_few<ENGRAM_T_BF16, 64>(a, s) : launch_few<ENGRAM_T_F16, 64>(a, s);
}

}  // namespace engram
