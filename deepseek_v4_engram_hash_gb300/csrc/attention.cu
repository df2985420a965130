// attention.cu -- causal attention over the paged 8-bit cache (engram_attention)
// for up to 16 query rows a key/value head (rows = new tokens x query heads that
// share the head): single tokens and a few tokens at once.
//
// Mathematics.  With a power-of-two scale 2^ek, 2^ev a (page, head) block and
// codes kc, vc, the scores in log2 units are s_j = <q, kc_j> 2^ek scale log2(e),
// and  out = sum_j 2^(s_j) 2^ev vc_j / sum_j 2^(s_j).  The value scale goes into
// the exponent: t_j = s_j + ev, p_j = 2^(t_j - M) with M a running bound of the
// row's t, out = sum p_j vc_j / L, L = sum p_j 2^-ev, so the f16 probabilities
// always hold the row's largest contributions with full precision, while L keeps the
// weight of a token whose p 2^-ev counts: of value scales up to 2^100 apart.  M is set 7 under the row's largest t so far, and moves (and the sums are
// rescaled) only when a t exceeds it by more than 15: until then p <= 2^15, which f16
// and the f32 sums hold.
//
// Bound by the cache's bytes, so what counts is instructions a byte.  The tokens are
// the M side of both products (m16n8k16 with f16 operands: S^T = K Q^T and
// O^T = V^T P^T), 8 query rows the N side: one mma covers 16 tokens x 8 rows, and
// codes become operands in registers (e4m3 to f16 is exact) once for all rows.
// A CTA takes a contiguous range of the call's (sequence, head, 128-token tile) list,
// with kEntryCost places more an entry (what joining the warps takes), cut evenly over the
// grid, so any mix of lengths keeps every SM busy; ranges that
// cut an entry leave partial results, which the last CTA to arrive joins in
// CTA order.  Inside a CTA each warp streams its own 32-token units through a
// private ring of TMA copies (one thread issues, the warp itself consumes: no
// barrier between warps) and keeps its own softmax state; the warps join through
// shared memory at the end of an entry.
#include "attn.cuh"

namespace engram {

namespace {

using namespace attn;

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kUnit = 32, kSub = 16;                 // tokens a warp step, in two parts of one page each
constexpr int kTile = kUnit * kWarps;                // tokens a CTA step
constexpr int kMaxRows = 16;
// CTAs an SM; one less for 9 to 16 rows, which need 248 registers (with 168 they spill: 32 sequences of 4 tokens, 4 query
// heads a key/value head, behind 4000: 57 against 68 us).
constexpr int kCtasPerSm = 3;
// Places of an entry in the list beside its tiles: 64 single tokens behind 500 to 8191 take 97.3 us, without 104.7.
constexpr int kEntryCost = 2;
constexpr uint32_t kNever = 0x7FFFFFFF;
// A row's bound M is set kRoom (log2) under its largest t so far, and t may pass M by kLazy: the probabilities go up to
// f16's 2^15, and one 2^-32 of the row's largest is still half of f16's least number.
constexpr float kRoom = 7.f, kLazy = 15.f;

struct FewParams {
    AttnArgs a;
    CUtensorMap mk, mv;
};

template <int D>
struct Few {
    static constexpr int kStages = 256 / D;          // 16 KB a warp
    static constexpr int kHalf = kUnit * D;          // bytes of a unit's keys (or values)
    static constexpr int kRing = kStages * 2 * kHalf;
    static constexpr int kRegion = kWarps * kRing;
    // behind the rings: bounds and sums of the warps, the copies' barriers, two flags
    static constexpr int oBars = kRegion + 2 * kWarps * kMaxRows * 4, oFlags = oBars + kWarps * kStages * 8;
    static constexpr size_t kSmem = 1024 + oFlags + 16;
    static_assert(kMaxRows * D * 4 <= kRing && kCtasPerSm * (kSmem + 1024) <= 227 * 1024, "shared memory");
    static_assert(kThreads * 16 + (kMaxRows * kCtasPerSm * kMaxSms + 2 * kMaxRows) * 4 <= kRegion, "factors of a join");
    static constexpr int kPart = kMaxRows * (D + 2); // floats of a partial result
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The transpose of an 8 x 8 matrix of f16 held two a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// A sequence's entries, one a head, each of `tiles` 128-token tiles from token lo; its rows see tokens from `first` on.
struct Plan {
    Seq s;
    int first, lo, tiles;
};
__device__ __forceinline__ Plan plan_of(const AttnArgs &a, int b) {
    Plan p;
    p.s = sequence(a.c, b);
    p.first = a.window ? max(0, p.s.kv - p.s.n - a.window + 1) : 0;
    p.lo = p.first / kUnit * kUnit;
    p.tiles = p.s.n == 0 ? 0 : max(1, (p.s.kv - p.lo + kTile - 1) / kTile);
    return p;
}

// An entry's places in the list; none for a sequence without rows.
__device__ __forceinline__ int64_t places_of(const Plan &p) { return p.tiles ? p.tiles + kEntryCost : 0; }

// Joins the n partial results of an entry ([row][D] values, then the bounds and the
// sums of kMaxRows rows; the first in slot 1 of CTA `first`, the others in slot 0 of
// theirs) and stores them.  The factors 2^(M_c - M) go through shared memory, then
// a thread adds up one float4 over every groups-th part, sixteen loads at a time,
// and the groups are added in order.
template <int TYPE, int D>
__device__ __forceinline__ void join_parts(const AttnArgs &a, int row0, int head, int n_rows, int64_t first, int n,
                                           uint8_t *smem) {
    constexpr int kPart = Few<D>::kPart, kAhead = 16;
    float *fac = reinterpret_cast<float *>(smem) + 4 * kThreads;         // [n_rows][n]
    float4 *sums = reinterpret_cast<float4 *>(smem);                     // [groups][items]
    float *row_m = fac + n_rows * n, *row_l = row_m + kMaxRows;
    const int tid = threadIdx.x, lane = tid & 31;
    auto at = [&](int c) { return a.ws.part + ((first + c) * 2 + (c == 0 ? 1 : 0)) * kPart; };
    const int items = n_rows * (D / 4), groups = items >= kThreads ? 1 : kThreads / items;
    const int grp = groups > 1 ? tid / items : 0;
    float4 x[kAhead];
    auto load = [&](int i, int c0) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            x[j] = __ldcg(reinterpret_cast<const float4 *>(at(min(c0 + j * groups, n - 1))) + min(i, items - 1));
    };
    int i = groups > 1 ? tid % items : tid;
    load(i, grp);                                                        // beside the factors
    for (int r = tid >> 5; r < n_rows; r += kWarps) {
        float m = -INFINITY, l = 0.f, mc = -INFINITY, lc = 0.f;
        if (lane < n) mc = __ldcg(at(lane) + kMaxRows * D + r), lc = __ldcg(at(lane) + kMaxRows * D + kMaxRows + r);
        m = mc;
        for (int c = lane + 32; c < n; c += 32) m = fmaxf(m, __ldcg(at(c) + kMaxRows * D + r));
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        for (int c = lane; c < n; c += 32) {
            if (c != lane) mc = __ldcg(at(c) + kMaxRows * D + r), lc = __ldcg(at(c) + kMaxRows * D + kMaxRows + r);
            const float f = mc == -INFINITY ? (lc == 0.f ? 0.f : 1.f) : exp2_approx(mc - m);
            fac[r * n + c] = f;
            l = fmaf(lc, f, l);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
        if (lane == 0) row_m[r] = m, row_l[r] = l;
    }
    __syncthreads();
    for (int i0 = 0; i0 < items; i0 += kThreads, i += kThreads) {
        const int r = i / (D / 4);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i0) load(i, grp);
        if (i < items && grp < groups) {
            for (int c0 = grp; c0 < n; c0 += kAhead * groups) {
                if (c0 != grp) load(i, c0);
#pragma unroll
                for (int j = 0; j < kAhead; ++j) {
                    const int c = c0 + j * groups;
                    const float f = c < n ? fac[r * n + c] : 0.f;
                    if (c < n) acc.x = fmaf(x[j].x, f, acc.x), acc.y = fmaf(x[j].y, f, acc.y), acc.z = fmaf(x[j].z, f, acc.z), acc.w = fmaf(x[j].w, f, acc.w);
                }
            }
        }
        if (groups > 1) {
            sums[tid] = acc;
            __syncthreads();
            if (grp == 0)
                for (int k = 1; k < groups; ++k) {
                    const float4 y = sums[k * items + i];
                    acc.x += y.x, acc.y += y.y, acc.z += y.z, acc.w += y.w;
                }
        }
        if (i < items && grp == 0) store_row4<TYPE, D>(a, row0, head, r, i % (D / 4), acc, row_m[r], row_l[r]);
    }
}

// NT: groups of 8 query rows.
template <int TYPE, int D, int NT>
__global__ void __launch_bounds__(kThreads, kCtasPerSm + 1 - NT) attn_few_kernel(const __grid_constant__ FewParams p) {
    using F = Few<D>;
    constexpr int KS = D / 16;                       // k steps of K Q^T, and 16-dim tiles of V^T P^T
    extern __shared__ uint8_t smem_raw[];
    const AttnArgs &a = p.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q4 = lane & 3;
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw);
    const uint32_t ring = base + warp * F::kRing;
    float *stat = reinterpret_cast<float *>(smem + F::kRegion);          // [2][kWarps][kMaxRows]
    const uint32_t bars = smem_u32(smem + F::oBars) + warp * F::kStages * 8;
    int *flags = reinterpret_cast<int *>(smem + F::oFlags);
    volatile int *abort_flag = flags;
    if (tid == 0) flags[0] = 0;
    if (lane == 0) {
        for (int i = 0; i < F::kStages; ++i) mbar_init(bars + 8 * i, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncthreads();

    // this CTA's range of the list
    int b = 0;
    int64_t before = 0, total;
    Plan pl;
    const int lanes_per = (a.c.batch + 31) / 32;
    int64_t mine = 0, upto = 0;
    if (a.c.batch == 1) {
        pl = plan_of(a, 0);
        total = places_of(pl) * a.c.KH;
    } else {
        for (int j = 0; j < lanes_per; ++j) {
            const int i = lane * lanes_per + j;
            if (i < a.c.batch) mine += places_of(plan_of(a, i)) * a.c.KH;
        }
        upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xFFFFFFFFu, upto, o);
            if (lane >= o) upto += x;
        }
        total = __shfl_sync(0xFFFFFFFFu, upto, 31);
    }
    const int64_t per = max((int64_t)1, divide(total + gridDim.x - 1, gridDim.x));
    int64_t t = blockIdx.x * per;
    const int64_t end = min(total, t + per);
    if (t >= end) return;
    if (a.c.batch > 1) {
        const int owner = __ffs(__ballot_sync(0xFFFFFFFFu, t < upto)) - 1;
        b = owner * lanes_per;
        before = __shfl_sync(0xFFFFFFFFu, upto - mine, owner);
        pl = plan_of(a, b);
    }

    uint32_t phase = 0;                              // parity of each stage's next wait
    int stage = 0;
    while (t < end) {
        while (t >= before + places_of(pl) * a.c.KH && b + 1 < a.c.batch) {
            before += places_of(pl) * a.c.KH;
            pl = plan_of(a, ++b);
        }
        const int64_t rel = t - before;
        const int head = (int)divide(rel, places_of(pl));
        const int64_t tiles_t0 = before + head * places_of(pl) + kEntryCost, stop = min(end, tiles_t0 + pl.tiles);
        const int tile0 = (int)max((int64_t)0, t - tiles_t0), count = (int)max((int64_t)0, stop - max(t, tiles_t0));
        t = max(t + 1, stop);
        if (count == 0) continue;                     // no tile of the entry in the range

        const int tok0 = pl.lo + tile0 * kTile + warp * kUnit, tok1 = min(pl.s.kv, pl.lo + (tile0 + count) * kTile);
        const int units = tok0 < tok1 ? (tok1 - tok0 + kTile - 1) / kTile : 0;
        const int n_rows = min(8 * NT, pl.s.n * a.group);

        // pages and scales of 16 units at a time, one part a lane: id, key byte | value byte << 8.  A page that ends before
        // the first token that a row sees is not looked up: a sliding window's pages may have been given back.
        auto load_id = [&](int k) {
            const int tok = tok0 + (16 * k + (lane >> 1)) * kTile + (lane & 1) * kSub;
            return tok < tok1 && (tok | (a.c.pt - 1)) >= pl.first ? page_of(a.c, b, tok >> a.c.pt_log2) : -1;
        };
        auto load_scales = [&](int id) {
            if (id < 0) return 0u;
            const int64_t i = (int64_t)id * a.c.KH + head;
            return (uint32_t)a.c.k_scales[i] | (uint32_t)a.c.v_scales[i] << 8;
        };
        int id_cur = load_id(0), id_next = load_id(1);
        // the queries, asked for beside the page ids
        uint32_t raw_q[NT][D / 8];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = 8 * nt + g;
            const int64_t at = (int64_t)(pl.s.row0 + r / a.group) * a.q_stride + (int64_t)(head * a.group + r % a.group) * D + q4 * (D / 4);
            const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q) + at);
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
                const uint4 x = r < n_rows ? src[k] : make_uint4(0u, 0u, 0u, 0u);
                raw_q[nt][4 * k] = x.x, raw_q[nt][4 * k + 1] = x.y, raw_q[nt][4 * k + 2] = x.z, raw_q[nt][4 * k + 3] = x.w;
            }
        }
        auto issue = [&](int u, int st, int cur_block) {
            const int ids = (u >> 4) == cur_block ? id_cur : id_next;
            const int id0 = __shfl_sync(0xFFFFFFFFu, ids, 2 * (u & 15)), id1 = __shfl_sync(0xFFFFFFFFu, ids, 2 * (u & 15) + 1);
            if (lane == 0) {
                const int at = (tok0 + u * kTile) & (a.c.pt - 1);
                const int p0 = id0 < 0 ? a.c.n_pages : id0, p1 = id1 < 0 ? a.c.n_pages : id1;   // outside the cache: zeros
                const uint32_t dst = ring + st * 2 * F::kHalf, bar = bars + 8 * st;
                mbar_expect_tx(bar, 2 * F::kHalf);
                tma_load_4d(dst, &p.mk, 0, at, head, p0, bar);
                tma_load_4d(dst + F::kHalf, &p.mv, 0, at, head, p0, bar);
                if (a.c.pt == kSub) {
                    tma_load_4d(dst + F::kHalf / 2, &p.mk, 0, 0, head, p1, bar);
                    tma_load_4d(dst + F::kHalf + F::kHalf / 2, &p.mv, 0, 0, head, p1, bar);
                }
            }
        };
        for (int u = 0; u < min(units, F::kStages); ++u) issue(u, (stage + u) % F::kStages, 0);
        uint32_t sc_cur = load_scales(id_cur), sc_next = 0;

        // query row 8 nt + g, the lane's D / 4 dims, as f16 of about 1; bounds and factors of rows 8 nt + 2 q4 + e
        uint32_t qb[NT][KS][2];
        float kf[NT][2];
        int lim[NT][2], low[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            uint32_t m = 0;
#pragma unroll
            for (int k = 0; k < D / 8; ++k) {
                const float2 f = q_pair<TYPE>(raw_q[nt][k]);
                m = max(m, max(__float_as_uint(f.x) & 0x7FFFFFFFu, __float_as_uint(f.y) & 0x7FFFFFFFu));
            }
            m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
            m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
            float down, f;
            q_scale(m, a.scale_log2, down, f);
#pragma unroll
            for (int k = 0; k < D / 8; ++k) {
                const float2 x = q_pair<TYPE>(raw_q[nt][k]);
                qb[nt][k >> 1][k & 1] = pack_f16x2(x.x * down, x.y * down);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                kf[nt][e] = __shfl_sync(0xFFFFFFFFu, f, 4 * (2 * q4 + e));
                const int row = 8 * nt + 2 * q4 + e, pos = pl.s.kv - pl.s.n + row / a.group;
                lim[nt][e] = row < n_rows ? pos + 1 : (int)kNever;
                low[nt][e] = row < n_rows && a.window ? pos - a.window + 1 : 0;
            }
        }
        // tokens that every row sees
        const int first_pos = pl.s.kv - pl.s.n, last_pos = first_pos + (n_rows - 1) / a.group;
        const int all_lo = a.window ? last_pos - a.window + 1 : 0, all_hi = first_pos + 1;

        float o[NT][KS][4] = {};
        float M[NT][2], L[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)                                 // places without a row never ask for a rescaling
                M[nt][e] = 8 * nt + 2 * q4 + e < n_rows ? -INFINITY : INFINITY, L[nt][e] = 0.f;
#pragma unroll 1
        for (int u = 0; u < units; ++u) {
            const int tb = tok0 + u * kTile;
            if ((u & 15) == 0 && u) {
                id_cur = id_next;
                sc_cur = sc_next;
                id_next = load_id((u >> 4) + 1);
            }
            if ((u & 15) == 8) sc_next = load_scales(id_next);
            const int st = stage;
            stage = stage + 1 == F::kStages ? 0 : stage + 1;
            const bool here = wait_bar(bars + 8 * st, (phase >> st) & 1, abort_flag, a.c.err);
            phase ^= 1u << st;
            if (!__all_sync(0xFFFFFFFFu, here)) break;
            const uint32_t ks = ring + st * 2 * F::kHalf, vs = ks + F::kHalf;
            uint32_t sc[2];
            bool known[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                sc[h] = __shfl_sync(0xFFFFFFFFu, sc_cur, 2 * (u & 15) + h);
                known[h] = __shfl_sync(0xFFFFFFFFu, id_cur, 2 * (u & 15) + h) >= 0;
            }

            // scores of tokens g and g + 8 of a part (mma rows) and rows 2 q4, 2 q4 + 1; dims go to the k slots in the order of qb
            float s[2][NT][4] = {};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t w0[KS], w1[KS];
                load_k_row<D>(ks, kSub * h + g, q4, w0);
                load_k_row<D>(ks, kSub * h + g + 8, q4, w1);
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    const uint32_t a0 = e4m3_lo(w0[k]), a1 = e4m3_lo(w1[k]), a2 = e4m3_hi(w0[k]), a3 = e4m3_hi(w1[k]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma16816(s[h][nt], a0, a1, a2, a3, qb[nt][k][0], qb[nt][k][1]);
                }
            }
            bool over = false;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float ek = e8m0_to_f32(sc[h] & 255u), ev = value_exp(sc[h] >> 8);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[h][nt][e] = fmaf(s[h][nt][e], kf[nt][e & 1] * ek, ev);
            }
            if (!(tb >= all_lo && tb + kUnit <= all_hi && known[0] && known[1])) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int tok = tb + kSub * h + g + 8 * (e >> 1);
                            if (tok >= lim[nt][e & 1] || tok < low[nt][e & 1] || !known[h]) s[h][nt][e] = -INFINITY;
                        }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    over |= fmaxf(fmaxf(s[0][nt][e], s[0][nt][2 + e]), fmaxf(s[1][nt][e], s[1][nt][2 + e])) > M[nt][e] + kLazy;
            if (__any_sync(0xFFFFFFFFu, over)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float m = fmaxf(fmaxf(s[0][nt][e], s[0][nt][2 + e]), fmaxf(s[1][nt][e], s[1][nt][2 + e]));
                        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
                        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 8));
                        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 16));
                        m = fmaxf(m - kRoom, M[nt][e]);
                        const float f = M[nt][e] == m ? 1.f : exp2_approx(M[nt][e] - m);
                        M[nt][e] = m;
                        L[nt][e] *= f;
#pragma unroll
                        for (int k = 0; k < KS; ++k) o[nt][k][e] *= f, o[nt][k][2 + e] *= f;
                    }
            }
            uint32_t pb[2][NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float m0 = M[nt][0] == -INFINITY ? 0.f : M[nt][0], m1 = M[nt][1] == -INFINITY ? 0.f : M[nt][1];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float back = value_unscale(sc[h] >> 8);
                    const float x0 = exp2_approx(s[h][nt][0] - m0), x1 = exp2_approx(s[h][nt][1] - m1);
                    const float y0 = exp2_approx(s[h][nt][2] - m0), y1 = exp2_approx(s[h][nt][3] - m1);
                    L[nt][0] = fmaf(x0 + y0, back, L[nt][0]);
                    L[nt][1] = fmaf(x1 + y1, back, L[nt][1]);
                    pb[h][nt][0] = transpose8(pack_f16x2(x0, x1));      // row g, tokens 2 q4, 2 q4 + 1
                    pb[h][nt][1] = transpose8(pack_f16x2(y0, y1));      // and those + 8
                }
            }
            // out: mma rows g and g + 8 of tile i are the dims D / 8 g + 2 i and + 1, k slots the tokens 2 q4, 2 q4 + 1 (+ 8)
            const bool cut = tb + kUnit > pl.s.kv || tb < pl.first || (int)min(sc[0], sc[1]) >> 8 < kLeastValueByte;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                constexpr int VW = D / 32;                              // 32-bit words of a lane's dims
                uint32_t v[4][VW];
#pragma unroll
                for (int r = 0; r < 4; ++r) load_v_row<D>(vs, kSub * h + 2 * q4 + (r & 1) + 8 * (r >> 1), g, v[r]);
                if (cut) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int tok = tb + kSub * h + 2 * q4 + (r & 1) + 8 * (r >> 1);
                        if (tok >= pl.s.kv || tok < pl.first || (int)(sc[h] >> 8) < kLeastValueByte)
#pragma unroll
                            for (int i = 0; i < VW; ++i) v[r][i] = 0u;  // anything may be there, or it does not count
                    }
                }
#pragma unroll
                for (int i = 0; i < VW; ++i) {
                    const uint32_t a01 = __byte_perm(v[0][i], v[1][i], 0x5140), a23 = __byte_perm(v[0][i], v[1][i], 0x7362);
                    const uint32_t b01 = __byte_perm(v[2][i], v[3][i], 0x5140), b23 = __byte_perm(v[2][i], v[3][i], 0x7362);
                    const uint32_t a0 = e4m3_lo(a01), a1 = e4m3_hi(a01), a2 = e4m3_lo(b01), a3 = e4m3_hi(b01);
                    const uint32_t c0 = e4m3_lo(a23), c1 = e4m3_hi(a23), c2 = e4m3_lo(b23), c3 = e4m3_hi(b23);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma16816(o[nt][2 * i], a0, a1, a2, a3, pb[h][nt][0], pb[h][nt][1]);
                        mma16816(o[nt][2 * i + 1], c0, c1, c2, c3, pb[h][nt][0], pb[h][nt][1]);
                    }
                }
            }
            __syncwarp();                                               // the stage is read
            if (u + F::kStages < units) issue(u + F::kStages, st, u >> 4);
        }
        if (__syncthreads_or(*abort_flag)) break;                       // copies in flight are waited for below

        // join the warps: each leaves its sums in its own ring
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float l = L[nt][e];
                l += __shfl_xor_sync(0xFFFFFFFFu, l, 4);
                l += __shfl_xor_sync(0xFFFFFFFFu, l, 8);
                l += __shfl_xor_sync(0xFFFFFFFFu, l, 16);
                const int r = 8 * nt + 2 * q4 + e;
                if (r >= n_rows) continue;
                if (g == 0) stat[warp * kMaxRows + r] = M[nt][e], stat[(kWarps + warp) * kMaxRows + r] = l;
                float4 *dst = reinterpret_cast<float4 *>(smem + warp * F::kRing) + r * (D / 4);
#pragma unroll
                for (int i = 0; i < D / 32; ++i)                        // dims D / 8 g + 4 i ..
                    dst[swz(r, g * (D / 32) + i)] =
                        make_float4(o[nt][2 * i][e], o[nt][2 * i][2 + e], o[nt][2 * i + 1][e], o[nt][2 * i + 1][2 + e]);
            }
        __syncthreads();
        const int64_t first_cta = divide(tiles_t0, per), last_cta = divide(tiles_t0 + pl.tiles - 1, per);
        const bool alone = first_cta == last_cta;
        float *part = a.ws.part + ((int64_t)blockIdx.x * 2 + (blockIdx.x == first_cta ? 1 : 0)) * F::kPart;
        for (int i = tid; i < n_rows * (D / 4); i += kThreads) {
            const int r = i / (D / 4), d4 = i % (D / 4);
            float m = stat[r], l = 0.f;
#pragma unroll
            for (int w = 1; w < kWarps; ++w) m = fmaxf(m, stat[w * kMaxRows + r]);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float mw = stat[w * kMaxRows + r], lw = stat[(kWarps + w) * kMaxRows + r];
                const float f = mw == -INFINITY ? (lw == 0.f ? 0.f : 1.f) : exp2_approx(mw - m);
                const float4 x = reinterpret_cast<const float4 *>(smem + w * F::kRing)[r * (D / 4) + swz(r, d4)];
                l = fmaf(lw, f, l);
                acc.x = fmaf(x.x, f, acc.x), acc.y = fmaf(x.y, f, acc.y), acc.z = fmaf(x.z, f, acc.z), acc.w = fmaf(x.w, f, acc.w);
            }
            if (alone) {
                store_row4<TYPE, D>(a, pl.s.row0, head, r, d4, acc, m, l);
            } else {
                reinterpret_cast<float4 *>(part)[i] = acc;
                if (d4 == 0) part[kMaxRows * D + r] = m, part[kMaxRows * D + kMaxRows + r] = l;
            }
        }
        if (!alone) {
            // the last CTA of the entry to arrive joins the partial results, in CTA order
            __syncthreads();
            if (tid == 0) {
                const int n = (int)(last_cta - first_cta);
                const bool last = arrive(&a.ws.arrived[first_cta]) == n;
                if (last) a.ws.arrived[first_cta] = 0;
                flags[1] = last;
            }
            __syncthreads();
            if (flags[1]) join_parts<TYPE, D>(a, pl.s.row0, head, n_rows, first_cta, (int)(last_cta - first_cta) + 1, smem);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");    // the rings go back to the copies
        __syncthreads();
    }
    if (*abort_flag) {                                                  // leave no copy in flight behind
        const uint64_t t0 = now_ns();
        for (int i = 0; i < F::kStages; ++i)
            while (!mbar_try(bars + 8 * i, (phase >> i) & 1) && now_ns() - t0 < 10000000ull) {
            }
    }
}

template <int TYPE, int D, int NT>
cudaError_t launch_few(const AttnArgs &a, cudaStream_t s) {
    FewParams p;
    p.a = a;
    const int box = a.c.pt < kUnit ? a.c.pt : kUnit;
    if (!make_cache_map(&p.mk, a.c, a.c.k, box) || !make_cache_map(&p.mv, a.c, a.c.v, box)) return cudaErrorInvalidValue;
    int dev = 0;
    cudaGetDevice(&dev);
    static bool attr[64] = {};
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(attn_few_kernel<TYPE, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)Few<D>::kSmem);
        if (e != cudaSuccess) return e;
        attr[dev] = true;
    }
    attn_few_kernel<TYPE, D, NT><<<a.sms * (kCtasPerSm + 1 - NT), kThreads, Few<D>::kSmem, s>>>(p);
    return cudaGetLastError();
}

template <int TYPE, int D>
cudaError_t launch_rows(const AttnArgs &a, cudaStream_t s) {
    return a.c.max_rows * a.group <= 8 ? launch_few<TYPE, D, 1>(a, s) : launch_few<TYPE, D, 2>(a, s);
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
    if ((int64_t)a.c.max_rows * a.group > kMaxRows) return launch_attn_tile(a, s);
    const bool bf = a.type == ENGRAM_T_BF16;
    if (a.c.D == 128) return bf ? launch_rows<ENGRAM_T_BF16, 128>(a, s) : launch_rows<ENGRAM_T_F16, 128>(a, s);
    return bf ? launch_rows<ENGRAM_T_BF16, 64>(a, s) : launch_rows<ENGRAM_T_F16, 64>(a, s);
}

}  // namespace engram
