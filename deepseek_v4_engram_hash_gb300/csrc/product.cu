// product.cu -- products of e4m3 rows with e4m3 weights that have a scale for each
// block of 128 (engram_project_fp8), and the gated pair of them with an 8-bit
// output (engram_glu_fp8), dense or with a matrix an expert.
//
// out[r, n] = sum_b sx[r, b] sw[n / 128, b] sum_{k in block b} x[r, k] W[n, k].  The inner sum
// of 128 products is tcgen05.mma kind::f8f6f4 (products exact, f32 sums in tensor memory); the
// outer one is f32 FMAs in registers.  Weights are the M side of the MMA (two blocks of
// 128 rows: neighbours, or the gate's and the other's), rows of x the N side, so that one token
// costs the tensor cores N = 16 and a prompt N = 128 by the same code, and a thread that holds
// weight row m for all tokens writes neighbouring addresses beside its warp's others.
//
// Roles (11 warps):
//   warp 0       TMA: two 128 x 128 weight tiles a block, and the tile's rows of x in boxes of
//                16, or gathered four at a time by the lists;
//   warp 1       issues the MMAs;
//   warp 2       the factors sx sw of a block's rows, to shared memory;
//   warps 3..10  take a block's sums from tensor memory (two buffers) into their f32
//                accumulators; at the end of a tile they write it.  Warps 3..6 and 7..10 take
//                chunks of 16 rows in turn.
// A CTA an SM walks the list of (expert, weight rows, rows) tiles; an expert's row tiles stand side by side, so
// that its weights are read from DRAM once.  Where there are fewer tiles than SMs, a cluster shares a tile: each CTA takes a part of K, and
// their sums are added in CTA order through distributed shared memory (no atomics, no workspace).
// Every wait is bounded (2 s); on expiry ENGRAM_E_TIMEOUT is raised, every role leaves its loops and
// tensor memory is freed.
#include "experts.cuh"
#include "tcgen05.cuh"

namespace engram {

namespace {

using namespace tcg;

constexpr int kM = 128;                              // weight rows of an MMA, values of a K block
constexpr int kThreads = 352;
constexpr int kEpiWarps = 8;
constexpr uint32_t kTileA = kM * 128;                // bytes

template <int NT> struct Cfg {
    static constexpr uint32_t kStage = 2 * kTileA + NT * 128;
    static constexpr int kStages = NT == 128 ? 4 : 5;
    static constexpr int kFactors = kStages + 2;     // slots of [2][NT] f32
    static constexpr uint32_t oFactor = kStages * kStage;
    static constexpr uint32_t oCodes = oFactor + kFactors * 2 * NT * 4;   // glu: [2 groups][2][16][128] codes
    static constexpr uint32_t oMax = oCodes + 2 * 2 * 16 * 128;           // [2 groups][2][16][4] f32 bits
    static constexpr uint32_t oBar = oMax + 2 * 2 * 16 * 4 * 4;
    static constexpr uint32_t oFlag = oBar + 8 * (2 * kStages + 2 * kFactors + 4 + 1);
    static constexpr uint32_t oLists = oFlag + 16;                        // first [E], rows [E], tiles before [E + 1]
    static size_t bytes(int E) { return 1024 + oLists + (3 * (size_t)E + 1) * 4; }
    static constexpr int kChunks = NT / 32;          // chunks of 16 rows a group of warps
};

struct Params {
    ProductArgs a;
    CUtensorMap mw, mx;
    int KB, NB;                                      // blocks of K, of N
    int m_tiles;                                     // of an expert
    int split;                                       // CTAs that share a tile
    int group;                                       // row tiles side by side
};

struct TileAt {
    int e, row, n, m0;                               // expert, first row, rows, first weight row
};

__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t da, uint64_t db, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(da), "l"(db), "r"(idesc), "r"(accumulate)
        : "memory");
}
// kind::f8f6f4, e4m3 x e4m3 (formats 0), f32 sums, both K-major.
__device__ __forceinline__ uint32_t idesc_f8(int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(kM >> 4) << 24);
}
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tma_weights(uint32_t dst, const CUtensorMap *map, int k, int n, int part, int e, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(k), "r"(n), "r"(part), "r"(e), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap *map, int k, int row, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(k), "r"(row), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap *map, int k, const int (&row)[4], uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(k), "r"(row[0]), "r"(row[1]), "r"(row[2]), "r"(row[3]), "r"(bar)
        : "memory");
}
// 16 columns of this warp's 32 tensor-memory lanes (without the wait).
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&u)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
          "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// Uses of these registers stay behind the wait before it.
__device__ __forceinline__ void pin16(uint32_t (&u)[16]) {
    asm volatile(""
                 : "+r"(u[0]), "+r"(u[1]), "+r"(u[2]), "+r"(u[3]), "+r"(u[4]), "+r"(u[5]), "+r"(u[6]), "+r"(u[7]),
                   "+r"(u[8]), "+r"(u[9]), "+r"(u[10]), "+r"(u[11]), "+r"(u[12]), "+r"(u[13]), "+r"(u[14]), "+r"(u[15]));
}
__device__ __forceinline__ uint64_t pack2(uint32_t x, uint32_t y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(x), "r"(y));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t r, float &x, float &y) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(r));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ void lds_2x64(uint32_t addr, uint64_t &a, uint64_t &b) {
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(addr));
}
__device__ __forceinline__ float lds_cluster(uint32_t addr) {
    float r;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(r) : "r"(addr) : "memory");
    return r;
}
__device__ __forceinline__ uint32_t mapa(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void group_sync(int g) { asm volatile("bar.sync %0, 128;" ::"r"(1 + g) : "memory"); }

// Four scales from index i on, of which `left` exist, as they lie in memory: f32 bits, or bytes (packed in .x if vec).
__device__ __forceinline__ uint4 load_scales(const void *p, int fmt, bool vec, int64_t i, int left) {
    uint4 r = make_uint4(0u, 0u, 0u, 0u);
    if (fmt == ENGRAM_FMT_FP8_E8M0) {
        const uint8_t *b = static_cast<const uint8_t *>(p) + i;
        if (vec) {
            r.x = __ldg(reinterpret_cast<const uint32_t *>(b));
        } else {
            r.x = __ldg(b);
            if (left > 1) r.y = __ldg(b + 1);
            if (left > 2) r.z = __ldg(b + 2);
            if (left > 3) r.w = __ldg(b + 3);
        }
    } else {
        const uint32_t *f = static_cast<const uint32_t *>(p) + i;
        if (vec) {
            r = __ldg(reinterpret_cast<const uint4 *>(f));
        } else {
            r.x = __ldg(f);
            if (left > 1) r.y = __ldg(f + 1);
            if (left > 2) r.z = __ldg(f + 2);
            if (left > 3) r.w = __ldg(f + 3);
        }
    }
    return r;
}
__device__ __forceinline__ float scale_at(const uint4 &r, int fmt, bool vec, int j) {
    const uint32_t w = j == 0 ? r.x : j == 1 ? r.y : j == 2 ? r.z : r.w;
    if (fmt != ENGRAM_FMT_FP8_E8M0) return __uint_as_float(w);
    return e8m0_to_f32(vec ? (r.x >> (8 * j)) & 255u : w);
}

template <bool GLU, int NT>
__global__ void __launch_bounds__(kThreads, 1) product_kernel(const __grid_constant__ Params p) {
    using C = Cfg<NT>;
    constexpr int ST = C::kStages, FS = C::kFactors, NC = C::kChunks;
    extern __shared__ uint8_t smem_raw[];
    const ProductArgs &a = p.a;
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw);
    auto full = [&](int s) { return base + C::oBar + 8u * s; };
    auto empty = [&](int s) { return base + C::oBar + 8u * (ST + s); };
    auto ffull = [&](int s) { return base + C::oBar + 8u * (2 * ST + s); };
    auto fempty = [&](int s) { return base + C::oBar + 8u * (2 * ST + FS + s); };
    auto tfull = [&](int b) { return base + C::oBar + 8u * (2 * ST + 2 * FS + b); };
    auto tempty = [&](int b) { return base + C::oBar + 8u * (2 * ST + 2 * FS + 2 + b); };
    const uint32_t drain = base + C::oBar + 8u * (2 * ST + 2 * FS + 4);
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(smem + C::oFlag);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::oFlag + 4);
    int *first = reinterpret_cast<int *>(smem + C::oLists), *count = first + a.E, *before = count + a.E;
    constexpr uint32_t kCols = 4 * NT;               // two buffers of two blocks

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < ST; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int s = 0; s < FS; ++s) {
            mbar_init(ffull(s), 1);
            mbar_init(fempty(s), kEpiWarps);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull(b), 1);
            mbar_init(tempty(b), kEpiWarps);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32((const void *)tmem_slot)), "r"(kCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // the experts' rows and how many row tiles come before each
    for (int e = threadIdx.x; e < a.E; e += kThreads) {
        int lo = 0, n = a.n_pairs;
        if (a.offsets) {
            lo = a.offsets[e];
            const int hi = a.offsets[e + 1];
            n = hi - lo;
            if (lo < 0 || hi < lo || hi > a.n_pairs) {
                set_err(a.err, ENGRAM_E_LENGTH);
                lo = n = 0;
            }
        }
        first[e] = lo;
        count[e] = n;
    }
    __syncthreads();
    if (warp == 2) {
        int carry = 0;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = e0 + lane, x = e < a.E ? (count[e] + NT - 1) / NT : 0;
            int s = x;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xFFFFFFFFu, s, o);
                if (lane >= o) s += y;
            }
            if (e < a.E) before[e] = carry + s - x;
            carry += __shfl_sync(0xFFFFFFFFu, s, 31);
        }
        if (lane == 0) before[a.E] = carry;
    }
    tc_fence_before();
    __syncthreads();
    if (p.split > 1) cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    const int rank = p.split > 1 ? (int)cluster_rank() : 0;
    const int t0 = blockIdx.x / p.split, t_step = gridDim.x / p.split;
    const int tiles = before[a.E] * p.m_tiles;
    const int kb0 = p.KB * rank / p.split, kb1 = p.KB * (rank + 1) / p.split;
    auto tile_at = [&](int t) {
        TileAt r;
        int lo = 0, hi = a.E;                        // the last expert with before[e] * m_tiles <= t
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (before[mid] * p.m_tiles <= t)
                lo = mid;
            else
                hi = mid;
        }
        r.e = lo;
        const int nt = before[lo + 1] - before[lo];
        int i, m;
        tile_coords(t - before[lo] * p.m_tiles, nt, p.m_tiles, min(p.group, nt), i, m);
        const int n = count[lo];
        const int r0 = (int)((int64_t)n * i / nt);
        r.row = first[lo] + r0;
        r.n = (int)((int64_t)n * (i + 1) / nt) - r0;
        r.m0 = m * (GLU ? kM : 2 * kM);
        return r;
    };
    // whether the tile has a second block of weight rows
    auto two = [&](const TileAt &t) { return GLU || t.m0 + kM < a.N; };
    auto wait = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity & 1, abort_flag, a.err)) != 0;
    };
    // x row of a pair's place in the lists; a bad pair reads row 0
    auto token_of = [&](int row) {
        const int pair = __ldg(a.pairs + row);
        if ((uint32_t)pair < (uint32_t)a.n_pairs) return pair / a.top_k;
        set_err(a.err, ENGRAM_E_ROW);
        return 0;
    };
    const bool gather = GLU && a.pairs;

    if (warp == 0) {
        // ---- copies ----
        uint32_t it = 0;
        bool ok = true;
        for (int t = t0; t < tiles && ok; t += t_step) {
            const TileAt w = tile_at(t);
            const bool both = two(w);
            const int n16 = (w.n + 15) & ~15;
            const uint32_t bytes = (both ? 2u : 1u) * kTileA + (uint32_t)n16 * 128u;
            int tok[4];
            if (gather && 4 * lane < n16) {
#pragma unroll
                for (int i = 0; i < 4; ++i) tok[i] = token_of(w.row + min(4 * lane + i, w.n - 1));
            }
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int s = it % ST;
                if (!(ok = wait(empty(s), (it / ST) & 1 ^ 1))) break;
                const uint32_t at = base + s * C::kStage, bar = full(s);
                if (lane == 0) {
                    mbar_expect_tx(bar, bytes);
                    tma_weights(at, &p.mw, kb * 128, w.m0, 0, w.e, bar);
                    if (both) tma_weights(at + kTileA, &p.mw, kb * 128, GLU ? w.m0 : w.m0 + kM, GLU ? 1 : 0, w.e, bar);
                }
                __syncwarp();
                if (gather) {
                    if (4 * lane < n16) tma_gather4(at + 2 * kTileA + lane * 512, &p.mx, kb * 128, tok, bar);
                } else if (16 * lane < n16) {
                    tma_rows(at + 2 * kTileA + lane * 2048, &p.mx, kb * 128, w.row + 16 * lane, bar);
                }
            }
        }
        // copies already issued land before the CTA can leave
        for (uint32_t d = 1; d <= (uint32_t)ST && d <= it; ++d) {
            const uint32_t last = it - d;
            const uint64_t began = now_ns();
            while (!mbar_try(full(last % ST), (last / ST) & 1) && now_ns() - began < 10000000ull) {
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---- MMA ----
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (int t = t0; t < tiles && ok; t += t_step) {
                const TileAt w = tile_at(t);
                const bool both = two(w);
                const uint32_t idesc = idesc_f8((w.n + 15) & ~15);
                for (int kb = kb0; kb < kb1; ++kb, ++it) {
                    const int s = it % ST, b = it & 1;
                    if (!(ok = mbar_wait(tempty(b), (it >> 1) & 1 ^ 1, abort_flag, a.err))) break;
                    if (!(ok = mbar_wait(full(s), (it / ST) & 1, abort_flag, a.err))) break;
                    tc_fence_after();
                    const uint32_t at = base + s * C::kStage, d = tmem + b * 2 * NT;
                    const uint64_t d0 = sdesc(at), d1 = sdesc(at + kTileA), db = sdesc(at + 2 * kTileA);
#pragma unroll
                    for (int k = 0; k < 4; ++k) mma_f8(d, d0 + 2u * k, db + 2u * k, idesc, k != 0);
                    if (both) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) mma_f8(d + NT, d1 + 2u * k, db + 2u * k, idesc, k != 0);
                    }
                    commit(empty(s));
                    commit(tfull(b));
                }
            }
            // every MMA issued has finished before tensor memory can be freed
            commit(drain);
            const uint64_t began = now_ns();
            while (!mbar_try(drain, 0) && now_ns() - began < 100000000ull) {
            }
        }
        __syncwarp();
    } else if (warp == 2) {
        // ---- factors ----
        constexpr int NV = NT / 32;
        const bool vec_x = p.KB % 4 == 0 && reinterpret_cast<uintptr_t>(a.x_scales) % (a.x_fmt == ENGRAM_FMT_FP8 ? 16 : 4) == 0;
        const bool vec_w = p.KB % 4 == 0 && reinterpret_cast<uintptr_t>(a.w_scales) % (a.w_fmt == ENGRAM_FMT_FP8 ? 16 : 4) == 0;
        uint32_t it = 0;
        bool ok = true;
        for (int t = t0; t < tiles && ok; t += t_step) {
            const TileAt w = tile_at(t);
            const bool both = two(w);
            int64_t xi[NV];
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c = v * 32 + lane;
                xi[v] = c < w.n ? (int64_t)(gather ? token_of(w.row + c) : w.row + c) * p.KB : -1;
            }
            const int nb = w.m0 / kM;
            const int64_t w0 = ((int64_t)w.e * (GLU ? 2 : 1) * p.NB + nb) * p.KB, w1 = w0 + (int64_t)(GLU ? p.NB : 1) * p.KB;
            uint4 x[NV], s0 = make_uint4(0u, 0u, 0u, 0u), s1 = s0;
            auto fetch = [&](int kb) {               // kb a multiple of 4
                const int left = p.KB - kb;
#pragma unroll
                for (int v = 0; v < NV; ++v)
                    if (xi[v] >= 0) x[v] = load_scales(a.x_scales, a.x_fmt, vec_x, xi[v] + kb, left);
                s0 = load_scales(a.w_scales, a.w_fmt, vec_w, w0 + kb, left);
                if (both) s1 = load_scales(a.w_scales, a.w_fmt, vec_w, w1 + kb, left);
            };
            fetch(kb0 & ~3);
            for (int kb4 = kb0 & ~3; kb4 < kb1 && ok; kb4 += 4) {
                uint4 y[NV];
                const uint4 z0 = s0, z1 = s1;
#pragma unroll
                for (int v = 0; v < NV; ++v) y[v] = x[v];
                if (kb4 + 4 < kb1) fetch(kb4 + 4);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int kb = kb4 + j;
                    if (kb < kb0 || kb >= kb1 || !ok) continue;
                    const int s = it % FS;
                    if (!(ok = wait(fempty(s), (it / FS) & 1 ^ 1))) continue;
                    float *f = reinterpret_cast<float *>(smem + C::oFactor) + s * 2 * NT;
                    const float g0 = scale_at(z0, a.w_fmt, vec_w, j), g1 = scale_at(z1, a.w_fmt, vec_w, j);
#pragma unroll
                    for (int v = 0; v < NV; ++v) {
                        const float sx = xi[v] >= 0 ? scale_at(y[v], a.x_fmt, vec_x, j) : 0.f;
                        f[v * 32 + lane] = sx * g0;
                        f[NT + v * 32 + lane] = sx * g1;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(ffull(s));
                    ++it;
                }
            }
        }
    } else {
        // ---- sums and output ----
        const int g = (warp - 3) >> 2, q = warp & 3, m = 32 * q + lane, tw = threadIdx.x - 96 - 128 * g;
        const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16);
        uint32_t it = 0, turn = 0;
        // Writes rows c0 .. c0 + n - 1 of tile w, n <= 16: v0, v1 the sums of weight rows m of its two blocks.
        auto finish = [&](const TileAt &w, float (&v0)[16], float (&v1)[16], int c0, int n) {
            if (GLU) {
                const int par = turn++ & 1;
                uint32_t *amax = reinterpret_cast<uint32_t *>(smem + C::oMax) + (g * 2 + par) * 64;
                uint8_t *codes = smem + C::oCodes + (g * 2 + par) * 2048;
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    float x = v0[j], u = v1[j];
                    if (a.limit > 0.f) {
                        x = x > a.limit ? a.limit : x;              // NaN stays
                        u = u > a.limit ? a.limit : u < -a.limit ? -a.limit : u;
                    }
                    v0[j] = x / (1.f + expf(-x)) * u;
                    const uint32_t big = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(fabsf(v0[j])));
                    if (lane == j) amax[4 * j + q] = big;
                }
                group_sync(g);
                auto block_byte = [&](int j) {
                    const uint4 b = *reinterpret_cast<const uint4 *>(amax + 4 * j);
                    return block_scale_byte(max(max(b.x, b.y), max(b.z, b.w)));
                };
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const uint32_t byte = block_byte(j);
                    const float y = byte == 255u ? 0.f : v0[j] * inv_scale(byte);
                    codes[j * 128 + m] = (uint8_t)__nv_cvt_float_to_fp8(y, __NV_SATFINITE, __NV_E4M3);
                }
                group_sync(g);
                const int j = tw >> 3, at = (tw & 7) * 16;
                if (j < n && w.m0 + at < a.N)
                    *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(a.out) + (int64_t)(w.row + c0 + j) * a.N + w.m0 + at) =
                        *reinterpret_cast<const uint4 *>(codes + j * 128 + at);
                if (tw < n) {
                    const uint32_t byte = block_byte(tw);
                    const int64_t i = (int64_t)(w.row + c0 + tw) * p.NB + w.m0 / kM;
                    if (a.out_type == ENGRAM_FMT_FP8_E8M0)
                        static_cast<uint8_t *>(a.out_scales)[i] = (uint8_t)byte;
                    else
                        static_cast<float *>(a.out_scales)[i] = e8m0_to_f32(byte);
                }
            } else {
                const int col = w.m0 + m;
                const bool in0 = col < a.N, in1 = col + kM < a.N;
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    if (j >= n) break;
                    int64_t r = w.row + c0 + j;
                    if (a.pairs) {
                        r = __ldg(a.pairs + r);
                        if ((uint64_t)r >= (uint64_t)a.n_pairs) {
                            set_err(a.err, ENGRAM_E_ROW);
                            continue;
                        }
                    }
                    r = r * a.out_stride + col;
                    if (a.out_type == ENGRAM_T_BF16) {
                        if (in0) static_cast<__nv_bfloat16 *>(a.out)[r] = __float2bfloat16_rn(v0[j]);
                        if (in1) static_cast<__nv_bfloat16 *>(a.out)[r + kM] = __float2bfloat16_rn(v1[j]);
                    } else if (a.out_type == ENGRAM_T_F16) {
                        if (in0) static_cast<__half *>(a.out)[r] = __float2half_rn(v0[j]);
                        if (in1) static_cast<__half *>(a.out)[r + kM] = __float2half_rn(v1[j]);
                    } else {
                        if (in0) static_cast<float *>(a.out)[r] = v0[j];
                        if (in1) static_cast<float *>(a.out)[r + kM] = v1[j];
                    }
                }
            }
        };
        bool ok = true;
        for (int t = t0; t < tiles && ok; t += t_step) {
            const TileAt w = tile_at(t);
            const bool both = two(w);
            uint64_t acc0[NC][8], acc1[NC][8];
#pragma unroll
            for (int i = 0; i < NC; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) acc0[i][j] = acc1[i][j] = 0;
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int b = it & 1, s = it % FS;
                if (!(ok = wait(ffull(s), it / FS) && wait(tfull(b), it >> 1))) break;
                tc_fence_after();
                const uint32_t f = base + C::oFactor + s * 2 * NT * 4, d = lanes + b * 2 * NT;
#pragma unroll
                for (int i = 0; i < NC; ++i) {
                    const int c0 = (2 * i + g) * 16;
                    if (c0 >= w.n) break;
                    uint32_t u0[16], u1[16];
                    tmem_ld16(d + c0, u0);
                    if (both) tmem_ld16(d + NT + c0, u1);
                    tmem_wait_ld();
                    pin16(u0);
#pragma unroll
                    for (int j = 0; j < 8; j += 2) {
                        uint64_t x, y;
                        lds_2x64(f + (c0 + 2 * j) * 4, x, y);
                        acc0[i][j] = fma2(pack2(u0[2 * j], u0[2 * j + 1]), x, acc0[i][j]);
                        acc0[i][j + 1] = fma2(pack2(u0[2 * j + 2], u0[2 * j + 3]), y, acc0[i][j + 1]);
                    }
                    if (both) {
                        pin16(u1);
#pragma unroll
                        for (int j = 0; j < 8; j += 2) {
                            uint64_t x, y;
                            lds_2x64(f + (NT + c0 + 2 * j) * 4, x, y);
                            acc1[i][j] = fma2(pack2(u1[2 * j], u1[2 * j + 1]), x, acc1[i][j]);
                            acc1[i][j + 1] = fma2(pack2(u1[2 * j + 2], u1[2 * j + 3]), y, acc1[i][j + 1]);
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(tempty(b));
                    mbar_arrive(fempty(s));
                }
            }
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int c0 = (2 * i + g) * 16;
                if (c0 >= w.n) break;
                float v0[16], v1[16];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    unpack2(acc0[i][j], v0[2 * j], v0[2 * j + 1]);
                    unpack2(acc1[i][j], v1[2 * j], v1[2 * j + 1]);
                }
                if (p.split == 1) {
                    finish(w, v0, v1, c0, min(16, w.n - c0));
                } else {
                    // this part's sums as [row][256]; the ring they overwrite is drained: a cluster has one tile
                    float *part = reinterpret_cast<float *>(smem) + c0 * 2 * kM + m;
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        part[j * 2 * kM] = v0[j];
                        part[j * 2 * kM + kM] = v1[j];
                    }
                }
            }
        }
        __syncwarp();
        if (p.split > 1) {
            cluster_sync();
            if (t0 < tiles && ok) {
                const TileAt w = tile_at(t0);
                const int lo = w.n * rank / p.split, hi = w.n * (rank + 1) / p.split;
                for (int c0 = lo + 16 * g; c0 < hi; c0 += 32) {
                    float v0[16], v1[16];
                    const int n = min(16, hi - c0);
#pragma unroll
                    for (int j = 0; j < 16; ++j) v0[j] = v1[j] = 0.f;
                    for (int r = 0; r < p.split; ++r) {
                        const uint32_t part = mapa(base, (uint32_t)r) + (uint32_t)(c0 * 2 * kM + m) * 4;
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            if (j >= n) break;
                            v0[j] += lds_cluster(part + j * 2 * kM * 4);
                            v1[j] += lds_cluster(part + j * 2 * kM * 4 + kM * 4);
                        }
                    }
                    finish(w, v0, v1, c0, n);
                }
            }
            cluster_sync();
        }
    }
    if (p.split > 1 && warp < 3) {
        __syncwarp();
        cluster_sync();
        cluster_sync();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols) : "memory");
}

template <bool GLU, int NT>
cudaError_t launch_tile(Params &p, cudaStream_t s) {
    using C = Cfg<NT>;
    const ProductArgs &a = p.a;
    static bool attr[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(product_kernel<GLU, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)C::bytes(kMaxExperts));
        if (e != cudaSuccess) return e;
        attr[dev] = true;
    }
    p.m_tiles = (a.N + (GLU ? kM : 2 * kM) - 1) / (GLU ? kM : 2 * kM);
    // row tiles at most
    const int64_t row_tiles = a.offsets ? (int64_t)(a.n_pairs < a.E ? a.n_pairs : a.E) + a.n_pairs / NT : (a.n_pairs + NT - 1) / NT;
    const int64_t tiles = row_tiles * p.m_tiles;
    if (tiles > 0x3FFFFFFF) return cudaErrorInvalidConfiguration;
    // a cluster shares a tile while that leaves SMs idle otherwise, with two K blocks a CTA at least
    p.split = 1;
    while (p.split < 8 && tiles * p.split * 2 <= a.sms && p.KB >= p.split * 4) p.split *= 2;
    // row tiles of a dense product side by side whose rows stay in L2
    const int64_t rows_l2 = (int64_t(48) << 20) / a.K / NT;
    p.group = (int)(rows_l2 < 8 ? 8 : rows_l2 > 0x3FFFFFFF ? 0x3FFFFFFF : rows_l2);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.split > 1 ? tiles * p.split : tiles < a.sms ? tiles : a.sms));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::bytes(a.E);
    cfg.stream = s;
    cudaLaunchAttribute la[1];
    la[0].id = cudaLaunchAttributeClusterDimension;
    la[0].val.clusterDim.x = (unsigned)p.split;
    la[0].val.clusterDim.y = la[0].val.clusterDim.z = 1;
    cfg.attrs = la;
    cfg.numAttrs = p.split > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, product_kernel<GLU, NT>, p);
}

}  // namespace

cudaError_t launch_product(const ProductArgs &a, cudaStream_t s) {
    Params p;
    p.a = a;
    p.KB = (a.K + kScaleBlock - 1) / kScaleBlock;
    p.NB = (a.N + kScaleBlock - 1) / kScaleBlock;
    const uint64_t parts = a.glu ? 2 : 1, K = (uint64_t)a.K, N = (uint64_t)a.N;
    const uint64_t wd[4] = {K, N, parts, (uint64_t)a.E}, wst[3] = {K, N * K, parts * N * K};
    const uint32_t wbox[4] = {128, kM, 1, 1};
    const uint64_t xd[2] = {K, (uint64_t)a.rows}, xst[1] = {(uint64_t)a.x_stride};
    const uint32_t xbox[2] = {128, a.glu && a.pairs ? 1u : 16u};
    if (!make_map_u8(&p.mw, a.w, 4, wd, wst, wbox) || !make_map_u8(&p.mx, a.x, 2, xd, xst, xbox)) return cudaErrorInvalidValue;
    // rows an expert has on average: a tile of few rows leaves shared memory to the weights on their way
    const int rows = a.offsets ? (a.n_pairs + a.E - 1) / a.E : a.n_pairs;
    if (a.glu) return rows <= 24 ? launch_tile<true, 32>(p, s) : rows <= 56 ? launch_tile<true, 64>(p, s) : launch_tile<true, 128>(p, s);
    return rows <= 24 ? launch_tile<false, 32>(p, s) : rows <= 56 ? launch_tile<false, 64>(p, s) : launch_tile<false, 128>(p, s);
}

}  // namespace engram
