// product.cuh -- what the two kernels of the 8-bit products share (product.cu: few
// rows, product_rows.cu: many): their parameters, the walk over the (expert, weight
// rows, rows) tiles, scales, copies and MMAs.
#pragma once

#include "experts.cuh"
#include "tcgen05.cuh"

#include <mutex>

namespace engram {

namespace product {

using namespace tcg;

constexpr int kM = 128;                              // values of a K block, weight rows of a scale
constexpr uint32_t kTileA = kM * 128;                // bytes of 128 rows of a K block

struct Params {
    ProductArgs a;
    CUtensorMap mw, mx, mx16;                        // weights (256 rows of a part, or 128 of both); rows of x in large and small boxes
    int KB, NB;                                      // blocks of K, of N
    int m_tiles;                                     // of an expert
    int split;                                       // CTAs that share a tile
    int group;                                       // row tiles side by side
    int wide;                                        // outputs may be written 16 (1) or 32 (2) bytes at a time
};

struct TileAt {
    int e, row, n, m0;                               // expert, first row, rows, first weight row
};

constexpr long long kWaitClocks = 2 * (long long)kWaitNs;
// Bounded wait as common.cuh's mbar_wait, for a whole warp, by the SM's clock (about 2 s; reading the timer takes longer than most waits
// here).  (One lane that waits for its warp is slow: 1245 clocks for a hand-over that takes all lanes 513.)
// Once the flag is up a wait ends after 64 tests, so that loops may vote on the outcome at their end alone.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort_flag, int *err) {
    bool ok = true;
    long long began = 0;
    for (uint32_t i = 1; !mbar_try(bar, parity); ++i) {
        if (i & 63) continue;
        if (*abort_flag) {
            ok = false;
            break;
        }
        const long long now = clock64();
        if (!began) began = now;
        if (now - began > kWaitClocks) {
            *abort_flag = 1;
            set_err(err, ENGRAM_E_TIMEOUT);
            ok = false;
            break;
        }
    }
    __syncwarp();
    return ok;                                       // of this lane
}
// One lane of a converged warp.  (Issued by "lane == 0" instead, a block's four MMAs and two commits took the warp 700 clocks.)
__device__ __forceinline__ bool elect() {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
}
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t da, uint64_t db, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(da), "l"(db), "r"(idesc), "r"(accumulate)
        : "memory");
}
// kind::f8f6f4, e4m3 x e4m3 (formats 0), f32 sums, both K-major.
__device__ __forceinline__ uint32_t idesc_f8(int N) {   // M 128
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
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
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool real) {   // zeros unless real
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
// 16 columns of this warp's 32 tensor-memory lanes (without the wait).
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&u)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
          "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;"); }
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
// acc += u * f over 16 columns.
__device__ __forceinline__ void add_chunk(uint64_t (&acc)[8], const uint32_t (&u)[16], const float *f) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(f + 2 * j);
        acc[j] = fma2(pack2(u[2 * j], u[2 * j + 1]), x.x, acc[j]);
        acc[j + 1] = fma2(pack2(u[2 * j + 2], u[2 * j + 3]), x.y, acc[j + 1]);
    }
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
// The sums of all CTAs' f32 values at base + at[j], j < n <= N, in CTA order; their loads are all under way at once.
template <int N>
__device__ __forceinline__ void sum_of_cluster(uint32_t base, int split, const uint32_t (&at)[N], int n, float (&sum)[N]) {
    float x[8][N];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        const uint32_t of = mapa(base, (uint32_t)min(r, split - 1));
#pragma unroll
        for (int j = 0; j < N; ++j) x[r][j] = r < split && j < n ? lds_cluster(of + at[j]) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
        sum[j] = x[0][j];
#pragma unroll
        for (int r = 1; r < 8; ++r) sum[j] += x[r][j];
    }
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// 32 bytes, 32-byte aligned: a whole sector of L2.
__device__ __forceinline__ void st32(void *p, const uint32_t (&u)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 ::"l"(p), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]) : "memory");
}
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


// The experts' rows (global memory: after griddep_wait) and how many tiles of up to `rows` rows come before each: shared memory, by all threads.
// An expert counts only if its offsets rise from where those before it that count have ended: their rows are at most n_pairs in all, and
// their tiles at most product_row_tiles(), for which the grid of clusters is made.
__device__ __forceinline__ void set_lists(const ProductArgs &a, int *first, int *count, int *before, int rows, int threads) {
    int bad = 0;
    for (int e = threadIdx.x; e < a.E; e += threads) {
        int lo = 0, n = a.n_pairs;
        if (a.offsets) {
            lo = a.offsets[e];
            const int hi = a.offsets[e + 1];
            n = hi - lo;
            if (lo < 0 || hi < lo || hi > a.n_pairs) {
                set_err(a.err, ENGRAM_E_LENGTH);
                lo = n = 0;
                bad = 1;
            }
        }
        first[e] = lo;
        count[e] = n;
    }
    // offsets that rise everywhere need no more than that
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) {
            int end = 0;
            for (int e = 0; e < a.E; ++e) {
                if (!count[e]) continue;
                if (first[e] < end) {
                    set_err(a.err, ENGRAM_E_LENGTH);
                    first[e] = count[e] = 0;
                } else {
                    end = first[e] + count[e];
                }
            }
        }
        __syncthreads();
    }
    if (threadIdx.x >= 32) return;
    const int lane = threadIdx.x;
    int carry = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
        const int e = e0 + lane, x = e < a.E ? (count[e] + rows - 1) / rows : 0;
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

// Tile t of the list; an expert's rows are cut into tiles of like size.
__device__ __forceinline__ TileAt tile_of(const Params &p, const int *first, const int *count, const int *before, int t, int m_rows) {
    TileAt r;
    int lo = 0, hi = p.a.E;                          // the last expert with before[e] * m_tiles <= t
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
    const int at = t - before[lo] * p.m_tiles;
    if (p.group >= nt) {
        m = (int)((unsigned)at / (unsigned)nt);
        i = at - m * nt;
    } else {
        tile_coords(at, nt, p.m_tiles, p.group, i, m);
    }
    const int n = count[lo], each = (int)((unsigned)n / (unsigned)nt), more = n - each * nt;
    r.row = first[lo] + i * each + min(i, more);
    r.n = each + (i < more);
    r.m0 = m * m_rows;
    return r;
}

// x row of a pair's place in the lists; a bad pair reads row 0.
__device__ __forceinline__ int token_of(const ProductArgs &a, int row) {
    const int pair = __ldg(a.pairs + row);
    if ((uint32_t)pair < (uint32_t)a.n_pairs) return pair / a.top_k;
    set_err(a.err, ENGRAM_E_ROW);
    return 0;
}
// Output row of a place in the lists; -1 for a bad pair.
__device__ __forceinline__ int out_row_of(const ProductArgs &a, int row) {
    const int pair = __ldg(a.pairs + row);
    if ((uint32_t)pair < (uint32_t)a.n_pairs) return pair;
    set_err(a.err, ENGRAM_E_ROW);
    return -1;
}
// g / (1 + e^-g) u of the clamped g and u; NaN stays.  (The quotient is off by 2 ulp; a denominator over 2^126, g under -87, gives 0.)
__device__ __forceinline__ float gated(float g, float u, float limit) {
    if (limit > 0.f) {
        g = g > limit ? limit : g;
        u = u > limit ? limit : u < -limit ? -limit : u;
    }
    return __fdividef(g, 1.f + expf(-g)) * u;
}
// Whether four scales can be loaded at once.
__device__ __forceinline__ bool four_at_once(const void *scales, int fmt, int KB) {
    return KB % 4 == 0 && reinterpret_cast<uintptr_t>(scales) % (fmt == ENGRAM_FMT_FP8 ? 16 : 4) == 0;
}

using Kernel = void (*)(const Params);

// Of one kernel on one device: whether its shared memory is allowed, and how many clusters of each size run at once.
struct Fit {
    bool ready;
    int clusters[9];
};
// The current device's of fits[64] (a kernel's, made at its first call), copied to *out.  smem: what the most experts need.
inline cudaError_t fit_of(Fit *fits, Kernel kernel, int threads, size_t smem, Fit *out) {
    static std::mutex mutex;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mutex);
    Fit *fit = fits + dev;
    *out = *fit;
    if (fit->ready) return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    for (int s = 2; s <= 8 && e == cudaSuccess; ++s) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)s);
        cfg.blockDim = dim3((unsigned)threads);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute la[1];
        la[0].id = cudaLaunchAttributeClusterDimension;
        la[0].val.clusterDim.x = (unsigned)s;
        la[0].val.clusterDim.y = la[0].val.clusterDim.z = 1;
        cfg.attrs = la;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&fit->clusters[s], kernel, &cfg);
    }
    fit->ready = e == cudaSuccess;
    *out = *fit;
    return e;
}
// How many CTAs share a tile (at most `most`): the most of 2..8 (powers of two) for which all clusters run at once, or 1.
inline int fitting_split(const Fit &fit, int64_t tiles, int most, bool powers) {
    for (int s = 8; s > 1; s = powers ? s / 2 : s - 1)
        if (s <= most && tiles <= fit.clusters[s]) return s;
    return 1;
}
inline cudaError_t launch_split(Kernel kernel, const Params &p, int64_t tiles, int threads, size_t smem, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.split > 1 ? tiles * p.split : tiles < p.a.sms ? tiles : p.a.sms));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute la[2];
    la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // the set-up runs beside the end of the kernel before
    la[0].val.programmaticStreamSerializationAllowed = 1;
    la[1].id = cudaLaunchAttributeClusterDimension;
    la[1].val.clusterDim.x = (unsigned)p.split;
    la[1].val.clusterDim.y = la[1].val.clusterDim.z = 1;
    cfg.attrs = la;
    cfg.numAttrs = p.split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace product

cudaError_t launch_product_rows(product::Params &p, cudaStream_t s);   // product_rows.cu
int product_row_tiles(const ProductArgs &a, int rows);                // tiles of up to `rows` rows, at most

}  // namespace engram
