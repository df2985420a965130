// product_rows.cu -- the products of product.cu for many rows (prompts): 128 rows of x
// on the M side of the MMA, 256 weight rows (or 128 of the gate and the other's 128) on its N side.
//
// With weights on M a factor belongs to a column, and reading it from shared memory for
// every column, beside operands that two N = 128 MMAs read twice, bounds a block at 1500
// clocks.  Here a thread has one row: its factors sx sw are two registers a block, an
// MMA of M 128, N 256, K 32 reads 12 KB for 128 clocks, and a row's largest output is
// found by the threads that hold it.
//
// Roles (16 warps, or 12):
//   warp 0       TMA: a block's 256 weight rows and, unless they are gathered, its 128 rows of x;
//   warp 1       issues the MMAs, two 256-column buffers in tensor memory;
//   warps 2, 3   scales of a block's rows and weights, to shared memory (a load of theirs takes the better part of
//                two blocks beside the copies);
//   warps 4..7   (where there are any) rows of x that the lists gather, by 16-byte asynchronous copies (a block of 128 rows
//                takes four warps 290 clocks, one warp 690; as tile::gather4 2200 to 2900);
//   the last 8   take a block's sums into their f32 accumulators (thread: a row, 128 columns,
//                for glu 64 of each part; 128 KB of them in about 300 clocks); at the end of a tile they write it.
// Where both scales are powers of two (e8m0 bytes) the tensor cores apply them: tcgen05.mma kind::mxf8f6f4 with a
// block's bytes in tensor memory (four blocks to a 32-bit column; an MMA names its byte).  Sums then stay in tensor memory over
// all of K, in one 256-column buffer, and the last warps take them once a tile: f32, but each MMA of 32 values cuts off what lies under the last
// bit of the running sum, which 65536 products of one sign feel (9e-6 of the sum; 4096: 9e-8; blocks added in registers 7e-8).
// Where there are fewer tiles than SMs a cluster shares a tile as in product.cu, K cut at groups of four blocks.
// Waits are bounded as in product.cu.
//
// Bounds, measured: powers of two, 8192 rows, 4096 -> 6144: 132 us, 3.1 PFLOP/s; a block's 48 KB come from L2 at 64 bytes a clock and SM in
// 750 clocks, its MMAs take 514, and in long runs power holds the clock at 1.7 GHz.  Other scales: about 1000 clocks a block, of which the
// last warps' eight loads of 64 clocks in turn are half; the other half (waits for the hand-over, latency that two warps a scheduler do not
// cover) is not accounted for: the same product 180 us; 4096 tokens, 8 of 64 experts, 4096 -> 2 x 1024 325 us, and back 173; with powers of two
// 254 and 136.  Outputs whose rows are no multiples of 16 bytes are written element by element, a thread a row: 4096 rows, 4096 -> 4096 in
// bf16 52 us, 4096 -> 4095 183.
#include "product.cuh"

#include <type_traits>

namespace engram {

namespace {

using namespace product;

constexpr int kRows = 128, kCols = 256;
constexpr int kScaleWarp = 2, kCopyWarp = 4, kCopyWarps = 4, kEpiWarps = 8;
// Without gathered rows there are no copying warps (but where the tensor cores apply scales, which needs no more registers: 134 us for 140).
constexpr int epi_warp(bool mx, bool gather) { return mx || gather ? kCopyWarp + kCopyWarps : kCopyWarp; }
constexpr int threads_of(bool mx, bool gather) { return 32 * (epi_warp(mx, gather) + kEpiWarps); }
constexpr uint32_t kStage = 3 * kTileA;              // x, then the weights
constexpr int kStages = 4;
// Scales of four blocks at a time (the last of a tile: what is left), [4][128] of rows and [4][2] of weights.
constexpr int kSlots = 3;
constexpr uint32_t kSlotBytes = 4 * kRows * 4 + 128;
// For the tensor cores: a 32-bit word (a byte a block) for each row of x and weight row, 32 x 4 of them an image of 512 bytes.
constexpr uint32_t kImage = 512, kScaleCols = 16;         // tensor-memory columns of a group of four blocks: 4 of rows, 8 of weights
constexpr uint32_t kScaleTmem = kCols;                    // behind the sums
static_assert(3 * kImage <= kSlotBytes, "images in a slot of scales");
// What the last warps need to know of a tile: the first weight row, and where its 128 rows go (-1: nowhere).  The scales' warps, which
// write it, are up to three groups of blocks ahead of the MMAs, and these a tile ahead of the last warps: with tiles of one group, five tiles.
constexpr int kRecords = 6;
constexpr uint32_t kRecordBytes = kRows * 4 + 16;
constexpr uint32_t oScale = kStages * kStage;             // a multiple of 16
constexpr uint32_t oMax = oScale + kSlots * kSlotBytes;   // glu: [2][2 groups][128] f32 bits
constexpr uint32_t oRecord = oMax + 2 * 2 * kRows * 4;
constexpr uint32_t oBar = oRecord + kRecords * kRecordBytes;
constexpr uint32_t oFlag = oBar + 8 * (2 * kStages + 2 + 2 + 2 * kSlots + 1);
constexpr uint32_t oLists = oFlag + 16;
constexpr size_t smem_bytes(int E) { return 1024 + oLists + (3 * (size_t)E + 1) * 4; }

// acc += u f, with f in both halves of a register pair.
__device__ __forceinline__ void add16(uint64_t *acc, const uint32_t (&u)[16], uint64_t f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = fma2(pack2(u[2 * j], u[2 * j + 1]), f, acc[j]);
}

// 32 outputs of one row from column `col` on, of which `left` exist.
template <class T>
__device__ __forceinline__ void store32(void *out, int64_t at, const uint64_t (&acc)[16], int left, int wide) {
    if (left <= 0) return;
    T *o = static_cast<T *>(out) + at;
    if (wide && left >= 32) {
        constexpr int kWords = sizeof(T) == 4 ? 32 : 16;
        uint32_t w[kWords];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            float x, y;
            unpack2(acc[j], x, y);
            if (sizeof(T) == 4) {
                w[(2 * j) % kWords] = __float_as_uint(x), w[(2 * j + 1) % kWords] = __float_as_uint(y);
            } else {
                w[j] = sizeof(T) == 2 && std::is_same<T, __half>::value ? pack_f16x2(x, y) : pack_bf16x2(x, y);
            }
        }
        if (wide == 2) {
#pragma unroll
            for (int j = 0; j < kWords; j += 8) {
                const uint32_t u[8] = {w[j], w[j + 1], w[j + 2], w[j + 3], w[j + 4], w[j + 5], w[j + 6], w[j + 7]};
                st32(reinterpret_cast<uint32_t *>(o) + j, u);
            }
        } else {
#pragma unroll
            for (int j = 0; j < kWords; j += 4)
                reinterpret_cast<uint4 *>(o)[j / 4] = make_uint4(w[j], w[j + 1], w[j + 2], w[j + 3]);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        float x, y;
        unpack2(acc[j], x, y);
        if (2 * j < left) o[2 * j] = T(x);
        if (2 * j + 1 < left) o[2 * j + 1] = T(y);
    }
}

// kind::mxf8f6f4: scales of A and B in tensor memory, power-of-two bytes (bit 23); which byte of a column's four in bits 29.. and 4...
__device__ __forceinline__ void mma_mx(uint32_t d, uint64_t da, uint64_t db, uint32_t idesc, uint32_t sa, uint32_t sb, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(d), "l"(da), "l"(db), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ uint32_t idesc_mx(int N, uint32_t byte) {
    return (byte << 4) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | (1u << 27) | (byte << 29);
}
// An image of 32 rows of 16 bytes to 4 columns of all lanes.  Its descriptor: no swizzle, groups of 8 rows 128 bytes apart.
__device__ __forceinline__ void copy_image(uint32_t taddr, uint32_t saddr) {
    const uint64_t desc = (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)1u << 16 | (uint64_t)(128u >> 4) << 32 | (uint64_t)1u << 46;
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// Four bytes of scales from index i on, of which `left` exist (others: 1).
__device__ __forceinline__ uint32_t four_bytes(const void *p, bool vec, int64_t i, int left) {
    const uint8_t *b = static_cast<const uint8_t *>(p) + i;
    if (vec) return __ldg(reinterpret_cast<const uint32_t *>(b));
    uint32_t r = 0x7F7F7F00u | __ldg(b);
    if (left > 1) r = (r & 0xFFFF00FFu) | (uint32_t)__ldg(b + 1) << 8;
    if (left > 2) r = (r & 0xFF00FFFFu) | (uint32_t)__ldg(b + 2) << 16;
    if (left > 3) r = (r & 0x00FFFFFFu) | (uint32_t)__ldg(b + 3) << 24;
    return r;
}

// The part of CTA `rank` of a cluster of S that shares tile w: 128 / S of its rows, from all CTAs' sums, added in CTA order.
// Thread i of 256: a row, and a slice of the columns, half of it (64 loads from the others' shared memory) at a time.
template <bool GLU, int S, class Sync>
__device__ __forceinline__ void share_of_tile(const Params &p, const TileAt &w, uint32_t base, uint8_t *smem, int rank, int i, Sync together) {
    constexpr int kPer = kRows / S, kSlices = 2 * S, kWidth = (GLU ? kM : kCols) / kSlices, kStep = kWidth / 2;
    const ProductArgs &a = p.a;
    const int row = rank * kPer + i % kPer, slice = i / kPer, c0 = slice * kWidth;
    int to = row < w.n ? w.row + row : -1;
    if (!GLU && a.pairs && to >= 0) to = out_row_of(a, to);
    auto sums = [&](int c, float (&v)[kStep]) {
        float x[S][kStep];
#pragma unroll
        for (int r = 0; r < S; ++r) {
            const uint32_t at = mapa(base, (uint32_t)r) + (uint32_t)(c * kRows + row) * 4;
#pragma unroll
            for (int j = 0; j < kStep; ++j) x[r][j] = lds_cluster(at + j * kRows * 4);
        }
#pragma unroll
        for (int j = 0; j < kStep; ++j) {
            v[j] = x[0][j];
#pragma unroll
            for (int r = 1; r < S; ++r) v[j] += x[r][j];
        }
    };
    if (!GLU) {
        if (to < 0) return;
#pragma unroll 1
        for (int c = c0; c < c0 + kWidth && w.m0 + c < a.N; c += kStep) {
            float v[kStep];
            sums(c, v);
#pragma unroll
            for (int j = 0; j < kStep; j += 8) {
                const int col = w.m0 + c + j;
                const int64_t at = (int64_t)to * a.out_stride + col;
                const float y[8] = {v[j % kStep], v[(j + 1) % kStep], v[(j + 2) % kStep], v[(j + 3) % kStep],
                                    v[(j + 4) % kStep], v[(j + 5) % kStep], v[(j + 6) % kStep], v[(j + 7) % kStep]};
                const bool whole = p.wide && col + 8 <= a.N;
                if (whole && a.out_type == ENGRAM_T_BF16) {
                    store8<ENGRAM_T_BF16>(a.out, at, y);
                } else if (whole && a.out_type == ENGRAM_T_F16) {
                    store8<ENGRAM_T_F16>(a.out, at, y);
                } else if (whole) {
                    store8<ENGRAM_T_F32>(a.out, at, y);
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        if (col + k >= a.N) break;
                        if (a.out_type == ENGRAM_T_BF16)
                            static_cast<__nv_bfloat16 *>(a.out)[at + k] = __float2bfloat16_rn(y[k]);
                        else if (a.out_type == ENGRAM_T_F16)
                            static_cast<__half *>(a.out)[at + k] = __float2half_rn(y[k]);
                        else
                            static_cast<float *>(a.out)[at + k] = y[k];
                    }
                }
            }
        }
        return;
    }
    // gated values of the slice ([value][thread] behind the parts), then the row's largest over its slices
    float *mine = reinterpret_cast<float *>(smem + kCols * kRows * 4) + i;
    uint32_t *amax = reinterpret_cast<uint32_t *>(smem + oMax);       // [slices][rows], 256 in all
    float big = 0.f;
#pragma unroll 1
    for (int c = c0; c < c0 + kWidth; c += kStep) {
        float g[kStep], u[kStep];
        sums(c, g);
        sums(kM + c, u);
#pragma unroll
        for (int j = 0; j < kStep; ++j) {
            g[j] = gated(g[j], u[j], a.limit);
            big = amax3(big, g[j], 0.f);
            mine[(c - c0 + j) * 256] = g[j];
        }
    }
    amax[i] = __float_as_uint(big);
    if (!together() || to < 0) return;
    uint32_t most = 0;
#pragma unroll
    for (int s = 0; s < kSlices; ++s) most = max(most, amax[s * kPer + i % kPer]);
    const uint32_t byte = block_scale_byte(most);
    const float inv = byte == 255u ? 0.f : inv_scale(byte);
    for (int c = c0; c < c0 + kWidth && w.m0 + c < a.N; c += 8) {
        uint2 code = make_uint2(0u, 0u);
        if (byte != 255u) {
            const float *v = mine + (c - c0) * 256;
            code.x = e4m3x4(v[0] * inv, v[256] * inv, v[512] * inv, v[768] * inv);
            code.y = e4m3x4(v[1024] * inv, v[1280] * inv, v[1536] * inv, v[1792] * inv);
        }
        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.out) + (int64_t)to * a.N + w.m0 + c) = code;
    }
    if (slice == 0) {
        const int64_t at = (int64_t)to * p.NB + w.m0 / kM;
        if (a.out_type == ENGRAM_FMT_FP8_E8M0)
            static_cast<uint8_t *>(a.out_scales)[at] = (uint8_t)byte;
        else
            static_cast<float *>(a.out_scales)[at] = e8m0_to_f32(byte);
    }
}

// GATHER: rows of x come by the lists (glu).
template <bool GLU, bool MX, bool GATHER>
__global__ void __launch_bounds__(threads_of(MX, GATHER), 1) product_rows_kernel(const __grid_constant__ Params p) {
    constexpr int ST = kStages, kEpiWarp = epi_warp(MX, GATHER), kThreads = threads_of(MX, GATHER);
    extern __shared__ uint8_t smem_raw[];
    const ProductArgs &a = p.a;
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw);
    auto full = [&](int s) { return base + oBar + 8u * s; };
    auto done = [&](int s) { return base + oBar + 8u * (ST + s); };
    auto tempty = [&](int b) { return base + oBar + 8u * (2 * ST + b); };
    const uint32_t drain = base + oBar + 8u * (2 * ST + 2);
    const uint32_t together = drain + 8;
    auto sfull = [&](int i) { return together + 8u * (1 + i); };
    auto sempty = [&](int i) { return together + 8u * (1 + kSlots + i); };
    const uint32_t sums_ready = together + 8u * (1 + 2 * kSlots);
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(smem + oFlag);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + oFlag + 4);
    int *first = reinterpret_cast<int *>(smem + oLists), *count = first + a.E, *before = count + a.E;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < ST; ++s) {
            mbar_init(full(s), GATHER ? 1 + kCopyWarps : 1);
            mbar_init(done(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tempty(b), kEpiWarps);
        }
        mbar_init(drain, 1);
        mbar_init(together, kEpiWarps);
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(sfull(i), 2);
            mbar_init(sempty(i), MX ? 1 : kEpiWarps);
        }
        mbar_init(sums_ready, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32((const void *)tmem_slot)), "r"(512u) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    griddep_wait();
    griddep_launch();
    set_lists(a, first, count, before, kRows, kThreads);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    const int rank = p.split > 1 ? (int)cluster_rank() : 0;
    const int t0 = blockIdx.x / p.split, t_step = gridDim.x / p.split, tiles = before[a.E] * p.m_tiles, KB = p.KB;
    const int fours = (KB + 3) / 4, kb0 = fours * rank / p.split * 4, kb1 = min(KB, fours * (rank + 1) / p.split * 4);
    auto tile_at = [&](int t) { return tile_of(p, first, count, before, t, GLU ? kM : kCols); };
    // whether the tile has weight rows for its second 128 columns
    auto two = [&](const TileAt &t) { return GLU || t.m0 + kM < a.N; };
    auto wait = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xFFFFFFFFu, warp_wait(bar, parity & 1, abort_flag, a.err)) != 0; };
    auto lane_wait = [&](uint32_t bar, uint32_t parity) { return warp_wait(bar, parity & 1, abort_flag, a.err); };

    // 512 threads launch with 128 registers each, and 256 x 64 + 256 x 192 are as many; 384 with 168: 128 x 88 + 256 x 208.  (What
    // the last warps keep in local memory costs a block's step: 184 for 208 took 4096 rows' way back 186 us for 170.)
    if (warp < kEpiWarp) {
        if (kThreads == 512)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        else
            asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    }
    if (warp == 0) {
        // ---- weights, and rows that stand together ----
        uint32_t it = 0;
        bool ok = true;
        for (int t = t0; t < tiles && ok; t += t_step) {
            const TileAt w = tile_at(t);
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int s = it % ST;
                if (!(ok = wait(done(s), it / ST ^ 1))) break;
                if (elect()) {
                    const uint32_t at = base + s * kStage, bar = full(s);
                    mbar_expect_tx(bar, GATHER ? 2 * kTileA : 3 * kTileA);
                    tma_weights(at + kTileA, &p.mw, kb * 128, w.m0, 0, w.e, bar);
                    if (!GATHER) tma_rows(at, &p.mx, kb * 128, w.row, bar);
                }
                __syncwarp();
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
        // (After a wait that ran out, what it issues reads anything and goes to sums that nobody writes.)
        uint32_t it = 0, group = 0, turn = 0;
        bool ok = true;
        const uint64_t desc = sdesc(base);
        for (int t = t0; MX && t < tiles && ok; t += t_step, ++turn) {
            const int N = two(tile_at(t)) ? kCols : kM;
            if (!lane_wait(tempty(0), turn ^ 1)) ok = false;
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int s = it % ST, slot = group % kSlots, byte = kb & 3;
                const uint32_t sa = tmem + kScaleTmem + (group & 1) * kScaleCols, sb = sa + 4;
                const uint64_t da = desc + s * (kStage >> 4), db = da + (kTileA >> 4);
                if (!byte) {
                    if (!lane_wait(sfull(slot), group / kSlots)) ok = false;
                    tc_fence_after();
                    if (elect()) {
                        const uint32_t image = base + oScale + slot * kSlotBytes;
                        copy_image(sa, image);
                        copy_image(sb, image + kImage);
                        copy_image(sb + 4, image + 2 * kImage);
                        commit(sempty(slot));
                    }
                    __syncwarp();
                }
                if (byte == 3) ++group;
                const uint32_t idesc = idesc_mx(N, byte);
                if (!lane_wait(full(s), it / ST)) ok = false;
                tc_fence_after();
                if (elect()) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) mma_mx(tmem, da + 2u * k, db + 2u * k, idesc, sa, sb, (kb - kb0) | k);
                    commit(done(s));
                    if (kb + 1 == kb1) commit(sums_ready);
                }
                __syncwarp();
            }
            if (kb1 & 3) ++group;
            ok = __all_sync(0xFFFFFFFFu, ok);
        }
        for (int t = t0; !MX && t < tiles && ok; t += t_step) {
            const uint32_t idesc = idesc_f8(two(tile_at(t)) ? kCols : kM);
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int s = it % ST;
                const uint32_t d = tmem + (it & 1) * kCols;
                const uint64_t da = desc + s * (kStage >> 4), db = da + (kTileA >> 4);
                if (!lane_wait(full(s), it / ST)) ok = false;
                if (!lane_wait(tempty(it & 1), it >> 1 ^ 1)) ok = false;
                tc_fence_after();
                if (elect()) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) mma_f8(d, da + 2u * k, db + 2u * k, idesc, k != 0);
                    commit(done(s));
                }
                __syncwarp();
            }
            ok = __all_sync(0xFFFFFFFFu, ok);
        }
        // every MMA issued has finished before tensor memory can be freed
        if (elect()) commit(drain);
        __syncwarp();
        const uint64_t began = now_ns();
        while (!mbar_try(drain, 0) && now_ns() - began < 100000000ull) {
        }
        __syncwarp();
    } else if (warp < kCopyWarp) {
        // ---- scales: 64 rows a warp ----
        const int c0 = (warp - kScaleWarp) * 64 + lane;
        const bool vec_x = four_at_once(a.x_scales, a.x_fmt, KB), vec_w = four_at_once(a.w_scales, a.w_fmt, KB);
        uint32_t it = 0, record = 0;
        bool ok = true;
        for (int t = t0; t < tiles && ok; t += t_step, record = record + 1 == kRecords ? 0 : record + 1) {
            const TileAt w = tile_at(t);
            const bool both = two(w);
            int *to = reinterpret_cast<int *>(smem + oRecord + record * kRecordBytes);
            int xi[2];
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const int c = c0 + v * 32;
                xi[v] = c < w.n ? GATHER ? token_of(a, w.row + c) : w.row + c : -1;
                to[c] = c >= w.n ? -1 : GLU || !a.pairs ? w.row + c : out_row_of(a, w.row + c);
            }
            if (warp == kScaleWarp && lane == 0) to[kRows] = w.m0;
            const int64_t w0 = ((int64_t)w.e * (GLU ? 2 : 1) * p.NB + w.m0 / kM) * KB, w1 = w0 + (int64_t)(GLU ? p.NB : 1) * KB;
            if (MX) {
                // this warp's images: rows of x (0 is 2^-127: rows behind the last have 1), or the two blocks of weight rows
                int r4[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c = i * 32 + lane;
                    r4[i] = warp == kScaleWarp && c < w.n ? GATHER ? token_of(a, w.row + c) : w.row + c : -1;
                }
                for (int kb4 = kb0; kb4 < kb1; kb4 += 4, ++it) {
                    const int left = KB - kb4, slot = it % kSlots;
                    uint4 u = make_uint4(0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
                    uint32_t b0 = 0, b1 = 0;
                    if (warp == kScaleWarp) {
                        if (r4[0] >= 0) u.x = four_bytes(a.x_scales, vec_x, (int64_t)r4[0] * KB + kb4, left);
                        if (r4[1] >= 0) u.y = four_bytes(a.x_scales, vec_x, (int64_t)r4[1] * KB + kb4, left);
                        if (r4[2] >= 0) u.z = four_bytes(a.x_scales, vec_x, (int64_t)r4[2] * KB + kb4, left);
                        if (r4[3] >= 0) u.w = four_bytes(a.x_scales, vec_x, (int64_t)r4[3] * KB + kb4, left);
                    } else {
                        b0 = four_bytes(a.w_scales, vec_w, w0 + kb4, left);
                        b1 = both ? four_bytes(a.w_scales, vec_w, w1 + kb4, left) : b0;
                    }
                    if (!(ok = wait(sempty(slot), it / kSlots ^ 1))) break;
                    uint4 *image = reinterpret_cast<uint4 *>(smem + oScale + slot * kSlotBytes) + lane;
                    if (warp == kScaleWarp) {
                        image[0] = u;
                    } else {
                        image[kImage / 16] = make_uint4(b0, b0, b0, b0);
                        image[2 * kImage / 16] = make_uint4(b1, b1, b1, b1);
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sfull(slot));
                }
                continue;
            }
            // where there are registers for it, the next four blocks' scales are on their way while these are written
            constexpr bool kAhead = !GATHER;
            uint4 next_x[2], next_w[2];
            auto fetch = [&](int kb4) {
                const int left = KB - kb4;
#pragma unroll
                for (int v = 0; v < 2; ++v)
                    if (xi[v] >= 0) next_x[v] = load_scales(a.x_scales, a.x_fmt, vec_x, (int64_t)xi[v] * KB + kb4, left);
                next_w[0] = load_scales(a.w_scales, a.w_fmt, vec_w, w0 + kb4, left);
                if (both) next_w[1] = load_scales(a.w_scales, a.w_fmt, vec_w, w1 + kb4, left);
            };
            if (kAhead) fetch(kb0);
            for (int kb4 = kb0; kb4 < kb1; kb4 += 4, ++it) {
                if (!kAhead) fetch(kb4);
                const uint4 x[2] = {next_x[0], next_x[1]}, s0 = next_w[0], s1 = both ? next_w[1] : s0;
                if (kAhead && kb4 + 4 < kb1) fetch(kb4 + 4);
                const int slot = it % kSlots;
                float *f = reinterpret_cast<float *>(smem + oScale + slot * kSlotBytes);
                if (!(ok = wait(sempty(slot), it / kSlots ^ 1))) break;
#pragma unroll
                for (int j = 0; j < 4; ++j)          // blocks behind the last: anything
#pragma unroll
                    for (int v = 0; v < 2; ++v) f[j * kRows + c0 + v * 32] = xi[v] >= 0 ? scale_at(x[v], a.x_fmt, vec_x, j) : 0.f;
                if (warp == kScaleWarp && lane < 8)
                    f[4 * kRows + lane] = scale_at(lane & 1 ? s1 : s0, a.w_fmt, vec_w, lane >> 1);
                __syncwarp();
                if (lane == 0) mbar_arrive(sfull(slot));
            }
        }
    } else if (warp < kEpiWarp) {
        // ---- gathered rows: eight lanes a row of 128 bytes, this warp's four of each 16 rows ----
        constexpr int LAG = 1, NR = kRows / (4 * kCopyWarps);   // blocks in flight behind the newest; rows a lane
        const int r0 = (warp - kCopyWarp) * 4 + (lane >> 3), chunk = lane & 7;
        uint32_t it = 0;
        bool ok = true;
        // the copies of block `done` have landed: its stage is full as far as this warp goes
        auto landed = [&](uint32_t done) {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(full(done % ST));
        };
        for (int t = t0; GATHER && t < tiles && ok; t += t_step) {
            const TileAt w = tile_at(t);
            uint32_t from[NR];                       // where the rows begin, in 16 bytes
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const int r = r0 + i * 4 * kCopyWarps;
                from[i] = r < w.n ? (uint32_t)(token_of(a, w.row + r) * (a.x_stride >> 4)) : 0u;
            }
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int s = it % ST;
                if (!(ok = wait(done(s), it / ST ^ 1))) break;
                const bool real = kb * 128 + chunk * 16 < a.K;
                const uint8_t *src = a.x + (real ? kb * 128 + chunk * 16 : 0);
                // rows 16 apart have the same place in the swizzle
                const uint32_t at = base + s * kStage + r0 * 128 + (chunk ^ (r0 & 7)) * 16;
#pragma unroll
                for (int i = 0; i < NR; ++i)
                    if (16 * i < w.n) cp16(at + i * 2048, src + (uint64_t)from[i] * 16, real);
                asm volatile("cp.async.commit_group;" ::: "memory");
                if (it >= LAG) {
                    cp_wait<LAG>();
                    landed(it - LAG);
                }
            }
        }
        cp_wait<0>();
        for (uint32_t done = it > LAG ? it - LAG : 0; GATHER && ok && done < it; ++done) landed(done);
        __syncwarp();
    } else {
        // ---- sums and output ----
        if (kThreads == 512)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
        else
            asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        const int g = (warp - kEpiWarp) >> 2, q = warp & 3, row = 32 * q + lane;
        // this thread's columns: 128 g .. + 127 in quarters, or 64 g .. + 63 of both parts in halves (parts in turn)
        auto column = [&](int i) { return GLU ? (i & 1) * kM + 64 * g + (i >> 1) * 32 : kM * g + 32 * i; };
        const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16);
        uint32_t it = 0, turn = 0, group = 0, record = 0;   // blocks, tiles, groups of scales, tiles' records
        bool ok = true;
        for (int t = t0; t < tiles && ok; t += t_step) {
            uint64_t acc[4][16];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 16; ++j) acc[i][j] = 0;
            if (MX) {
                ok = lane_wait(sums_ready, turn) && ok;
                tc_fence_after();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t u[32];
                    tmem_ld32(lanes + column(i), u);
#pragma unroll
                    for (int j = 0; j < 16; ++j) acc[i][j] = pack2(u[2 * j], u[2 * j + 1]);
                }
                tc_fence_before();                   // the buffer is free: it is in registers
                __syncwarp();
                if (lane == 0) mbar_arrive(tempty(0));
            } else {
            // Steps of 16 columns: while one is added up the next is on its way from tensor memory, over the end of a block, too.
            // Columns without weight rows are added up as well, nobody writes their sums: a test of them for every step
            // took a block to 1100 clocks.
            auto step_at = [&](int j) { return lanes + (it & 1) * kCols + column(j >> 1) + 16 * (j & 1); };
            uint32_t u[2][16];
            ok = lane_wait(done(it % ST), it / ST) && ok;
            tc_fence_after();
            tmem_ld16(step_at(0), u[0]);
            for (int kb = kb0; kb < kb1; ++kb) {
                const uint32_t slot = group % kSlots, four = kb & 3;
                if (!four) ok = lane_wait(sfull(slot), group / kSlots) && ok;
                const float *f = reinterpret_cast<const float *>(smem + oScale + slot * kSlotBytes), *fw = f + 4 * kRows + 2 * four;
                const float sx = f[four * kRows + row], f0 = sx * fw[GLU ? 0 : g], f1 = GLU ? sx * fw[1] : f0;
                if (four == 3 || kb + 1 == kb1) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sempty(slot));
                    ++group;
                }
                const uint64_t ff[2] = {pack2(__float_as_uint(f0), __float_as_uint(f0)), pack2(__float_as_uint(f1), __float_as_uint(f1))};
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    tmem_wait_ld();
                    pin16(u[j & 1]);
                    if (j < 7) {
                        tmem_ld16(step_at(j + 1), u[(j + 1) & 1]);
                    } else {
                        tc_fence_before();           // the buffer is free: it is in registers
                        __syncwarp();
                        if (lane == 0) mbar_arrive(tempty(it & 1));
                        ++it;
                        if (kb + 1 < kb1) {
                            ok = lane_wait(done(it % ST), it / ST) && ok;
                            tc_fence_after();
                            tmem_ld16(step_at(0), u[0]);
                        }
                    }
                    add16(&acc[j >> 1][8 * (j & 1)], u[j & 1], ff[j >> 1 & 1]);
                }
            }
            }
            ++turn;
            ok = __all_sync(0xFFFFFFFFu, ok) != 0;   // a warp's lanes leave together: what follows meets at barriers
            if (!ok) break;
            if (p.split > 1) {
                // this part's sums as [column][row]; the ring they overwrite is drained: a cluster has one tile
                float *part = reinterpret_cast<float *>(smem) + row;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        float x, y;
                        unpack2(acc[i][j], x, y);
                        part[(column(i) + 2 * j) * kRows] = x;
                        part[(column(i) + 2 * j + 1) * kRows] = y;
                    }
                break;
            }
            const int *tile = reinterpret_cast<const int *>(smem + oRecord + record * kRecordBytes);
            const int to = tile[row], m0 = tile[kRows];
            record = record + 1 == kRecords ? 0 : record + 1;
            if (GLU) {
                uint32_t *amax = reinterpret_cast<uint32_t *>(smem + oMax) + (turn & 1) * 2 * kRows + row;
                float big = 0.f;
#pragma unroll
                for (int i = 0; i < 4; i += 2)
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        float x0, y0, x1, y1;
                        unpack2(acc[i][j], x0, y0);
                        unpack2(acc[i + 1][j], x1, y1);
                        x0 = gated(x0, x1, a.limit);
                        y0 = gated(y0, y1, a.limit);
                        big = amax3(big, x0, y0);
                        acc[i][j] = pack2(__float_as_uint(x0), __float_as_uint(y0));
                    }
                amax[g * kRows] = __float_as_uint(big);
                __syncwarp();
                if (lane == 0) mbar_arrive(together);
                if (!(ok = wait(together, turn - 1))) break;   // the next tile's go to the other half
                const uint32_t byte = block_scale_byte(max(amax[0], amax[kRows]));
                const float inv = byte == 255u ? 0.f : inv_scale(byte);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int at = m0 + 64 * g + 32 * i;
                    if (to < 0 || at >= a.N) continue;
                    uint32_t c[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float x0, y0, x1, y1;
                        unpack2(acc[2 * i][2 * j], x0, y0);
                        unpack2(acc[2 * i][2 * j + 1], x1, y1);
                        c[j] = byte == 255u ? 0u : e4m3x4(x0 * inv, y0 * inv, x1 * inv, y1 * inv);
                    }
                    uint4 *o = reinterpret_cast<uint4 *>(static_cast<uint8_t *>(a.out) + (int64_t)to * a.N + at);
                    if (p.wide == 2) {               // n is a multiple of 32
                        st32(o, c);
                    } else {
                        o[0] = make_uint4(c[0], c[1], c[2], c[3]);
                        if (at + 16 < a.N) o[1] = make_uint4(c[4], c[5], c[6], c[7]);
                    }
                }
                if (g == 0 && to >= 0) {
                    const int64_t i = (int64_t)to * p.NB + m0 / kM;
                    if (a.out_type == ENGRAM_FMT_FP8_E8M0)
                        static_cast<uint8_t *>(a.out_scales)[i] = (uint8_t)byte;
                    else
                        static_cast<float *>(a.out_scales)[i] = e8m0_to_f32(byte);
                }
            } else if (to >= 0) {
                const int at = m0 + kM * g, left = a.N - at;
                const int64_t o = (int64_t)to * a.out_stride + at;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (a.out_type == ENGRAM_T_BF16)
                        store32<__nv_bfloat16>(a.out, o + 32 * i, acc[i], left - 32 * i, p.wide);
                    else if (a.out_type == ENGRAM_T_F16)
                        store32<__half>(a.out, o + 32 * i, acc[i], left - 32 * i, p.wide);
                    else
                        store32<float>(a.out, o + 32 * i, acc[i], left - 32 * i, p.wide);
                }
            }
        }
        __syncwarp();
        if (p.split > 1) {
            cluster_sync();
            auto all_meet = [&]() {
                __syncwarp();
                if (lane == 0) mbar_arrive(together);
                return wait(together, 0);
            };
            if (t0 < tiles && ok) {
                const TileAt w = tile_at(t0);
                const int i = threadIdx.x - 32 * kEpiWarp;
                if (p.split == 2)
                    share_of_tile<GLU, 2>(p, w, base, smem, rank, i, all_meet);
                else if (p.split == 4)
                    share_of_tile<GLU, 4>(p, w, base, smem, rank, i, all_meet);
                else
                    share_of_tile<GLU, 8>(p, w, base, smem, rank, i, all_meet);
            }
            cluster_sync();
        }
    }
    if (p.split > 1 && warp < kEpiWarp) {
        __syncwarp();
        cluster_sync();
        cluster_sync();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

template <bool GLU, bool MX, bool GATHER>
cudaError_t launch(Params &p, cudaStream_t s) {
    const ProductArgs &a = p.a;
    static Fit fits[64] = {};
    Fit fit;
    const cudaError_t e = fit_of(fits, product_rows_kernel<GLU, MX, GATHER>, threads_of(MX, GATHER), smem_bytes(kMaxExperts), &fit);
    if (e != cudaSuccess) return e;
    const uint64_t xd[2] = {(uint64_t)a.K, (uint64_t)a.rows}, xst[1] = {(uint64_t)a.x_stride};
    const uint32_t box[2] = {128, kRows};
    if (!make_map_u8(&p.mx, a.x, 2, xd, xst, box)) return cudaErrorInvalidValue;
    p.m_tiles = (a.N + (GLU ? kM : kCols) - 1) / (GLU ? kM : kCols);
    const int64_t tiles = (int64_t)product_row_tiles(a, kRows) * p.m_tiles;
    if (tiles > 0x3FFFFFFF) return cudaErrorInvalidConfiguration;
    p.split = fitting_split(fit, tiles, (p.KB + 3) / 4, true);
    // row tiles side by side whose rows stay in L2
    const int64_t rows_l2 = (int64_t(48) << 20) / a.K / kRows;
    p.group = (int)(rows_l2 < 8 ? 8 : rows_l2 > 0x3FFFFFFF ? 0x3FFFFFFF : rows_l2);
    return launch_split(product_rows_kernel<GLU, MX, GATHER>, p, tiles, threads_of(MX, GATHER), smem_bytes(a.E), s);
}

}  // namespace

cudaError_t launch_product_rows(product::Params &p, cudaStream_t s) {
    const bool mx = p.a.x_fmt == ENGRAM_FMT_FP8_E8M0 && p.a.w_fmt == ENGRAM_FMT_FP8_E8M0;
    if (!p.a.glu) return mx ? launch<false, true, false>(p, s) : launch<false, false, false>(p, s);
    if (!p.a.pairs) return mx ? launch<true, true, false>(p, s) : launch<true, false, false>(p, s);
    return mx ? launch<true, true, true>(p, s) : launch<true, false, true>(p, s);
}

}  // namespace engram
