// product.cu -- products of e4m3 rows with e4m3 weights that have a scale for each
// block of 128 (engram_project_fp8), and the gated pair of them with an 8-bit
// output (engram_glu_fp8), dense or with a matrix an expert: up to 24 rows (an expert, on
// average) here, more in product_rows.cu.
//
// out[r, n] = sum_b sx[r, b] sw[n / 128, b] sum_{k in block b} x[r, k] W[n, k].  The inner sum
// of 128 products is tcgen05.mma kind::f8f6f4 (products exact, f32 sums in tensor memory); the
// outer one is f32 FMAs in registers.  Weights are the M side of the MMA (two blocks of
// 128 rows: neighbours, or the gate's and the other's), up to 32 rows of x the N side, so that one token
// costs the tensor cores N = 16.
//
// Bound by the weights on their way from DRAM (five stages of 32 KB a CTA): 64 tokens, 8 of 256 experts, 4096 -> 2 x 2048:
// 403 us for 2.87 GB; the second product 212 us for 1.44 GB: the measured copy rate.  One token's eight experts, 134 MB, take 28 us (0.70 of it:
// 4 us are start and end; what holds the rest under the copy rate is not known); 4096 -> 6144 for one token, 25 MB, 9.5 us: 4.3 us is what one block of a
// single CTA takes, 2.2 more the exchange in a cluster.
//
// Roles (12 warps):
//   warp 0       TMA: a block's two 128 x 128 weight tiles, and its rows of x unless they are gathered
//                (one instruction each: issuing one takes a warp about 100 clocks);
//   warp 1       issues the MMAs;
//   warp 2       the factors sx sw of a block's rows, and where the tile's rows go, to shared memory;
//   warp 3       rows of x that the lists gather, by 16-byte asynchronous copies;
//   warps 4..11  take a block's sums from tensor memory (two buffers) into their f32
//                accumulators; at the end of a tile they write it.  A group of four warps has 16 of
//                the tile's rows.
// A CTA an SM walks the list of (expert, weight rows, rows) tiles; an expert's row tiles stand side by side, so
// that its weights are read from DRAM once.  Where there are fewer tiles than SMs, a cluster shares a tile: each CTA takes a part of K, and
// their sums are added in CTA order through distributed shared memory (no atomics, no workspace).
// Every wait is bounded (2 s); on expiry ENGRAM_E_TIMEOUT is raised, every role leaves its loops and
// tensor memory is freed.
#include "product.cuh"

namespace engram {

namespace {

using namespace product;


constexpr int kEpiWarp = 4;                          // first of the warps that take sums

constexpr int NT = 32;                               // rows of x a tile
constexpr int kGroups = 2, kEpiWarps = 4 * kGroups, kThreads = 32 * (kEpiWarp + kEpiWarps);
constexpr uint32_t kStage = 2 * kTileA + NT * 128;
constexpr int kStages = 5, kFactors = kStages + 2;   // slots of [2][NT] f32
// Tiles whose rows are known: factors may be kFactors + 1 tiles (of one block) ahead of the one that is written.
constexpr int kRowSlots = kFactors + 2;
constexpr uint32_t oFactor = kStages * kStage;
constexpr uint32_t oRows = oFactor + kFactors * 2 * NT * 4;    // [slots][NT] rows of the output
constexpr uint32_t oStage = oRows + kRowSlots * NT * 4;        // outputs: 512 bytes a warp (glu: [16][128] codes a group)
constexpr uint32_t oMax = oStage + kEpiWarps * 512;            // [groups][16][4] f32 bits
constexpr uint32_t oBar = oMax + kGroups * 16 * 4 * 4;
constexpr uint32_t oFlag = oBar + 8 * (2 * kStages + 2 * kFactors + 2 + 1 + kGroups);
constexpr uint32_t oLists = oFlag + 16;                        // first [E], rows [E], tiles before [E + 1]
constexpr size_t smem_bytes(int E) { return 1024 + oLists + (3 * (size_t)E + 1) * 4; }

template <bool GLU>
__global__ void __launch_bounds__(kThreads, 1) product_kernel(const __grid_constant__ Params p) {
    constexpr int ST = kStages, FS = kFactors, G = kGroups;
    extern __shared__ uint8_t smem_raw[];
    const ProductArgs &a = p.a;
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw);
    auto full = [&](int s) { return base + oBar + 8u * s; };
    auto done = [&](int s) { return base + oBar + 8u * (ST + s); };
    auto ffull = [&](int s) { return base + oBar + 8u * (2 * ST + s); };
    auto fempty = [&](int s) { return base + oBar + 8u * (2 * ST + FS + s); };
    auto tempty = [&](int b) { return base + oBar + 8u * (2 * ST + 2 * FS + b); };
    const uint32_t drain = base + oBar + 8u * (2 * ST + 2 * FS + 2);
    auto together = [&](int g) { return drain + 8u * (1 + g); };
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(smem + oFlag);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + oFlag + 4);
    int *first = reinterpret_cast<int *>(smem + oLists), *count = first + a.E, *before = count + a.E;
    constexpr uint32_t kCols = 4 * NT;               // two buffers of two blocks

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < ST; ++s) {
            mbar_init(full(s), GLU && a.pairs ? 2 : 1);
            mbar_init(done(s), 1);
        }
        for (int s = 0; s < FS; ++s) {
            mbar_init(ffull(s), 1);
            mbar_init(fempty(s), kEpiWarps);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tempty(b), kEpiWarps);
        }
        mbar_init(drain, 1);
        for (int g = 0; g < G; ++g) mbar_init(together(g), 4);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32((const void *)tmem_slot)), "r"(kCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    griddep_wait();
    griddep_launch();
    set_lists(a, first, count, before, NT, kThreads);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    const int rank = p.split > 1 ? (int)cluster_rank() : 0;
    const int t0 = blockIdx.x / p.split, t_step = gridDim.x / p.split;
    const int tiles = before[a.E] * p.m_tiles;
    const int kb0 = p.KB * rank / p.split, kb1 = p.KB * (rank + 1) / p.split;
    auto tile_at = [&](int t) { return tile_of(p, first, count, before, t, GLU ? kM : 2 * kM); };
    // whether the tile has a second block of weight rows
    auto two = [&](const TileAt &t) { return GLU || t.m0 + kM < a.N; };
    auto wait = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xFFFFFFFFu, warp_wait(bar, parity & 1, abort_flag, a.err)) != 0; };
    const bool gather = GLU && a.pairs;

    if (warp == 0) {
        // ---- weights, and rows that stand together ----
        uint32_t it = 0;
        bool ok = true;
        for (int t = t0; t < tiles && ok; t += t_step) {
            const TileAt w = tile_at(t);
            const bool few = w.n <= 16;
            const uint32_t bytes = 2 * kTileA + (gather ? 0u : few ? 16u * 128u : NT * 128u);
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int s = it % ST;
                if (!(ok = wait(done(s), it / ST ^ 1))) break;
                if (elect()) {
                    const uint32_t at = base + s * kStage, bar = full(s);
                    mbar_expect_tx(bar, bytes);
                    tma_weights(at, &p.mw, kb * 128, w.m0, 0, w.e, bar);
                    if (!gather) tma_rows(at + 2 * kTileA, few ? &p.mx16 : &p.mx, kb * 128, w.row, bar);
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
        uint32_t it = 0;
        bool ok = true;
        for (int t = t0; t < tiles && ok; t += t_step) {
            const TileAt w = tile_at(t);
            const bool both = two(w);
            const uint32_t idesc = idesc_f8((w.n + 15) & ~15);
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int s = it % ST, b = it & 1;
                if (!(ok = wait(tempty(b), it >> 1 ^ 1) && wait(full(s), it / ST))) break;
                tc_fence_after();
                const uint32_t at = base + s * kStage, d = tmem + b * 2 * NT;
                const uint64_t d0 = sdesc(at), d1 = sdesc(at + kTileA), db = sdesc(at + 2 * kTileA);
                if (elect()) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) mma_f8(d, d0 + 2u * k, db + 2u * k, idesc, k != 0);
                    if (both) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) mma_f8(d + NT, d1 + 2u * k, db + 2u * k, idesc, k != 0);
                    }
                    commit(done(s));
                }
                __syncwarp();
            }
        }
        // every MMA issued has finished before tensor memory can be freed
        if (elect()) commit(drain);
        __syncwarp();
        const uint64_t began = now_ns();
        while (!mbar_try(drain, 0) && now_ns() - began < 100000000ull) {
        }
        __syncwarp();
    } else if (warp == 2) {
        // ---- factors ----
        const bool vec_x = four_at_once(a.x_scales, a.x_fmt, p.KB);
        const bool vec_w = four_at_once(a.w_scales, a.w_fmt, p.KB);
        uint32_t it = 0, slot = 0;
        bool ok = true;
        for (int t = t0; t < tiles && ok; t += t_step, slot = slot + 1 == kRowSlots ? 0 : slot + 1) {
            const TileAt w = tile_at(t);
            const bool both = two(w);
            int *rows = reinterpret_cast<int *>(smem + oRows) + slot * NT;
            const int xi = lane < w.n ? gather ? token_of(a, w.row + lane) : w.row + lane : -1;
            rows[lane] = lane >= w.n ? -1 : GLU || !a.pairs ? w.row + lane : out_row_of(a, w.row + lane);
            const int64_t w0 = ((int64_t)w.e * (GLU ? 2 : 1) * p.NB + w.m0 / kM) * p.KB, w1 = w0 + (int64_t)(GLU ? p.NB : 1) * p.KB;
            // the next four blocks' scales are on their way while these are written
            uint4 next_x, next_w[2];
            auto fetch = [&](int kb4) {
                const int left = p.KB - kb4;
                if (xi >= 0) next_x = load_scales(a.x_scales, a.x_fmt, vec_x, (int64_t)xi * p.KB + kb4, left);
                next_w[0] = load_scales(a.w_scales, a.w_fmt, vec_w, w0 + kb4, left);
                if (both) next_w[1] = load_scales(a.w_scales, a.w_fmt, vec_w, w1 + kb4, left);
            };
            fetch(kb0 & ~3);
            for (int kb4 = kb0 & ~3; kb4 < kb1 && ok; kb4 += 4) {
                const uint4 x = next_x, s0 = next_w[0], s1 = both ? next_w[1] : s0;
                if (kb4 + 4 < kb1) fetch(kb4 + 4);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int kb = kb4 + j;
                    if (kb < kb0 || kb >= kb1 || !ok) continue;
                    const int s = it % FS;
                    if (!(ok = wait(fempty(s), it / FS ^ 1))) continue;
                    float *f = reinterpret_cast<float *>(smem + oFactor) + s * 2 * NT + lane;
                    const float g0 = scale_at(s0, a.w_fmt, vec_w, j), g1 = scale_at(s1, a.w_fmt, vec_w, j);
                    const float sx = xi >= 0 ? scale_at(x, a.x_fmt, vec_x, j) : 0.f;
                    f[0] = sx * g0;
                    f[NT] = sx * g1;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(ffull(s));
                    ++it;
                }
            }
        }
    } else if (warp == 3) {
        // ---- gathered rows: eight lanes a row of 128 bytes ----
        constexpr int LAG = 2;                       // blocks in flight behind the newest
        const int r0 = lane >> 3, chunk = lane & 7;
        uint32_t it = 0;
        bool ok = true;
        // the copies of block `done` have landed: its stage is full as far as this warp goes
        auto landed = [&](uint32_t done) {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(full(done % ST));
        };
        for (int t = t0; t < tiles && ok && gather; t += t_step) {
            const TileAt w = tile_at(t);
            uint32_t from[NT / 4];                    // rows r0, r0 + 4, ...: where they begin, in 16 bytes
#pragma unroll
            for (int i = 0; i < NT / 4; ++i)
                from[i] = r0 + 4 * i < w.n ? (uint32_t)(token_of(a, w.row + r0 + 4 * i) * (a.x_stride >> 4)) : 0u;
            const int n8 = (w.n + 7) / 8;
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int s = it % ST;
                if (!(ok = wait(done(s), it / ST ^ 1))) break;
                const bool real = kb * 128 + chunk * 16 < a.K;
                const uint8_t *src = a.x + (real ? kb * 128 + chunk * 16 : 0);
                // rows r0 and r0 + 4 of each 8: a chunk's place is turned by the row's last three bits
                const uint32_t at = base + s * kStage + 2 * kTileA + r0 * 128, lo = (chunk ^ r0) * 16, hi = (chunk ^ (r0 + 4)) * 16 + 512;
#pragma unroll
                for (int i = 0; i < NT / 8; ++i) {
                    if (i >= n8) break;
                    cp16(at + i * 1024 + lo, src + (uint64_t)from[2 * i] * 16, real);
                    cp16(at + i * 1024 + hi, src + (uint64_t)from[2 * i + 1] * 16, real);
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
                if (it >= LAG) {
                    cp_wait<LAG>();
                    landed(it - LAG);
                }
            }
        }
        cp_wait<0>();
        for (uint32_t done = it > LAG ? it - LAG : 0; ok && gather && done < it; ++done) landed(done);
        __syncwarp();
    } else {
        // ---- sums and output ----
        const int g = (warp - kEpiWarp) >> 2, q = warp & 3, m = 32 * q + lane, tw = threadIdx.x & 127;
        const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16);
        uint32_t it = 0, slot = 0, syncs = 0;
        // The group's four warps meet (a bounded wait, unlike bar.sync's).
        auto group_sync = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(together(g));
            return wait(together(g), syncs++);
        };
        // Writes rows c0 .. c0 + n - 1 of tile w, n <= 16: v0, v1 the sums of weight rows m of its two blocks.  False: a wait ran out.
        auto finish = [&](const TileAt &w, float (&v0)[16], float (&v1)[16], int c0, int n) {
            if (GLU) {
                uint32_t *amax = reinterpret_cast<uint32_t *>(smem + oMax) + g * 64;
                uint8_t *codes = smem + oStage + g * 2048;
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    v0[j] = gated(v0[j], v1[j], a.limit);
                    const uint32_t big = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(fabsf(v0[j])));
                    if (lane == j) amax[4 * j + q] = big;
                }
                if (!group_sync()) return false;
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
                if (!group_sync()) return false;
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
                return group_sync();                                // before the next chunk's
            } else {
                const int *rows = reinterpret_cast<const int *>(smem + oRows) + slot * NT + c0;
                const int col = w.m0 + m;
                if (a.out_type == ENGRAM_T_F32) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const int r = j < n ? rows[j] : -1;
                        float *o = static_cast<float *>(a.out) + (int64_t)r * a.out_stride + col;
                        if (r >= 0 && col < a.N) o[0] = v0[j];
                        if (r >= 0 && col + kM < a.N) o[kM] = v1[j];
                    }
                    return true;
                }
                // 16-bit: this warp's 32 weight rows of 8 rows of x through shared memory, 16 bytes a lane to global
                uint16_t *stage = reinterpret_cast<uint16_t *>(smem + oStage + (warp - kEpiWarp) * 512);
                const bool bf = a.out_type == ENGRAM_T_BF16;
                auto put = [&](const float (&v)[16], int first_col) {
                    const int at = (lane & 3) * 8, left = a.N - first_col - at;   // of this lane's eight columns
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        __syncwarp();
#pragma unroll
                        for (int j = 0; j < 8; j += 2) {
                            const uint32_t u = bf ? pack_bf16x2(v[8 * h + j], v[8 * h + j + 1]) : pack_f16x2(v[8 * h + j], v[8 * h + j + 1]);
                            stage[j * 32 + lane] = (uint16_t)u;
                            stage[j * 32 + 32 + lane] = (uint16_t)(u >> 16);
                        }
                        __syncwarp();
                        const int j = h * 8 + (lane >> 2);
                        const int r = j < n ? rows[j] : -1;
                        if (r < 0 || left <= 0) continue;
                        const uint4 x = *reinterpret_cast<const uint4 *>(stage + (lane >> 2) * 32 + at);
                        uint16_t *o = static_cast<uint16_t *>(a.out) + (int64_t)r * a.out_stride + first_col + at;
                        if (p.wide && left >= 8) {
                            *reinterpret_cast<uint4 *>(o) = x;
                        } else {
                            const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                if (k < left) o[k] = (uint16_t)(u[k >> 1] >> (16 * (k & 1)));
                        }
                    }
                };
                put(v0, w.m0 + 32 * q);
                put(v1, w.m0 + kM + 32 * q);
                return true;
            }
        };
        bool ok = true;
        for (int t = t0; t < tiles && ok; t += t_step, slot = slot + 1 == kRowSlots ? 0 : slot + 1) {
            const TileAt w = tile_at(t);
            const bool both = two(w);
            uint64_t acc0[8], acc1[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) acc0[j] = acc1[j] = 0;
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int b = it & 1, s = it % FS;
                if (!(ok = wait(ffull(s), it / FS) && wait(done(it % ST), it / ST))) break;
                tc_fence_after();
                const float *f = reinterpret_cast<const float *>(smem + oFactor) + s * 2 * NT;
                const uint32_t d = lanes + b * 2 * NT;
                // rows behind the tile's last are added up, too: nobody reads their sums
                if (g * 16 < w.n) {
                    uint32_t u[16];
                    tmem_ld16(d + g * 16, u);
                    tmem_wait_ld();
                    pin16(u);
                    add_chunk(acc0, u, f + g * 16);
                    if (both) {
                        tmem_ld16(d + NT + g * 16, u);
                        tmem_wait_ld();
                        pin16(u);
                        add_chunk(acc1, u, f + NT + g * 16);
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
            const int c0 = g * 16;
            if (c0 < w.n) {
                float v0[16], v1[16];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    unpack2(acc0[j], v0[2 * j], v0[2 * j + 1]);
                    unpack2(acc1[j], v1[2 * j], v1[2 * j + 1]);
                }
                if (p.split == 1) {
                    ok = finish(w, v0, v1, c0, min(16, w.n - c0));
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
                slot = 0;
                const int lo = w.n * rank / p.split, hi = w.n * (rank + 1) / p.split;
                for (int c0 = lo + 16 * g; c0 < hi && ok; c0 += 16 * G) {
                    float v0[16], v1[16];
                    const int n = min(16, hi - c0);
#pragma unroll
                    for (int j0 = 0; j0 < 16; j0 += 4) {
                        uint32_t at[8];
                        float v[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) at[j] = (uint32_t)((c0 + j0 + (j >> 1)) * 2 * kM + (j & 1) * kM + m) * 4;
                        if (j0 < n) sum_of_cluster(base, p.split, at, 2 * (n - j0), v);
#pragma unroll
                        for (int j = 0; j < 4; ++j) v0[j0 + j] = j0 < n ? v[2 * j] : 0.f, v1[j0 + j] = j0 < n ? v[2 * j + 1] : 0.f;
                    }
                    ok = finish(w, v0, v1, c0, n);
                }
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
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols) : "memory");
}

template <bool GLU>
cudaError_t launch_tile(Params &p, cudaStream_t s) {
    const ProductArgs &a = p.a;
    static Fit fits[64] = {};
    Fit fit;
    const cudaError_t e = fit_of(fits, product_kernel<GLU>, kThreads, smem_bytes(kMaxExperts), &fit);
    if (e != cudaSuccess) return e;
    const uint64_t xd[2] = {(uint64_t)a.K, (uint64_t)a.rows}, xst[1] = {(uint64_t)a.x_stride};
    const uint32_t box[2] = {128, NT}, box16[2] = {128, 16};
    if (!make_map_u8(&p.mx, a.x, 2, xd, xst, box) || !make_map_u8(&p.mx16, a.x, 2, xd, xst, box16)) return cudaErrorInvalidValue;
    p.m_tiles = (a.N + (GLU ? kM : 2 * kM) - 1) / (GLU ? kM : 2 * kM);
    const int64_t tiles = (int64_t)product_row_tiles(a, NT) * p.m_tiles;
    if (tiles > 0x3FFFFFFF) return cudaErrorInvalidConfiguration;
    p.split = fitting_split(fit, tiles, p.KB / 2, false);
    // row tiles of a dense product side by side whose rows stay in L2
    const int64_t rows_l2 = (int64_t(48) << 20) / a.K / NT;
    p.group = (int)(rows_l2 < 8 ? 8 : rows_l2 > 0x3FFFFFFF ? 0x3FFFFFFF : rows_l2);
    return launch_split(product_kernel<GLU>, p, tiles, kThreads, smem_bytes(a.E), s);
}

}  // namespace

cudaError_t launch_product(const ProductArgs &a, cudaStream_t s) {
    Params p;
    p.a = a;
    p.KB = (a.K + kScaleBlock - 1) / kScaleBlock;
    p.NB = (a.N + kScaleBlock - 1) / kScaleBlock;
    const uint64_t parts = a.glu ? 2 : 1, K = (uint64_t)a.K, N = (uint64_t)a.N;
    const uint64_t wd[4] = {K, N, parts, (uint64_t)a.E}, wst[3] = {K, N * K, parts * N * K};
    const uint32_t wbox[4] = {128, a.glu ? 128u : 256u, a.glu ? 2u : 1u, 1};
    if (!make_map_u8(&p.mw, a.w, 4, wd, wst, wbox)) return cudaErrorInvalidValue;
    const uint64_t row = (uint64_t)a.out_stride * (a.glu ? 1 : a.out_type == ENGRAM_T_F32 ? 4 : 2);
    const uint64_t either = row | reinterpret_cast<uintptr_t>(a.out);
    p.wide = either % 32 == 0 ? 2 : either % 16 == 0 ? 1 : 0;
    // rows (an expert, on average).  8 of 64 experts, 4096 -> 2 x 1024: at 16 rows 92 us here, 103 (weights' scales in 32 bits) or 91 with
    // tiles of 128 rows; at 32 rows 104 and 92; at 64, 125 (tiles of 64 rows here) and 103.
    const int rows = a.offsets ? (a.n_pairs + a.E - 1) / a.E : a.n_pairs;
    if (rows > 24) return launch_product_rows(p, s);
    return a.glu ? launch_tile<true>(p, s) : launch_tile<false>(p, s);
}

int product_row_tiles(const ProductArgs &a, int rows) {
    return a.offsets ? (a.n_pairs < a.E ? a.n_pairs : a.E) + a.n_pairs / rows : (a.n_pairs + rows - 1) / rows;
}

}  // namespace engram
