// attn_tile.cu -- causal attention over the paged 8-bit cache for more than 16
// query rows a key/value head (prompts, chunks, many query heads on one
// key/value head), on the 5th-generation tensor cores.
//
// Mathematics as in attention.cu: t_j = <q, kc_j> c + ev with the value scale in
// the exponent, p_j = 2^(t_j - M), out = sum p_j vc_j / sum p_j 2^-ev, M raised only
// when a t passes it by more than 8.
//
// A CTA works on up to 256 rows (two halves of 128: rows = new tokens x query
// heads of one key/value head) and 128 tokens a step, so a converted key or
// value tile serves both halves:
//   warps 0..3, 4..7   softmax of half 0 / 1, one thread a row: scores from tensor
//                      memory, probabilities back to tensor memory as f16, rescaling
//                      and the output;
//   warps 8..11        codes to f16 operand tiles in shared memory (e4m3 to f16 is exact);
//                      keys and values alike stay [token][dim]: values are the
//                      MN-major operand of the second product;
//   warps 12, 14       issue the MMAs of half 0 / 1 (M 128, N 128 / D, K 16): S_h = Q_h K^T,
//                      O_h += P_h V with P_h from tensor memory;
//   warp 13            pages, scales and TMA copies of the codes.
// While one half is in its softmax the tensor cores work for the other.  Tensor
// memory: S 2 x 128 columns, O 2 x D; P lies over its S for D = 128 (all 512 columns
// are taken), beside it for D = 64.
//
// The call's (sequence, head, row tile, 128-token tile) list is cut evenly
// over one CTA an SM; ranges that cut a row tile's tokens leave partial
// results that the last to arrive joins in CTA order.
// Every wait is bounded (2 s); on expiry ENGRAM_E_TIMEOUT is raised, the roles run
// out their loops without waiting, and tensor memory is freed.
#include "attn.cuh"

namespace engram {

namespace {

using namespace attn;
using namespace tcg;

constexpr int kHalf = 128;                           // rows of a half
constexpr int kRows = 2 * kHalf;
constexpr int kTok = 128;                            // tokens a step
constexpr int kThreads = 512;
constexpr int kGroups = kTok / 16;                   // scale groups a step (a page is at least 16 tokens)
constexpr int kMetaRing = 4;
constexpr uint32_t kNever = 0x7FFFFFFF;

struct TileParams {
    AttnArgs a;
    CUtensorMap mk, mv;
};

// Row tile rt of a sequence: its tokens from `lo`, in `tiles` tiles of 128.
struct RowTile {
    int r0, n_rows, lo, tiles;
};
__device__ __forceinline__ RowTile row_tile(const AttnArgs &a, const Seq &s, int rt) {
    RowTile t;
    t.r0 = rt * kRows;
    t.n_rows = min(kRows, s.n * a.group - t.r0);
    const int first = s.kv - s.n + t.r0 / a.group, last = s.kv - s.n + (t.r0 + t.n_rows - 1) / a.group;
    t.lo = a.window ? max(0, first - a.window + 1) / kTok * kTok : 0;
    t.tiles = max(1, (min(s.kv, last + 1) - t.lo + kTok - 1) / kTok);
    return t;
}
__device__ __forceinline__ int64_t head_tiles(const AttnArgs &a, const Seq &s) {
    int64_t n = 0;
    for (int rt = 0; rt < (s.n * a.group + kRows - 1) / kRows; ++rt) n += row_tile(a, s, rt).tiles;
    return n;
}

// This CTA's range of the list, entry by entry.  Every warp walks it by itself; the
// walk lies in shared memory (one a warp, stepped by its lane 0), so the roles'
// inner loops keep their registers.
struct Walk {
    int64_t t, end, per, entry_t0;
    Seq s;
    RowTile rt;
    int b, head, row_tile_no, tile0, count;

    // A whole warp calls this.
    __device__ __forceinline__ bool start(const AttnArgs &a) {
        const int lane = threadIdx.x & 31;
        const int lanes_per = (a.c.batch + 31) / 32;
        int64_t mine = 0;
        for (int j = 0; j < lanes_per; ++j) {
            const int i = lane * lanes_per + j;
            if (i < a.c.batch) mine += head_tiles(a, sequence(a.c, i)) * a.c.KH;
        }
        int64_t upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xFFFFFFFFu, upto, o);
            if (lane >= o) upto += x;
        }
        const int64_t total = __shfl_sync(0xFFFFFFFFu, upto, 31);
        const int64_t p = max((int64_t)1, (total + gridDim.x - 1) / gridDim.x), from = blockIdx.x * p;
        if (from >= total) return false;
        const int owner = __ffs(__ballot_sync(0xFFFFFFFFu, from < upto)) - 1;
        int64_t rel = from - __shfl_sync(0xFFFFFFFFu, upto - mine, owner);
        if (lane == 0) {
            b = owner * lanes_per;
            s = sequence(a.c, b);
            int64_t per_head = head_tiles(a, s);
            while (rel >= per_head * a.c.KH && b + 1 < a.c.batch) {
                rel -= per_head * a.c.KH;
                s = sequence(a.c, ++b);
                per_head = head_tiles(a, s);
            }
            head = (int)(rel / per_head);
            rel -= head * per_head;
            rt = row_tile(a, s, row_tile_no = 0);
            while (rel >= rt.tiles && rt.r0 + rt.n_rows < s.n * a.group) {
                rel -= rt.tiles;
                rt = row_tile(a, s, ++row_tile_no);
            }
            tile0 = (int)rel;
            t = from;
            end = min(total, from + p);
            per = p;
            count = 0;
        }
        return true;
    }
    // The next entry; `first` on the first call.  A whole warp calls this.
    __device__ __forceinline__ bool next(const AttnArgs &a, bool first) {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) {
            if (!first && t < end) {                  // the entry before ended with its row tile
                tile0 = 0;
                if (rt.r0 + rt.n_rows < s.n * a.group) {
                    rt = row_tile(a, s, ++row_tile_no);
                } else {
                    if (++head == a.c.KH) {
                        head = 0;
                        do {
                            if (b + 1 >= a.c.batch) {             // the arrays changed under the call
                                t = end;
                                break;
                            }
                            s = sequence(a.c, ++b);
                        } while (s.n == 0);
                    }
                    rt = row_tile(a, s, row_tile_no = 0);
                }
            }
            count = (int)min((int64_t)(rt.tiles - tile0), end - t);
            entry_t0 = t - tile0;
            t += count;
        }
        __syncwarp();
        return count > 0;
    }
};

template <int D>
struct Tile {
    static constexpr int kQ = kHalf * D * 2;         // bytes of a half's queries
    static constexpr int kF16 = kTok * D * 2;        // bytes of a converted tile
    static constexpr int kFp8 = kTok * D;            // bytes of a staged tile
    static constexpr int oQ = 0, oK = oQ + 2 * kQ, oV = oK + 2 * kF16, oS = oV + 2 * kF16, oAux = oS + 2 * kFp8;
    static constexpr int oWalk = 768;                // in aux, behind the scales, barriers and flags
    static constexpr size_t kSmem = 1024 + oAux + oWalk + 16 * sizeof(Walk);
    static_assert(kSmem <= 227 * 1024, "shared memory");
    static constexpr int kSub = kTok * 128;          // bytes of a 64-dim sub-tile (128 rows of 128 bytes)
    static constexpr int kPart = kRows * (D + 2);    // floats of a partial result
    static constexpr uint32_t cS = 0, cO = 256;      // tensor-memory columns
    static constexpr uint32_t cP = D == 128 ? 0 : 384, sP = D == 128 ? 128 : 64;
};

// Instruction descriptor, kind::f16 with f16 operands and an f32 accumulator;
// mn_b: the B operand is MN-major (bit 16).
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool mn_b) {
    return (1u << 4) | (mn_b ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// Shared-memory descriptors as two words: the upper one (8-row groups 1024 bytes
// apart, version 1, 128-byte swizzle) is the same for both operand layouts.  K-major:
// a row is 64 elements of K; MN-major: a row is 64 elements of the outer dimension,
// 8-row groups along K, the next 64 elements a sub-tile further (leading byte offset).
constexpr uint32_t kDescHi = (1024u >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lead_bytes) {
    return ((saddr >> 4) & 0x3FFFu) | (lead_bytes >> 4) << 16;
}
template <uint32_t IDESC>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
        "mov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n\t}"
        ::"r"(d), "r"(a_lo), "r"(b_lo), "r"(kDescHi), "r"(IDESC), "r"((uint32_t)accumulate)
        : "memory");
}
template <uint32_t IDESC>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t ta, uint32_t b_lo, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
        "mov.b64 db, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}"
        ::"r"(d), "r"(ta), "r"(b_lo), "r"(kDescHi), "r"(IDESC), "r"((uint32_t)accumulate)
        : "memory");
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect() {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
}
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_ld32_nowait(uint32_t taddr, float *r) {
    uint32_t *u = reinterpret_cast<uint32_t *>(r);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
          "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]),
          "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]),
          "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&u)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
          "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
// Two f32 at a time (the packed FMA and ADD of sm_100 and up), and the three-way maximum.
__device__ __forceinline__ uint64_t pack2(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
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
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&u)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};"
        ::"r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
          "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// One staged tile of codes to f16: [token][dim], 64-dim sub-tiles of 128-byte swizzled rows.  128 threads.
template <int D>
__device__ __forceinline__ void convert_tile(uint32_t src, uint32_t dst, int wt, bool values, int valid, const float4 *meta) {
    const int lane = wt & 31, w = wt >> 5;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {                // a warp: 8 tokens x 4 chunks of 16 codes a pass
        const int it = i * 4 + (lane >> 3);           // chunk index over (token group of 8, chunk)
        const int r = w * 32 + (it / (D / 16)) * 8 + (lane & 7), c = it % (D / 16);
        uint4 x = lds_v4(src + chunk_at<D>(r, c));
        if (values && (r >= valid || meta[r >> 4].w == 0.f)) x = make_uint4(0u, 0u, 0u, 0u);
        const uint32_t row = dst + (c >> 2) * Tile<D>::kSub + r * 128;
        const int k = 2 * c & 7;
        sts128(row + ((k ^ (r & 7)) << 4), e4m3_lo(x.x), e4m3_hi(x.x), e4m3_lo(x.y), e4m3_hi(x.y));
        sts128(row + (((k + 1) ^ (r & 7)) << 4), e4m3_lo(x.z), e4m3_hi(x.z), e4m3_lo(x.w), e4m3_hi(x.w));
    }
}

template <int TYPE, int D>
__global__ void __launch_bounds__(kThreads, 1) attn_tile_kernel(const __grid_constant__ TileParams p) {
    using T = Tile<D>;
    extern __shared__ uint8_t smem_raw[];
    const AttnArgs &a = p.a;
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t *aux = smem_raw + (base - raw) + T::oAux;
    float4 *meta = reinterpret_cast<float4 *>(aux);                       // [kMetaRing][kGroups]: 2^ek, ev, 2^-ev, counts
    const uint32_t bar0 = smem_u32(aux + kMetaRing * kGroups * 16);
    enum { Q_FULL = 0, ST_FULL = 2, ST_EMPTY = 4, K_FULL = 6, K_EMPTY = 8, V_FULL = 10, V_EMPTY = 12, S_FULL = 14, P_FULL = 16,
           PV_DONE = 18, DRAIN = 20, BARS = 22 };
    auto bar = [&](int i) { return bar0 + 8u * i; };
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(aux + kMetaRing * kGroups * 16 + BARS * 8);
    int *flags = reinterpret_cast<int *>(aux + kMetaRing * kGroups * 16 + BARS * 8 + 8);
    volatile int *abort_flag = flags;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(Q_FULL + i), kHalf);
            mbar_init(bar(ST_FULL + i), 1);
            mbar_init(bar(ST_EMPTY + i), 128);
            mbar_init(bar(K_FULL + i), 128);
            mbar_init(bar(K_EMPTY + i), 2);               // both halves' products
            mbar_init(bar(V_FULL + i), 128);
            mbar_init(bar(V_EMPTY + i), 2);
            mbar_init(bar(S_FULL + i), 1);
            mbar_init(bar(P_FULL + i), kHalf);
            mbar_init(bar(PV_DONE + i), 1);
            mbar_init(bar(DRAIN + i), 1);
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_smem();
    }
    if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32((const void *)tmem_slot)), "r"(512u) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    int *err = a.c.err;
    Walk &e = reinterpret_cast<Walk *>(aux + T::oWalk)[warp];

    // 512 threads launch with 128 registers each: 2 x 128 x 176 + 128 x 88 + 128 x 72 are as many
    if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == 13) {
            // ---- pages, scales, copies ----
            bool ok = e.start(a);
            int it = 0;
            for (bool first = true; ok && e.next(a, first); first = false) {
                const int tok0 = e.rt.lo + e.tile0 * kTok;
                const int at = 16 * (lane & 7);
                const bool leader = lane < 8 && (at & (a.c.pt - 1)) == 0;
                auto page_at = [&](int j) {
                    const int tok = tok0 + j * kTok + at;
                    return lane < 8 && j < e.count && tok < e.s.kv ? page_of(a.c, e.b, tok >> a.c.pt_log2) : -1;
                };
                auto scales_of = [&](int id) {
                    if (id < 0) return 0u;
                    const int64_t i = (int64_t)id * a.c.KH + e.head;
                    return (uint32_t)a.c.k_scales[i] | (uint32_t)a.c.v_scales[i] << 8;
                };
                int id = page_at(0), id1 = page_at(1);
                uint32_t sc = scales_of(id);
                for (int j = 0; j < e.count && ok; ++j, ++it) {
                    const int id2 = page_at(j + 2);
                    const uint32_t sc1 = scales_of(id1);
                    const int page = id < 0 ? a.c.n_pages : id;           // outside the cache: zeros
                    ok = wait_bar(bar(ST_EMPTY + 0), (it & 1) ^ 1, abort_flag, err);
                    if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
                    if (lane < 8)
                        meta[(it % kMetaRing) * kGroups + lane] =
                            id < 0 ? make_float4(1.f, -INFINITY, 0.f, 0.f)
                                   : make_float4(e8m0_to_f32(sc & 255u), value_exp(sc >> 8), value_unscale(sc >> 8),
                                                 (int)(sc >> 8) < kLeastValueByte ? 0.f : 1.f);
                    __syncwarp();
                    if (lane == 0) mbar_expect_tx(bar(ST_FULL + 0), T::kFp8);
                    __syncwarp();
                    if (leader) tma_load_4d(base + T::oS + at * D, &p.mk, 0, (tok0 + at) & (a.c.pt - 1), e.head, page, bar(ST_FULL + 0));
                    ok = wait_bar(bar(ST_EMPTY + 1), (it & 1) ^ 1, abort_flag, err);
                    if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
                    if (lane == 0) mbar_expect_tx(bar(ST_FULL + 1), T::kFp8);
                    __syncwarp();
                    if (leader) tma_load_4d(base + T::oS + T::kFp8 + at * D, &p.mv, 0, (tok0 + at) & (a.c.pt - 1), e.head, page, bar(ST_FULL + 1));
                    id = id1;
                    sc = sc1;
                    id1 = id2;
                }
            }
            // every copy issued has landed before the CTA can leave (only an abort leaves one behind)
            const uint64_t t0 = now_ns();
            for (int i = 0; i < 2; ++i)
                while (it > 0 && !mbar_try(bar(ST_FULL + i), (it - 1) & 1) && now_ns() - t0 < 10000000ull) {
                }
        } else if (warp != 15) {
            // ---- the tensor cores: warp 12 for half 0, warp 14 for half 1 ----
            const int h = (warp - 12) >> 1;
            bool ok = e.start(a);
            uint32_t n = 0, nh = 0, ent = 0;                              // steps, steps with rows in this half, such entries
            const uint32_t q_lo = desc_lo(base + T::oQ + h * T::kQ, 16);
            const uint32_t tS = tmem + T::cS + h * 128, tO = tmem + T::cO + h * D, tP = tmem + T::cP + h * T::sP;
            for (bool first = true; ok && e.next(a, first); first = false) {
                const int count = e.count;
                const bool both = e.rt.n_rows > kHalf;
                if (h && !both) {
                    // no rows in this half: keep step with the converted tiles (their barriers count both halves)
                    for (int j = 0; j < count && ok; ++j, ++n) {
                        ok = __all_sync(0xFFFFFFFFu, wait_bar(bar(K_FULL + (n & 1)), (n >> 1) & 1, abort_flag, err));
                        if (ok && lane == 0) mbar_arrive(bar(K_EMPTY + (n & 1)));
                        ok = ok && __all_sync(0xFFFFFFFFu, wait_bar(bar(V_FULL + (n & 1)), (n >> 1) & 1, abort_flag, err));
                        if (ok && lane == 0) mbar_arrive(bar(V_EMPTY + (n & 1)));
                    }
                    continue;
                }
                ok = __all_sync(0xFFFFFFFFu, wait_bar(bar(Q_FULL + h), ent++ & 1, abort_flag, err));
                for (int j = 0; j < count && ok; ++j, ++n, ++nh) {
                    // scores: over this half's last probabilities (D = 128), so their product has to be done
                    ok = wait_bar(bar(K_FULL + (n & 1)), (n >> 1) & 1, abort_flag, err) &&
                         (D == 64 || j == 0 || wait_bar(bar(PV_DONE + h), (nh - 1) & 1, abort_flag, err));
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect()) {
                        const uint32_t k_lo = desc_lo(base + T::oK + (n & 1) * T::kF16, 16);
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t off = ((kk >> 2) * T::kSub + (kk & 3) * 32) >> 4;
                            mma_ss<idesc_f16(kHalf, kTok, false)>(tS, q_lo + off, k_lo + off, kk != 0);
                        }
                        commit(bar(S_FULL + h));
                        commit(bar(K_EMPTY + (n & 1)));
                    }
                    __syncwarp();
                    ok = wait_bar(bar(V_FULL + (n & 1)), (n >> 1) & 1, abort_flag, err) &&
                         wait_bar(bar(P_FULL + h), nh & 1, abort_flag, err);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect()) {
                        const uint32_t v_lo = desc_lo(base + T::oV + (n & 1) * T::kF16, T::kSub);
                        mma_ts<idesc_f16(kHalf, D, true)>(tO, tP, v_lo, j != 0);
#pragma unroll
                        for (int kk = 1; kk < kTok / 16; ++kk)
                            mma_ts<idesc_f16(kHalf, D, true)>(tO, tP + kk * 8, v_lo + kk * (2048 >> 4), true);
                        commit(bar(PV_DONE + h));
                        commit(bar(V_EMPTY + (n & 1)));
                    }
                    __syncwarp();
                }
            }
            if (elect()) commit(bar(DRAIN + h));                          // from the lane that issued the MMAs
            const uint64_t t0 = now_ns();
            while (!mbar_try(bar(DRAIN + h), 0) && now_ns() - t0 < 100000000ull) {
            }
            __syncwarp();
        }
    } else if (warp >= 8) {
        // ---- codes to f16 ----
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        const int wt = threadIdx.x - 256;
        bool ok = e.start(a);
        uint32_t n = 0;
        for (bool first = true; ok && e.next(a, first); first = false) {
            const int left = e.s.kv - (e.rt.lo + e.tile0 * kTok), count = e.count;
            for (int j = 0; j < count; ++j, ++n) {
                const int valid = left - j * kTok;                        // tokens of the tile that exist
                for (int x = 0; x < 2 && ok; ++x) {
                    ok = wait_bar(bar(ST_FULL + x), n & 1, abort_flag, err) &&
                         wait_bar(bar((x ? V_EMPTY : K_EMPTY) + (n & 1)), ((n >> 1) & 1) ^ 1, abort_flag, err);
                    if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
                    convert_tile<D>(base + T::oS + x * T::kFp8, base + (x ? T::oV : T::oK) + (n & 1) * T::kF16, wt, x != 0, valid,
                                    meta + (n % kMetaRing) * kGroups);
                    fence_async_smem();
                    mbar_arrive(bar(ST_EMPTY + x));
                    mbar_arrive(bar((x ? V_FULL : K_FULL) + (n & 1)));
                }
                if (!ok) break;
            }
        }
    } else {
        // ---- softmax, one thread a row ----
        asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
        const int h = warp >> 2, row = (warp & 3) * 32 + lane;            // row of the half = tensor-memory lane
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t tS = lanes + T::cS + h * 128, tO = lanes + T::cO + h * D, tP = lanes + T::cP + h * T::sP;
        bool ok = true;
        uint32_t n = 0, nh = 0;
        const bool some = e.start(a);
        for (bool first = true; some && e.next(a, first); first = false) {
            const int count = e.count, tok0 = e.rt.lo + e.tile0 * kTok;
            if (h * kHalf >= e.rt.n_rows) {                               // no rows in this half
                n += count;
                continue;
            }
            const int rr = e.rt.r0 + h * kHalf + row;
            const bool live = h * kHalf + row < e.rt.n_rows;
            const int tok_i = rr / a.group, pos = e.s.kv - e.s.n + tok_i;
            const int lim = live ? pos + 1 : (int)kNever, low = live && a.window ? pos - a.window + 1 : 0;
            float kf;
            {
                const int64_t at = (int64_t)(e.s.row0 + tok_i) * a.q_stride + (int64_t)(e.head * a.group + rr % a.group) * D;
                uint32_t m = 0, w[D / 2];
                const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q) + at);
#pragma unroll
                for (int c = 0; c < D / 8; ++c) {
                    const uint4 x = live ? src[c] : make_uint4(0u, 0u, 0u, 0u);
                    w[4 * c] = x.x, w[4 * c + 1] = x.y, w[4 * c + 2] = x.z, w[4 * c + 3] = x.w;
                }
                auto pair = [&](uint32_t u) {
                    return TYPE == ENGRAM_T_BF16 ? make_float2(bf16_lo(u), bf16_hi(u)) : __half22float2(*reinterpret_cast<__half2 *>(&u));
                };
#pragma unroll
                for (int i = 0; i < D / 2; ++i) {
                    const float2 f = pair(w[i]);
                    m = max(m, max(__float_as_uint(f.x) & 0x7FFFFFFFu, __float_as_uint(f.y) & 0x7FFFFFFFu));
                }
                float down;
                q_scale(m, a.scale_log2, down, kf);
                const uint32_t dst = base + T::oQ + h * T::kQ + row * 128;
#pragma unroll
                for (int c = 0; c < D / 8; ++c) {
                    uint32_t o[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 f = pair(w[4 * c + i]);
                        o[i] = pack_f16x2(f.x * down, f.y * down);
                    }
                    sts128(dst + (c >> 3) * T::kSub + (((c & 7) ^ (row & 7)) << 4), o[0], o[1], o[2], o[3]);
                }
            }
            fence_async_smem();
            mbar_arrive(bar(Q_FULL + h));

            float M = -INFINITY, L = 0.f;
            for (int j = 0; j < count; ++j, ++n, ++nh) {
                const int tb = tok0 + j * kTok;
                const bool got = ok && wait_bar(bar(S_FULL + h), nh & 1, abort_flag, err);
                ok = __all_sync(0xFFFFFFFFu, got);
                if (!ok) continue;
                tc_fence_after();
                float t[128];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32_nowait(tS + 32 * c, t + 32 * c);
                const float4 *mt = meta + (n % kMetaRing) * kGroups;
                tmem_wait_ld();
                // u_j = t_j - M with the bound so far; what passes it by more than 8 raises the bound
                const float m0 = M == -INFINITY ? 0.f : M;
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    const float4 f = mt[g];
                    const uint64_t c2 = pack2(kf * f.x, kf * f.x), e2 = pack2(f.y - m0, f.y - m0);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float &x = t[16 * g + 2 * i], &y = t[16 * g + 2 * i + 1];
                        unpack2(fma2(pack2(x, y), c2, e2), x, y);
                    }
                }
                if (__any_sync(0xFFFFFFFFu, tb + kTok > lim || tb < low)) {
#pragma unroll
                    for (int i = 0; i < 128; ++i)
                        if (tb + i >= lim || tb + i < low) t[i] = -INFINITY;
                }
#pragma unroll
                for (int i = 0; i < 64; ++i) mx[i & 3] = max3(mx[i & 3], t[2 * i], t[2 * i + 1]);
                const float tmax = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                if (__any_sync(0xFFFFFFFFu, tmax > (M == -INFINITY ? -INFINITY : kLazy))) {
                    const float m2 = fmaxf(M, m0 + tmax), f = M == m2 ? 1.f : exp2_approx(M - m2);
                    if (m2 != -INFINITY) {
                        const float d = m0 - m2;
#pragma unroll
                        for (int i = 0; i < 128; ++i) t[i] += d;
                    }
                    M = m2;
                    L *= f;
                    if (j > 0) {
                        const bool done = wait_bar(bar(PV_DONE + h), (nh - 1) & 1, abort_flag, err);
                        ok = __all_sync(0xFFFFFFFFu, done);
                        if (!ok) continue;
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < D; c += 16) {
                            uint32_t o[16];
                            tmem_ld16(tO + c, o);
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tmem_st16(tO + c, o);
                        }
                    }
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t u[16];
                    uint64_t sum[2][2] = {};
#pragma unroll
                    for (int i = 0; i < 8; ++i)
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            const float x = exp2_approx(t[32 * c + 16 * g + 2 * i]), y = exp2_approx(t[32 * c + 16 * g + 2 * i + 1]);
                            sum[g][i & 1] = add2(sum[g][i & 1], pack2(x, y));
                            u[8 * g + i] = pack_f16x2(x, y);
                        }
                    tmem_st16(tP + 16 * c, u);
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        float x, y;
                        unpack2(add2(sum[g][0], sum[g][1]), x, y);
                        L = fmaf(x + y, mt[2 * c + g].z, L);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(bar(P_FULL + h));
            }

            // the entry's result, or a part of it
            if (ok) {
                const bool done = wait_bar(bar(PV_DONE + h), (nh - 1) & 1, abort_flag, err);
                ok = __all_sync(0xFFFFFFFFu, done);
                tc_fence_after();
            }
            const int64_t first_cta = e.entry_t0 / e.per, last_cta = (e.entry_t0 + e.rt.tiles - 1) / e.per;
            const bool alone = first_cta == last_cta;
            const int64_t out_at = (int64_t)(e.s.row0 + tok_i) * a.out_stride + (int64_t)(e.head * a.group + rr % a.group) * D;
            const float inv = L == 0.f ? 0.f : 1.f / L;
            auto put = [&](int c, const float *x, float f) {              // 16 values from dim c
                if (!live) return;
                uint32_t w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    w[i] = TYPE == ENGRAM_T_BF16 ? pack_bf16x2(x[2 * i] * f, x[2 * i + 1] * f) : pack_f16x2(x[2 * i] * f, x[2 * i + 1] * f);
                uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + out_at + c);
                dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
                dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
            };
            auto put_lse = [&](float m, float l) {
                if (live && a.lse)
                    a.lse[(int64_t)(e.s.row0 + tok_i) * a.H + e.head * a.group + rr % a.group] =
                        l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
            };
            const int64_t slot = (int64_t)blockIdx.x * 2 + (blockIdx.x == first_cta ? 1 : 0);
            // partial results are column-major: float4 d4 of row r at [d4][r]
            float4 *part = reinterpret_cast<float4 *>(a.ws.part + slot * T::kPart) + h * kHalf + row;
            float *stat = a.ws.part + slot * T::kPart + kRows * D + h * kHalf + row;
            if (ok) {
#pragma unroll 1
                for (int c = 0; c < D; c += 16) {
                    uint32_t o[16];
                    tmem_ld16(tO + c, o);
                    float x[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(o[i]);
                    if (alone) {
                        put(c, x, inv);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) part[(c / 4 + i) * kRows] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                    }
                }
                if (alone) put_lse(M, L);
                else stat[0] = M, stat[kRows] = L;
            }
            tc_fence_before();                                            // the sums are read: the next entry may overwrite them
            if (!alone) {
                __threadfence();
                asm volatile("bar.sync %0, 128;" ::"r"(1 + h) : "memory");
                if ((threadIdx.x & 127) == 0) {
                    int *arrived = a.ws.arrived + first_cta * 2 + h;
                    const bool last = atomicAdd(arrived, 1) == (int)(last_cta - first_cta);
                    if (last) *arrived = 0;
                    flags[1 + h] = last;
                    __threadfence();
                }
                asm volatile("bar.sync %0, 128;" ::"r"(1 + h) : "memory");
                if (flags[1 + h]) {
                    const float *st = a.ws.part + kRows * D + h * kHalf + row;
                    const int parts = (int)(last_cta - first_cta) + 1;
                    auto at = [&](int c) { return ((first_cta + c) * 2 + (c == 0 ? 1 : 0)) * T::kPart; };
                    float m = -INFINITY, l = 0.f;
                    for (int c = 0; c < parts; ++c) m = fmaxf(m, __ldcg(st + at(c)));
                    auto factor = [&](int c) {
                        const float mc = __ldcg(st + at(c));
                        return mc == -INFINITY ? (__ldcg(st + at(c) + kRows) == 0.f ? 0.f : 1.f) : exp2_approx(mc - m);
                    };
                    for (int c = 0; c < parts; ++c) l = fmaf(__ldcg(st + at(c) + kRows), factor(c), l);
                    const float il = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
                    for (int d = 0; d < D; d += 64) {                     // 16 float4 in flight
                        float x[64] = {};
#pragma unroll 1
                        for (int c = 0; c < parts; ++c) {
                            const float f = factor(c);
                            const float4 *src = reinterpret_cast<const float4 *>(a.ws.part + at(c)) + (d / 4) * kRows + h * kHalf + row;
                            float4 v[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) v[i] = __ldcg(src + i * kRows);
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                x[4 * i] = fmaf(v[i].x, f, x[4 * i]), x[4 * i + 1] = fmaf(v[i].y, f, x[4 * i + 1]);
                                x[4 * i + 2] = fmaf(v[i].z, f, x[4 * i + 2]), x[4 * i + 3] = fmaf(v[i].w, f, x[4 * i + 3]);
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) put(d + 16 * i, x + 16 * i, il);
                    }
                    put_lse(m, l);
                }
                asm volatile("bar.sync %0, 128;" ::"r"(1 + h) : "memory");   // flags[1 + h] is read
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 12)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

template <int TYPE, int D>
cudaError_t launch_typed(const AttnArgs &a, cudaStream_t s) {
    TileParams p;
    p.a = a;
    const int box = a.c.pt < kTok ? a.c.pt : kTok;
    if (!make_cache_map(&p.mk, a.c, a.c.k, box) || !make_cache_map(&p.mv, a.c, a.c.v, box)) return cudaErrorInvalidValue;
    int dev = 0;
    cudaGetDevice(&dev);
    static bool attr[64] = {};
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(attn_tile_kernel<TYPE, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)Tile<D>::kSmem);
        if (e != cudaSuccess) return e;
        attr[dev] = true;
    }
    attn_tile_kernel<TYPE, D><<<a.sms, kThreads, Tile<D>::kSmem, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

size_t attn_tile_part_floats(int sms) { return (size_t)sms * 2 * Tile<128>::kPart; }
size_t attn_tile_counters(int sms) { return (size_t)sms * 2; }

cudaError_t launch_attn_tile(const AttnArgs &a, cudaStream_t s) {
    const bool bf = a.type == ENGRAM_T_BF16;
    if (a.c.D == 128) return bf ? launch_typed<ENGRAM_T_BF16, 128>(a, s) : launch_typed<ENGRAM_T_F16, 128>(a, s);
    return bf ? launch_typed<ENGRAM_T_BF16, 64>(a, s) : launch_typed<ENGRAM_T_F16, 64>(a, s);
}

}  // namespace engram
