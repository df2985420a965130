// attn_tile.cu -- causal attention over the paged 8-bit cache for more than 16
// query rows a key/value head (prompts, chunks, many query heads on one
// key/value head), on the 5th-generation tensor cores.
//
// Mathematics as in attention.cu: t_j = <q, kc_j> c + ev with the value scale in
// the exponent, p_j = 2^(t_j - M), out = sum p_j vc_j / sum p_j 2^-ev, M (4 under the
// row's largest t when it is set) raised only when 16 p of one page add up to more than f16 holds.
//
// A CTA works on up to 256 rows (two halves of 128: rows = new tokens x query
// heads of one key/value head) and 128 tokens a step, so a converted key or
// value tile serves both halves:
//   warps 0..3, 4..7   softmax of half 0 / 1, one thread a row: scores from tensor
//                      memory, probabilities back to tensor memory as f16, rescaling and
//                      the output;
//   warps 8..11        codes to f16 operand tiles in shared memory (e4m3 to f16 is exact);
//                      keys and values alike stay [token][dim]: values are the
//                      MN-major operand of the second product;
//   warps 12, 14       issue the first product of half 0 / 1, S_h = Q_h K^T for 64 tokens at
//                      a time (M 128, N 64, K 16);
//   warps 16, 17       issue the second, O_h += P_h V with P_h from tensor memory (M 128, N D, K 16);
//   warp 13            pages, scales and TMA copies of the codes;
//   warp 15            the schedule: entries of the list for all others.
// A half's scores have two buffers of 64 tokens: while one is in its softmax, the
// tensor cores fill the other and take the probabilities before (with one buffer a
// half they were idle for the latencies between product, softmax and product: 432
// against 379 us).  Tensor memory: S 2 x 2 x 64 columns, O 2 x D; P lies over its S.
//
// Bound by latency between the roles: the longest is the softmax, two in-order warps a
// scheduler and about 1000 clocks for 64 tokens of both beside the converters, against 512 of
// tensor work a half, but no pipe is busy for more than 57 % of the time.  4096 tokens
// behind 4096, 32 query and 8 key/value heads of 128 (412 GFLOP in the visible pairs):
// 320 us, 69 % of the measured bf16 rate; an entry costs about 5 us in which the
// tensor cores wait (output, queries, first scores).  Times below are this call's, those of
// steps before kRoom with a bound at the row's largest score (11 us less).
//
// The call's (sequence, head, row tile, 128-token tile) list, with kEntryCost places more
// for each row tile (what beginning and ending one takes), is cut evenly over one CTA an
// SM; ranges that cut a row tile's tokens leave partial
// results that the last to arrive joins in CTA order.
// Every wait is bounded (2 s); on expiry ENGRAM_E_TIMEOUT is raised, every role leaves
// its loops (all waits are on mbarriers, and a warp votes before it branches on one)
// and tensor memory is freed.
#include "attn.cuh"

namespace engram {

namespace {

using namespace attn;
using namespace tcg;

constexpr int kHalf = 128;                           // rows of a half
constexpr int kRows = 2 * kHalf;
constexpr int kTok = 128, kPartTok = 64;             // tokens a step, and a score buffer
// Places of a row tile beside its tiles: 8 x 512 tokens behind 512 took 78 us, with 3 or 6 81, with 5 80 (81 with kRoom).
constexpr int kEntryCost = 4;
constexpr int kThreads = 640, kSoftWarps = 8;
constexpr int kGroups = kTok / 16;                   // scale groups a step (a page is at least 16 tokens)
constexpr int kMetaRing = 4;
// A row's bound M is set kRoom (log2) under its largest t so far, and 16 probabilities may add up to kLazySum, f16's
// largest number: one 2^-29 of the row's largest is still half of f16's least.  More room loses fewer of the small ones and
// rescales more often: 0 takes 306 us, 2 311, 4 319, 5 326; 7 with sums to 2^15 349.
constexpr float kRoom = 4.f, kLazySum = 65504.f;

struct TileParams {
    AttnArgs a;
    CUtensorMap mk, mv;
};

// x / group.
__device__ __forceinline__ int by_group(const AttnArgs &a, int x) { return a.group_log2 >= 0 ? x >> a.group_log2 : x / a.group; }

// Row tile rt of a sequence: its tokens from `lo`, in `tiles` tiles of 128; its rows see tokens from `first` on.
struct RowTile {
    int r0, n_rows, first, lo, tiles;
};
__device__ __forceinline__ RowTile row_tile(const AttnArgs &a, const Seq &s, int rt) {
    RowTile t;
    t.r0 = rt * kRows;
    t.n_rows = min(kRows, s.n * a.group - t.r0);
    const int first = s.kv - s.n + by_group(a, t.r0), last = s.kv - s.n + by_group(a, t.r0 + t.n_rows - 1);
    t.first = a.window ? max(0, first - a.window + 1) : 0;
    t.lo = t.first / kTok * kTok;
    t.tiles = max(1, (min(s.kv, last + 1) - t.lo + kTok - 1) / kTok);
    return t;
}
__device__ __forceinline__ int row_tiles(const AttnArgs &a, const Seq &s) { return (s.n * a.group + kRows - 1) / kRows; }
__device__ __forceinline__ int64_t warp_sum(int64_t v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
// Sum of v over lanes up to this one.
__device__ __forceinline__ int64_t warp_scan(int64_t v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if ((threadIdx.x & 31) >= o) v += x;
    }
    return v;
}
// Places of one head of sequence s in the list: by one lane, or by a whole warp.
__device__ __forceinline__ int64_t head_places(const AttnArgs &a, const Seq &s) {
    int64_t n = 0;
    for (int rt = 0; rt < row_tiles(a, s); ++rt) n += row_tile(a, s, rt).tiles + kEntryCost;
    return n;
}
__device__ __forceinline__ int64_t head_places_warp(const AttnArgs &a, const Seq &s) {
    int64_t n = 0;
    for (int rt = threadIdx.x & 31; rt < row_tiles(a, s); rt += 32) n += row_tile(a, s, rt).tiles + kEntryCost;
    return warp_sum(n);
}

// An entry of this CTA's range of the list.
struct Entry {
    Seq s;
    RowTile rt;
    int b, head, tile0, count;                       // count 0: no more
    int first_cta, last_cta;                         // those that share the row tile
};
constexpr int kEntries = 4, kEntryUsers = kSoftWarps + 4 + 5;

// This CTA's range, walked by one warp; all of its lanes hold the same.
struct Walk {
    int64_t t, end, per, t0;
    Entry e;
    int row_tile_no;

    __device__ __forceinline__ bool start(const AttnArgs &a) {
        const int lane = threadIdx.x & 31;
        // the sequence that holds this CTA's first tile: a lane on each sequence, or, where a few sequences
        // have many row tiles (about 600 clocks a sequence against 60 a row tile), the warp on each one's row tiles
        const bool few = a.c.batch <= 32 && 10ll * a.c.batch < ((int64_t)a.c.max_rows * a.group + kRows - 1) / kRows;
        const int lanes_per = (a.c.batch + 31) / 32;
        int64_t mine = 0;
        if (few) {
            const Seq q = lane < a.c.batch ? sequence(a.c, lane) : Seq{0, 0, 0};
            for (int i = 0; i < a.c.batch; ++i) {
                const Seq at = {0, __shfl_sync(0xFFFFFFFFu, q.n, i), __shfl_sync(0xFFFFFFFFu, q.kv, i)};
                const int64_t n = head_places_warp(a, at) * a.c.KH;
                if (lane == i) mine = n;
            }
        } else {
            for (int j = 0; j < lanes_per; ++j) {
                const int i = lane * lanes_per + j;
                if (i < a.c.batch) mine += head_places(a, sequence(a.c, i)) * a.c.KH;
            }
        }
        const int64_t upto = warp_scan(mine), total = __shfl_sync(0xFFFFFFFFu, upto, 31);
        per = max((int64_t)1, divide(total + gridDim.x - 1, gridDim.x));
        t = blockIdx.x * per;
        end = min(total, t + per);
        if (t >= total) return false;
        const int owner = __ffs(__ballot_sync(0xFFFFFFFFu, t < upto)) - 1;
        int64_t rel = t - __shfl_sync(0xFFFFFFFFu, upto - mine, owner);
        e.b = owner * lanes_per;
        e.s = sequence(a.c, e.b);
        int64_t per_head = head_places_warp(a, e.s);
        while (rel >= per_head * a.c.KH && e.b + 1 < a.c.batch) {
            rel -= per_head * a.c.KH;
            e.s = sequence(a.c, ++e.b);
            per_head = head_places_warp(a, e.s);
        }
        e.head = (int)divide(rel, per_head);
        rel -= e.head * per_head;
        // its row tile, 32 at a time
        row_tile_no = 0;
        const int n_tiles = row_tiles(a, e.s);
        for (int r0 = 0; r0 < n_tiles; r0 += 32) {
            const int64_t n = r0 + lane < n_tiles ? row_tile(a, e.s, r0 + lane).tiles + kEntryCost : 0, sum = warp_scan(n);
            const uint32_t has = __ballot_sync(0xFFFFFFFFu, rel < sum);
            if (has) {
                const int l = __ffs(has) - 1;
                row_tile_no = r0 + l;
                rel -= __shfl_sync(0xFFFFFFFFu, sum - n, l);
                break;
            }
            rel -= __shfl_sync(0xFFFFFFFFu, sum, 31);
        }
        e.rt = row_tile(a, e.s, row_tile_no);
        t0 = t - rel;
        return true;
    }
    // The entry at t, whose row tile has the places from t0: kEntryCost without a tile, then its tiles.  False if it gets
    // no tile here.
    __device__ __forceinline__ bool take() {
        const int64_t tiles0 = t0 + kEntryCost, stop = min(end, tiles0 + e.rt.tiles);
        e.tile0 = (int)max((int64_t)0, t - tiles0);
        e.count = (int)max((int64_t)0, stop - max(t, tiles0));
        e.first_cta = (int)divide(tiles0, per);
        e.last_cta = (int)divide(tiles0 + e.rt.tiles - 1, per);
        t = max(t + 1, stop);
        return e.count > 0;
    }
    // Goes to the row tile after it.
    __device__ __forceinline__ void next(const AttnArgs &a) {
        t0 = t;
        if (e.rt.r0 + e.rt.n_rows < e.s.n * a.group) {
            e.rt = row_tile(a, e.s, ++row_tile_no);
            return;
        }
        if (++e.head == a.c.KH) {
            e.head = 0;
            do {
                if (e.b + 1 >= a.c.batch) {                        // the arrays changed under the call
                    t = end;
                    return;
                }
                e.s = sequence(a.c, ++e.b);
            } while (e.s.n == 0);
        }
        e.rt = row_tile(a, e.s, row_tile_no = 0);
    }
};

template <int D>
struct Tile {
    static constexpr int kQ = kHalf * D * 2;         // bytes of a half's queries
    static constexpr int kF16 = kTok * D * 2;        // bytes of a converted tile
    static constexpr int kFp8 = kTok * D;            // bytes of a staged tile
    static constexpr int oQ = 0, oK = oQ + 2 * kQ, oV = oK + 2 * kF16, oS = oV + 2 * kF16, oAux = oS + 2 * kFp8;
    // behind the tiles (base 1024-aligned): scales, schedule, barriers, flags
    static constexpr int oMeta = oAux, oEntry = oMeta + kMetaRing * kGroups * 16, oBar = oEntry + kEntries * 64,
                         oFlag = oBar + 48 * 8;
    static constexpr size_t kSmem = oFlag + 64;
    static_assert(kSmem <= 227 * 1024 && sizeof(Entry) <= 64, "shared memory");
    static constexpr int kSub = kTok * 128;          // bytes of a 64-dim sub-tile (128 rows of 128 bytes)
    static constexpr int kPart = kRows * (D + 2);    // floats of a partial result
    static constexpr uint32_t cS = 0, cO = 256;      // tensor-memory columns
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
// Uses of these registers stay behind the wait before it.
__device__ __forceinline__ void pin32(float *r) {
    asm volatile(""
                 : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]),
                   "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15]),
                   "+f"(r[16]), "+f"(r[17]), "+f"(r[18]), "+f"(r[19]), "+f"(r[20]), "+f"(r[21]), "+f"(r[22]), "+f"(r[23]),
                   "+f"(r[24]), "+f"(r[25]), "+f"(r[26]), "+f"(r[27]), "+f"(r[28]), "+f"(r[29]), "+f"(r[30]), "+f"(r[31]));
}
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

// One staged tile of codes to f16: [token][dim], 64-dim sub-tiles of 128-byte swizzled rows.  128 threads.  Values of
// tokens outside from .. valid - 1 become zeros.
template <int D>
__device__ __forceinline__ void convert_tile(uint32_t src, uint32_t dst, int wt, bool values, int from, int valid,
                                             const float4 *meta) {
    const int lane = wt & 31, w = wt >> 5;
    const int rel = w * 32 + (lane & 7) - from;       // from <= r < valid in one comparison
    const uint32_t span = (uint32_t)max(0, valid - from);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {                // a warp: 8 tokens x 4 chunks of 16 codes a pass
        const int it = i * 4 + (lane >> 3);           // chunk index over (token group of 8, chunk)
        const int r = w * 32 + (it / (D / 16)) * 8 + (lane & 7), c = it % (D / 16);
        uint4 x = lds_v4(src + chunk_at<D>(r, c));
        if (values && ((uint32_t)(rel + it / (D / 16) * 8) >= span || meta[r >> 4].w == 0.f)) x = make_uint4(0u, 0u, 0u, 0u);
        const uint32_t row = dst + (c >> 2) * Tile<D>::kSub + r * 128;
        const int k = 2 * c & 7;
        sts128(row + ((k ^ (r & 7)) << 4), e4m3_lo(x.x), e4m3_hi(x.x), e4m3_lo(x.y), e4m3_hi(x.y));
        sts128(row + (((k + 1) ^ (r & 7)) << 4), e4m3_lo(x.z), e4m3_hi(x.z), e4m3_lo(x.w), e4m3_hi(x.w));
    }
}

// 16 bytes to shared memory behind the thread's back; zeros unless `real`.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}

template <int TYPE, int D>
__global__ void __launch_bounds__(kThreads, 1) attn_tile_kernel(const __grid_constant__ TileParams p) {
    using T = Tile<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const AttnArgs &a = p.a;
    const uint32_t base = smem_u32(smem);
    float4 *meta = reinterpret_cast<float4 *>(smem + T::oMeta);           // [kMetaRing][kGroups]: 2^ek, ev, 2^-ev, counts
    enum { Q_FULL = 0, ST_FULL = 2, ST_EMPTY = 4, K_FULL = 6, K_EMPTY = 8, V_FULL = 10, V_EMPTY = 12, HALF = 14, DRAIN = 16,
           S_FULL = 20, P_FULL = 24, PV_DONE = 28,                        // [2 halves][2 buffers]
           E_FULL = 32, E_EMPTY = 36 };
    auto bar = [&](int i) { return base + T::oBar + 8u * i; };
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(smem + T::oFlag);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + T::oFlag + 4);
    volatile int *last_flag = reinterpret_cast<volatile int *>(smem + T::oFlag + 8);           // [2]
    if (base & 1023u) {                                                   // the swizzles count on it
        set_err(a.c.err, ENGRAM_E_UNSUPPORTED);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(Q_FULL + i), 4);
            mbar_init(bar(ST_FULL + i), 1);
            mbar_init(bar(ST_EMPTY + i), 4);
            mbar_init(bar(K_FULL + i), 4);
            mbar_init(bar(K_EMPTY + i), 2);               // both halves' products
            mbar_init(bar(V_FULL + i), 4);
            mbar_init(bar(V_EMPTY + i), 2);
            mbar_init(bar(HALF + i), 4);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(bar(S_FULL + i), 1);
            mbar_init(bar(P_FULL + i), 4);
            mbar_init(bar(PV_DONE + i), 1);
            mbar_init(bar(DRAIN + i), 1);
        }
        for (int i = 0; i < kEntries; ++i) {
            mbar_init(bar(E_FULL + i), 1);
            mbar_init(bar(E_EMPTY + i), kEntryUsers);
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
    // A whole warp waits, and agrees on the outcome.
    auto wait = [&](int i, uint32_t parity) {
        return __all_sync(0xFFFFFFFFu, wait_bar(bar(i), parity & 1, abort_flag, err)) != 0;
    };
    // Entry number i of the CTA, and its release.
    auto entry = [&](uint32_t i) -> const Entry & {
        return *reinterpret_cast<const Entry *>(smem + T::oEntry + (i % kEntries) * 64);
    };
    auto open = [&](uint32_t i) { return wait(E_FULL + i % kEntries, i / kEntries) && entry(i).count > 0; };
    auto close = [&](uint32_t i) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(E_EMPTY + i % kEntries));
    };

    // 640 threads launch with 96 registers each: 2 x 128 x 136 + 128 x 80 + 2 x 128 x 64 are as many
    if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if (warp == 15) {
            // ---- the schedule ----
            Walk w;
            bool more = w.start(a);
            for (uint32_t i = 0;;) {
                if (more && !w.take()) {
                    more = w.t < w.end;
                    if (more) w.next(a);
                    continue;
                }
                if (!wait(E_EMPTY + i % kEntries, i / kEntries + 1)) break;
                if (!more) w.e.count = 0;
                if (lane == 0) *reinterpret_cast<Entry *>(smem + T::oEntry + (i % kEntries) * 64) = w.e;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(E_FULL + i % kEntries));
                if (!more) break;
                ++i;
                more = w.t < w.end;
                if (more) w.next(a);
            }
        } else if (warp == 13) {
            // ---- pages, scales, copies ----
            bool ok = true;
            uint32_t it = 0;
            for (uint32_t i = 0; ok && (ok = open(i)); close(i++)) {
                const Entry &e = entry(i);
                const int tok0 = e.rt.lo + e.tile0 * kTok, kv = e.s.kv, b = e.b, head = e.head, count = e.count;
                const int first = e.rt.first;
                const int at = 16 * (lane & 7);
                const bool leader = lane < 8 && (at & (a.c.pt - 1)) == 0;
                // a page that ends before the first token that a row sees is not looked up: a sliding window's pages may
                // have been given back
                auto page_at = [&](int j) {
                    const int tok = tok0 + j * kTok + at;
                    return lane < 8 && j < count && tok < kv && (tok | (a.c.pt - 1)) >= first ? page_of(a.c, b, tok >> a.c.pt_log2) : -1;
                };
                auto scales_of = [&](int id) {
                    if (id < 0) return 0u;
                    const int64_t k = (int64_t)id * a.c.KH + head;
                    return (uint32_t)a.c.k_scales[k] | (uint32_t)a.c.v_scales[k] << 8;
                };
                int id = page_at(0), id1 = page_at(1);
                uint32_t sc = scales_of(id);
                for (int j = 0; j < count; ++j, ++it) {
                    const int id2 = page_at(j + 2);
                    const uint32_t sc1 = scales_of(id1);
                    const int page = id < 0 ? a.c.n_pages : id;           // outside the cache: zeros
                    if (!(ok = wait(ST_EMPTY + 0, it + 1))) break;
                    if (lane < 8)
                        meta[(it % kMetaRing) * kGroups + lane] =
                            id < 0 ? make_float4(1.f, -INFINITY, 0.f, 0.f)
                                   : make_float4(e8m0_to_f32(sc & 255u), value_exp(sc >> 8), value_unscale(sc >> 8),
                                                 (int)(sc >> 8) < kLeastValueByte ? 0.f : 1.f);
                    __syncwarp();
                    if (lane == 0) mbar_expect_tx(bar(ST_FULL + 0), T::kFp8);
                    __syncwarp();
                    const int in_page = (tok0 + at) & (a.c.pt - 1);
                    if (leader) tma_load_4d(base + T::oS + at * D, &p.mk, 0, in_page, head, page, bar(ST_FULL + 0));
                    if (!(ok = wait(ST_EMPTY + 1, it + 1))) {
                        ++it;
                        break;
                    }
                    if (lane == 0) mbar_expect_tx(bar(ST_FULL + 1), T::kFp8);
                    __syncwarp();
                    if (leader) tma_load_4d(base + T::oS + T::kFp8 + at * D, &p.mv, 0, in_page, head, page, bar(ST_FULL + 1));
                    id = id1;
                    sc = sc1;
                    id1 = id2;
                }
            }
            // every copy issued has landed before the CTA can leave (only an abort leaves one behind)
            const uint64_t t0 = now_ns();
            for (int x = 0; x < 2; ++x)
                while (it > 0 && !mbar_try(bar(ST_FULL + x), (it - 1) & 1) && now_ns() - t0 < 10000000ull) {
                }
        } else if (warp < 18) {
            // ---- the tensor cores, a warp a product and half (one warp a half for both products waited for each
            // second one before the next first: 380 against 366 us for 4096 tokens behind 4096) ----
            const bool second = warp >= 16;
            const int h = second ? warp - 16 : (warp - 12) >> 1;
            const int full = second ? V_FULL : K_FULL, empty = second ? V_EMPTY : K_EMPTY;
            bool ok = true;
            uint32_t n = 0, ns = 0, ent = 0;                              // tiles; score buffers and entries of the half
            for (uint32_t i = 0; ok && (ok = open(i)); close(i++)) {
                const int count = entry(i).count;
                if (h && entry(i).rt.n_rows <= kHalf) {
                    // no rows in this half: keep step with the converted tiles (their barriers count both halves)
                    for (int j = 0; j < count; ++j, ++n) {
                        if (!(ok = wait(full + (n & 1), n >> 1))) break;
                        if (lane == 0) mbar_arrive(bar(empty + (n & 1)));
                    }
                    continue;
                }
                if (!second && !(ok = wait(Q_FULL + h, ent++))) continue;
                for (int s = 0; s < 2 * count; ++s, ++ns) {
                    // scores go over the probabilities two parts before: their product has to be done
                    ok = ((s & 1) || wait(full + (n & 1), n >> 1)) &&
                         (second ? wait(P_FULL + 2 * h + (s & 1), ns >> 1)
                                 : s < 2 || wait(PV_DONE + 2 * h + (s & 1), (ns >> 1) - 1));
                    if (!ok) break;
                    const uint32_t at = base + (second ? T::oV : T::oK) + (n & 1) * T::kF16 + (s & 1) * (kPartTok * 128);
                    const uint32_t tS = tmem + T::cS + h * 128 + (s & 1) * kPartTok;
                    tc_fence_after();
                    if (elect()) {
                        if (second) {
                            const uint32_t v_lo = desc_lo(at, T::kSub);
#pragma unroll
                            for (int kk = 0; kk < kPartTok / 16; ++kk)
                                mma_ts<idesc_f16(kHalf, D, true)>(tmem + T::cO + h * D, tS + kk * 8, v_lo + kk * (2048 >> 4),
                                                                  (s | kk) != 0);
                            commit(bar(PV_DONE + 2 * h + (s & 1)));
                        } else {
                            const uint32_t q_lo = desc_lo(base + T::oQ + h * T::kQ, 16), k_lo = desc_lo(at, 16);
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk) {
                                const uint32_t off = ((kk >> 2) * T::kSub + (kk & 3) * 32) >> 4;
                                mma_ss<idesc_f16(kHalf, kPartTok, false)>(tS, q_lo + off, k_lo + off, kk != 0);
                            }
                            commit(bar(S_FULL + 2 * h + (s & 1)));
                        }
                        if (s & 1) commit(bar(empty + (n & 1)));
                    }
                    __syncwarp();
                    n += s & 1;
                }
            }
            __syncwarp();
            const int drain = DRAIN + 2 * second + h;
            if (elect()) commit(bar(drain));                              // from the lane that issued the MMAs
            const uint64_t t0 = now_ns();
            while (!mbar_try(bar(drain), 0) && now_ns() - t0 < 100000000ull) {
            }
            __syncwarp();
        }
    } else if (warp >= kSoftWarps) {
        // ---- codes to f16 ----
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        const int wt = threadIdx.x - 32 * kSoftWarps;
        bool ok = true;
        uint32_t n = 0;
        for (uint32_t i = 0; ok && (ok = open(i)); close(i++)) {
            const int tok0 = entry(i).rt.lo + entry(i).tile0 * kTok, count = entry(i).count;
            const int left = entry(i).s.kv - tok0, unseen = max(0, entry(i).rt.first - tok0);   // under 128: the first tile's
            for (int j = 0; j < count && ok; ++j, ++n) {
                const int valid = left - j * kTok;                        // tokens of the tile that exist
                for (int x = 0; x < 2; ++x) {
                    ok = wait(ST_FULL + x, n) && wait((x ? V_EMPTY : K_EMPTY) + (n & 1), (n >> 1) + 1);
                    if (!ok) break;
                    convert_tile<D>(base + T::oS + x * T::kFp8, base + (x ? T::oV : T::oK) + (n & 1) * T::kF16, wt, x != 0,
                                    j == 0 ? unseen : 0, valid, meta + (n % kMetaRing) * kGroups);
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(bar(ST_EMPTY + x));
                        mbar_arrive(bar((x ? V_FULL : K_FULL) + (n & 1)));
                    }
                }
            }
        }
    } else {
        // ---- softmax, one thread a row ----
        asm volatile("setmaxnreg.inc.sync.aligned.u32 136;");
        const int h = warp >> 2, row = (warp & 3) * 32 + lane;            // row of the half = tensor-memory lane
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t tO = lanes + T::cO + h * D;
        uint32_t n = 0, ns = 0, half_syncs = 0;                          // tiles, score buffers of this half
        auto half_sync = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(HALF + h));
            return wait(HALF + h, half_syncs++);
        };
        // a row of the half is kChunks chunks of 16 bytes (swizzled, 64 dims a sub-tile); a warp moves kPerLoad rows at a time
        constexpr int kChunks = D / 8, kPerLoad = 32 / kChunks;
        auto q_chunk = [&](int r, int k) {
            return base + T::oQ + h * T::kQ + (k >> 3) * T::kSub + r * 128 + (((k & 7) ^ (r & 7)) << 4);
        };
        bool ok = true;
        for (uint32_t i = 0; ok && (ok = open(i)); close(i++)) {
            const Entry &e = entry(i);
            const int count = e.count;
            if (h * kHalf >= e.rt.n_rows) {                               // no rows in this half
                n += count;
                continue;
            }
            // the columns of the buffer that the row sees: lo_col <= column < hi_col, moving with the step
            int hi_col, lo_col, moving;
            float kf;
            {
                const int rr = e.rt.r0 + h * kHalf + row, tok_i = by_group(a, rr);
                const bool live = h * kHalf + row < e.rt.n_rows;
                const int64_t q_row = e.s.row0 + tok_i;
                const int q_head = e.head * a.group + rr - tok_i * a.group;
                const int pos = e.s.kv - e.s.n + tok_i, tb0 = e.rt.lo + e.tile0 * kTok;
                moving = live ? kPartTok : 0;
                hi_col = live ? pos + 1 - tb0 : kPartTok;
                lo_col = live && a.window ? pos - a.window + 1 - tb0 : 0;
                // the warp's rows come in kPerLoad whole rows a copy, then each thread scales its own (loads of 16 bytes of 32 rows
                // each: 4.1 against 2.2 us an entry)
                const int64_t off = live ? q_row * a.q_stride + (int64_t)q_head * D : -1;
#pragma unroll 4
                for (int k = 0; k < kChunks; ++k) {
                    const int r = k * kPerLoad + lane / kChunks, chunk = lane % kChunks;
                    const int64_t o = __shfl_sync(0xFFFFFFFFu, off, r);
                    copy16(q_chunk((warp & 3) * 32 + r, chunk),
                           static_cast<const uint16_t *>(a.q) + (o < 0 ? 0 : o + 8 * chunk), o >= 0);
                }
                asm volatile("cp.async.wait_all;" ::: "memory");
                __syncwarp();
                uint32_t m2 = 0;
#pragma unroll
                for (int k = 0; k < kChunks; ++k) {
                    const uint4 x = lds_v4(q_chunk(row, k));
                    m2 = __vmaxu2(__vmaxu2(m2, __vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu)),
                                  __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu));
                }
                const float2 m = q_pair<TYPE>(m2);
                float down;
                q_scale(max(__float_as_uint(m.x), __float_as_uint(m.y)), a.scale_log2, down, kf);
#pragma unroll 4
                for (int k = 0; k < kChunks; ++k) {
                    const uint32_t at = q_chunk(row, k);
                    const uint4 x = lds_v4(at);
                    auto scaled = [&](uint32_t w) {
                        const float2 f = q_pair<TYPE>(w);
                        return pack_f16x2(f.x * down, f.y * down);
                    };
                    sts128(at, scaled(x.x), scaled(x.y), scaled(x.z), scaled(x.w));
                }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(Q_FULL + h));

            float M = h * kHalf + row < e.rt.n_rows ? -INFINITY : INFINITY, L = 0.f;   // no row: never asks for a rescaling
            for (int j = 0; j < 2 * count; ++j, ++ns, hi_col -= moving, lo_col -= moving) {
                const uint32_t tS = lanes + T::cS + h * 128 + (j & 1) * kPartTok;
                if (!(ok = wait(S_FULL + 2 * h + (j & 1), ns >> 1))) break;
                tc_fence_after();
                // u_j = t_j - M with the bound so far.  The probabilities 2^u are formed at once and kept unless the sum of
                // 16 passes kLazySum; then, as on a row's first tokens, the largest u is found, M
                // raised to kRoom under it, and they are formed again.  (A search for the largest u beside each: 334 against 329 us.)
                const float4 *mt = meta + (n % kMetaRing) * kGroups + (j & 1) * (kGroups / 2);
                float t[64];
#pragma unroll
                for (int b = 0; b < 2; ++b) tmem_ld32_nowait(tS + 32 * b, t + 32 * b);
                tmem_wait_ld();
#pragma unroll
                for (int b = 0; b < 2; ++b) pin32(t + 32 * b);
                const float m0 = M == -INFINITY ? 0.f : M;
#pragma unroll
                for (int g = 0; g < kGroups / 2; ++g) {
                    const float4 f = mt[g];
                    const uint64_t c2 = pack2(kf * f.x, kf * f.x), e2 = pack2(f.y - m0, f.y - m0);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        float &x = t[16 * g + 2 * k], &y = t[16 * g + 2 * k + 1];
                        unpack2(fma2(pack2(x, y), c2, e2), x, y);
                    }
                }
                if (__any_sync(0xFFFFFFFFu, hi_col < kPartTok || lo_col > 0)) {
#pragma unroll
                    for (int k = 0; k < kPartTok; ++k)
                        if (k >= hi_col || k < lo_col) t[k] = -INFINITY;
                }
                uint32_t u[2][16];
                float l, big;                                             // their sum, and the largest sum of 16
                auto form = [&]() {
                    l = big = 0.f;
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        uint64_t sum[2][2] = {};
#pragma unroll
                        for (int k = 0; k < 8; ++k)
#pragma unroll
                            for (int g = 0; g < 2; ++g) {
                                const float *at = t + 32 * b + 16 * g + 2 * k;
                                const float x = exp2_approx(at[0]), y = exp2_approx(at[1]);
                                sum[g][k & 1] = add2(sum[g][k & 1], pack2(x, y));
                                u[b][8 * g + k] = pack_f16x2(x, y);
                            }
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            float x, y;
                            unpack2(add2(sum[g][0], sum[g][1]), x, y);
                            l = fmaf(x + y, mt[2 * b + g].z, l);
                            big = fmaxf(big, x + y);
                        }
                    }
                };
                form();
                if (__any_sync(0xFFFFFFFFu, M == -INFINITY || big > kLazySum)) {
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int k = 0; k < kPartTok / 2; ++k) mx[k & 3] = max3(mx[k & 3], t[2 * k], t[2 * k + 1]);
                    const float tmax = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    const float m2 = fmaxf(M, m0 + tmax - kRoom), f = M == m2 ? 1.f : exp2_approx(M - m2);
                    if (m2 != -INFINITY) {
                        const float d = m0 - m2;
#pragma unroll
                        for (int k = 0; k < kPartTok; ++k) t[k] += d;
                    }
                    M = m2;
                    L *= f;
                    if (j > 0) {
                        if (!(ok = wait(PV_DONE + 2 * h + (j + 1 & 1), (ns - 1) >> 1))) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int d = 0; d < D; d += 16) {
                            uint32_t o[16];
                            tmem_ld16(tO + d, o);
#pragma unroll
                            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                            tmem_st16(tO + d, o);
                        }
                    }
                    form();
                }
                tmem_st16(tS, u[0]);
                tmem_st16(tS + 16, u[1]);
                L += l;
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(P_FULL + 2 * h + (j & 1)));
                n += j & 1;
            }
            if (!ok) continue;

            // the entry's result, or a part of it
            if (!(ok = wait(PV_DONE + 2 * h + 1, (ns - 1) >> 1))) continue;   // the last product, and all before it
            tc_fence_after();
            const bool alone = e.first_cta == e.last_cta;
            const int rr = e.rt.r0 + h * kHalf + row, tok_i = by_group(a, rr);
            const bool live = h * kHalf + row < e.rt.n_rows;
            const int64_t q_row = e.s.row0 + tok_i;
            const int q_head = e.head * a.group + rr - tok_i * a.group;
            // the output goes through the place of the half's queries (no product reads them any more), for whole rows a store
            auto put = [&](int d, const float *x, float f) {              // 16 values from dim d
                uint32_t w[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    w[k] = TYPE == ENGRAM_T_BF16 ? pack_bf16x2(x[2 * k] * f, x[2 * k + 1] * f)
                                                 : pack_f16x2(x[2 * k] * f, x[2 * k + 1] * f);
                sts128(q_chunk(row, d / 8), w[0], w[1], w[2], w[3]);
                sts128(q_chunk(row, d / 8 + 1), w[4], w[5], w[6], w[7]);
            };
            auto put_rows = [&]() {
                const int64_t off = live ? q_row * a.out_stride + (int64_t)q_head * D : -1;
                __syncwarp();
#pragma unroll 4
                for (int k = 0; k < kChunks; ++k) {
                    const int r = k * kPerLoad + lane / kChunks;
                    const int64_t o = __shfl_sync(0xFFFFFFFFu, off, r);
                    const uint4 v = lds_v4(q_chunk((warp & 3) * 32 + r, lane % kChunks));
                    if (o >= 0) *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + o + lane % kChunks * 8) = v;
                }
                __syncwarp();
            };
            auto put_lse = [&](float m, float l) {
                if (live && a.lse) a.lse[q_row * a.H + q_head] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
            };
            const float inv = L == 0.f ? 0.f : 1.f / L;
            // partial results are column-major: float4 d4 of row r at [d4][r]
            const int64_t slot = (int64_t)blockIdx.x * 2 + ((int)blockIdx.x == e.first_cta ? 1 : 0);
            const int of = 4 * (h * kHalf + row);
#pragma unroll 1
            for (int d = 0; d < D; d += 16) {
                uint32_t o[16];
                tmem_ld16(tO + d, o);
                float x[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) x[k] = __uint_as_float(o[k]);
                if (alone) {
                    put(d, x, inv);
                } else {
                    float4 *part = reinterpret_cast<float4 *>(a.ws.part + slot * T::kPart + of) + d / 4 * kRows;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        part[k * kRows] = make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
                }
            }
            tc_fence_before();                                            // read: the next entry may overwrite them
            if (alone) {
                put_rows();
                put_lse(M, L);
                continue;
            }
            float *stat = a.ws.part + slot * T::kPart + kRows * D + h * kHalf + row;
            stat[0] = L == 0.f ? -INFINITY : M;
            stat[kRows] = L;
            if (!(ok = half_sync())) continue;
            if ((warp & 3) == 0 && lane == 0) {
                int *arrived = a.ws.arrived + e.first_cta * 2 + h;
                const bool last = arrive(arrived) == e.last_cta - e.first_cta;
                if (last) *arrived = 0;
                last_flag[h] = last;
            }
            if (!(ok = half_sync())) continue;
            if (last_flag[h]) {
                const float *st = a.ws.part + kRows * D + h * kHalf + row;
                const int parts = e.last_cta - e.first_cta + 1;
                auto at = [&](int k) { return ((int64_t)(e.first_cta + k) * 2 + (k == 0 ? 1 : 0)) * T::kPart; };
                // bounds and sums two parts at a time, then 32 dims of two parts at a time
                float m = -INFINITY, l = 0.f, f01[2] = {1.f, 1.f};
                auto last_of = [&](int k) { return min(k, parts - 1); };
                for (int k = 0; k < parts; k += 2) m = fmaxf(m, fmaxf(__ldcg(st + at(k)), __ldcg(st + at(last_of(k + 1)))));
                auto factor = [&](float mk, float lk) {
                    return mk == -INFINITY ? (lk == 0.f ? 0.f : 1.f) : exp2_approx(mk - m);
                };
                for (int k = 0; k < parts; k += 2) {
                    const float m0 = __ldcg(st + at(k)), l0 = __ldcg(st + at(k) + kRows), m1 = __ldcg(st + at(last_of(k + 1))),
                                l1 = __ldcg(st + at(last_of(k + 1)) + kRows);
                    const float f0 = factor(m0, l0), f1 = k + 1 < parts ? factor(m1, l1) : 0.f;
                    if (k == 0) f01[0] = f0, f01[1] = f1;
                    l = fmaf(l1, f1, fmaf(l0, f0, l));
                }
                const float il = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
                for (int d = 0; d < D; d += 32) {
                    float x[32] = {};
#pragma unroll 1
                    for (int k = 0; k < parts; k += 2) {
                        const int k1 = last_of(k + 1);
                        float f0 = f01[0], f1 = f01[1];
                        if (k) {
                            f0 = factor(__ldcg(st + at(k)), __ldcg(st + at(k) + kRows));
                            f1 = k + 1 < parts ? factor(__ldcg(st + at(k1)), __ldcg(st + at(k1) + kRows)) : 0.f;
                        }
                        const float4 *p0 = reinterpret_cast<const float4 *>(a.ws.part + at(k) + of) + d / 4 * kRows;
                        const float4 *p1 = reinterpret_cast<const float4 *>(a.ws.part + at(k1) + of) + d / 4 * kRows;
                        float4 v[8], w[8];
#pragma unroll
                        for (int q = 0; q < 8; ++q) v[q] = __ldcg(p0 + q * kRows), w[q] = __ldcg(p1 + q * kRows);
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            x[4 * q] = fmaf(w[q].x, f1, fmaf(v[q].x, f0, x[4 * q]));
                            x[4 * q + 1] = fmaf(w[q].y, f1, fmaf(v[q].y, f0, x[4 * q + 1]));
                            x[4 * q + 2] = fmaf(w[q].z, f1, fmaf(v[q].z, f0, x[4 * q + 2]));
                            x[4 * q + 3] = fmaf(w[q].w, f1, fmaf(v[q].w, f0, x[4 * q + 3]));
                        }
                    }
                    put(d, x, il);
                    put(d + 16, x + 16, il);
                }
                put_rows();
                put_lse(m, l);
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
