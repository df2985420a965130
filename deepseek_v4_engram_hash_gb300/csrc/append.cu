// append.cu -- keys and values into the paged 8-bit cache, rotated on the way
// (engram_kv_append).
//
// A unit is one (sequence, page, head, K or V) that the call touches: its new
// tokens are read once into registers and rotated, their largest |value| and
// the block's earlier scale give the block's scale, and the codes go out; the
// page's earlier codes are read and encoded again only when the scale grew.
// One group of threads owns a unit, so nothing is shared between units and no
// order matters.  Further blocks rotate the queries.
// Bound by latency: of launch and loads for single tokens, for prompts of 2.6 waves of blocks that each load, take a
// maximum and store.  64 registers a thread keep 1024 threads on an SM and spill (block-wide forms: 48 to 64 bytes stored,
// 64 to 104 loaded a thread): a 4096-token prompt of 32 query and 8 key/value heads of
// 128 (94 MB, 13.9 us at the copy rate) takes 21.4 to 22.1 us; without the bound over 26 us.
#include "sublayer.cuh"

namespace engram {

namespace {

// The sequence that holds row r: how many sequences end at or before it (a whole warp calls this).
__device__ __forceinline__ int sequence_of_row(const KvView &c, int r) {
    if (!c.row_start) return r / c.max_rows;
    int before = 0;
    for (int b = threadIdx.x & 31; b < c.batch; b += 32) before += c.row_start[b + 1] <= r ? 1 : 0;
    return __reduce_add_sync(0xFFFFFFFFu, before);
}

// Pages that sequence s appends to, from the page of its first new token on.
__device__ __forceinline__ int pages_touched(const AppendArgs &a, const Seq &s, int &first_page, int &first) {
    first = max(0, s.kv - s.n);
    if (a.rope && (int64_t)s.kv > a.rope_positions) {
        set_err(a.c.err, ENGRAM_E_LENGTH);
        return 0;
    }
    first_page = first >> a.c.pt_log2;
    return s.kv > first ? ((s.kv - 1) >> a.c.pt_log2) - first_page + 1 : 0;
}

// Slot `slot` of the call as (sequence, page number of its touched pages); false past the last.  A whole warp calls this.
__device__ __forceinline__ bool find_slot(const AppendArgs &a, int slot, int &b, int &u) {
    if (a.span) {
        b = slot / a.span;
        u = slot % a.span;
        return b < a.c.batch;
    }
    const int lane = threadIdx.x & 31;
    const int per = (a.c.batch + 31) / 32;
    int mine = 0, fp, f;
    for (int j = 0; j < per; ++j) {
        const int i = lane * per + j;
        if (i < a.c.batch) mine += pages_touched(a, sequence(a.c, i), fp, f);
    }
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o) upto += x;
    }
    const uint32_t has = __ballot_sync(0xFFFFFFFFu, slot < upto);
    if (!has) return false;
    const int owner = __ffs(has) - 1;
    int left = slot - (upto - mine), fb = 0, fu = 0;
    if (lane == owner) {
        for (int j = 0; j < per; ++j) {
            const int i = lane * per + j;
            const int n = i < a.c.batch ? pages_touched(a, sequence(a.c, i), fp, f) : 0;
            if (left < n) {
                fb = i;
                fu = left;
                break;
            }
            left -= n;
        }
    }
    b = __shfl_sync(0xFFFFFFFFu, fb, owner);
    u = __shfl_sync(0xFFFFFFFFu, fu, owner);
    return true;
}

// Sixteen elements of a head, as two chunks of eight: item j of a head that rotates
// by halves has the elements 8j.. and their partners rot / 2 + 8j.., past rot and
// in every other case 16 consecutive ones.
enum { kPlain = 0, kHalves = 1, kAdjacent = 2 };
struct Item {
    int c0, c1, turn;
};
__device__ __forceinline__ Item item_of(const AppendArgs &a, int j, bool turn) {
    if (turn && !a.interleaved && 16 * j < a.rot) return {8 * j, (a.rot >> 1) + 8 * j, kHalves};
    return {16 * j, 16 * j + 8, turn && 16 * j < a.rot ? kAdjacent : kPlain};
}
// The (cos, sin) pairs of an item at a position: eight of them (kHalves: elements c0 .. c0 + 7; kAdjacent: 16 elements
// from c0).
__device__ __forceinline__ void load_angles(const AppendArgs &a, const Item &it, int64_t pos, float (&t)[16]) {
    if (it.turn == kPlain) return;
    const float *cs = a.rope + pos * a.rot + (it.turn == kHalves ? 2 * it.c0 : it.c0);
    float u[8], w[8];
    load8<ENGRAM_T_F32>(cs, 0, u);
    load8<ENGRAM_T_F32>(cs, 8, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] = u[e], t[8 + e] = w[e];
}
template <int TYPE>
__device__ __forceinline__ void load_item(const void *p, int64_t base, const Item &it, float (&x)[8], float (&y)[8]) {
    load8<TYPE>(p, base + it.c0, x);
    load8<TYPE>(p, base + it.c1, y);
}
__device__ __forceinline__ void rotate(const Item &it, const float (&t)[16], float (&x)[8], float (&y)[8]) {
    if (it.turn == kHalves) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float c = t[2 * e], s = t[2 * e + 1], u = x[e], w = y[e];
            x[e] = fmaf(u, c, -(w * s));
            y[e] = fmaf(w, c, u * s);
        }
    } else if (it.turn == kAdjacent) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float c = t[2 * e], s = t[2 * e + 1], u = x[2 * e], w = x[2 * e + 1];
            x[2 * e] = fmaf(u, c, -(w * s));
            x[2 * e + 1] = fmaf(w, c, u * s);
            const float c2 = t[8 + 2 * e], s2 = t[9 + 2 * e], u2 = y[2 * e], w2 = y[2 * e + 1];
            y[2 * e] = fmaf(u2, c2, -(w2 * s2));
            y[2 * e + 1] = fmaf(w2, c2, u2 * s2);
        }
    }
}

// Query rows, `per` of a block at a time: a thread keeps its place in a head (and its angles) and goes
// through the heads, the first loaded beside the row's sequence and angles.
// It writes what it read alone, so q_out may be q.
template <int TYPE>
__device__ __forceinline__ void query_rows(const AppendArgs &a, int block) {
    const int per = a.rows_per_block, threads = blockDim.x / per, t = threadIdx.x % threads;
    const int r = block * per + threadIdx.x / threads;                // a warp lies within one row
    if (r >= a.c.rows) return;
    const int items = a.c.D >> 4;                                     // 4 or 8: divides the threads of a row
    const int step = threads / items;
    const Item it = item_of(a, t % items, a.rot > 0);
    const int64_t in = (int64_t)r * a.q_stride, to = (int64_t)r * a.q_out_stride;
    constexpr int kHeads = TYPE == ENGRAM_T_F32 ? 1 : 2;              // loaded at a time (64 registers a thread)
    Raw8<TYPE> x[kHeads], y[kHeads];
    auto load = [&](int h) {
#pragma unroll
        for (int i = 0; i < kHeads; ++i)
            if (h + i * step < a.H) {
                x[i].load(a.q, in + (int64_t)(h + i * step) * a.c.D + it.c0);
                y[i].load(a.q, in + (int64_t)(h + i * step) * a.c.D + it.c1);
            }
    };
    int h = t / items;
    load(h);
    const int b = sequence_of_row(a.c, r);
    if (b >= a.c.batch) return;
    const Seq s = sequence(a.c, b);
    if (r < s.row0 || r >= s.row0 + s.n) return;
    int fp, f;
    const bool known = pages_touched(a, s, fp, f) > 0;
    const int64_t pos = (int64_t)s.kv - s.n + (r - s.row0);
    const bool empty = pos < 0 || !known;
    float cs[16];
    if (!empty) load_angles(a, it, pos, cs);
    while (h < a.H) {
#pragma unroll
        for (int i = 0; i < kHeads; ++i) {
            float u[8], w[8];
            x[i].get(u);
            y[i].get(w);
            if (empty) {
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] = w[e] = 0.f;
            } else {
                rotate(it, cs, u, w);
            }
            if (h + i * step < a.H) {
                store8<TYPE>(a.q_out, to + (int64_t)(h + i * step) * a.c.D + it.c0, u);
                store8<TYPE>(a.q_out, to + (int64_t)(h + i * step) * a.c.D + it.c1, w);
            }
        }
        h += kHeads * step;
        if (h < a.H) load(h);
    }
}

// W threads a unit (32: a warp, four units a block; else a block).  A unit has at most NP x W items
// of 16 elements, so its values stay in registers between their maximum and their codes.
template <int TYPE, int W, int NP>
__global__ void __launch_bounds__(W == 32 ? 128 : W, W == 32 ? 4 : 1024 / W) kv_append_kernel(const AppendArgs a) {
    __shared__ uint32_t part[W / 32];
    const int q_blocks = a.q ? (a.c.rows + a.rows_per_block - 1) / a.rows_per_block : 0;
    if ((int)blockIdx.x < q_blocks) {
        query_rows<TYPE>(a, blockIdx.x);
        return;
    }
    constexpr int kUnits = W == 32 ? 4 : 1;
    const int64_t unit = (int64_t)(blockIdx.x - q_blocks) * kUnits + (W == 32 ? threadIdx.x >> 5 : 0);
    const int tid = W == 32 ? threadIdx.x & 31 : threadIdx.x;
    const int KH = a.c.KH, D = a.c.D;
    const int slot = (int)(unit / (2 * KH)), which = (int)(unit % (2 * KH)) & 1, head = (int)(unit % (2 * KH)) >> 1;
    if (slot >= a.slots) return;
    int b, u;
    if (!find_slot(a, slot, b, u)) return;
    const Seq s = sequence(a.c, b);
    int first_page, first;
    if (u >= pages_touched(a, s, first_page, first)) return;
    const int page = first_page + u, base = page << a.c.pt_log2;
    const int lo = max(first, base), n_new = min(s.kv, base + a.c.pt) - lo;   // the unit's new positions
    const int id = page_of(a.c, b, page);
    if (id < 0) return;
    uint8_t *codes = (which ? a.c.v : a.c.k) + id * a.c.page_stride + ((int64_t)head << a.c.pt_log2) * D;
    uint8_t *scale = (which ? a.c.v_scales : a.c.k_scales) + (int64_t)id * KH + head;
    const uint32_t old = lo > base ? *scale : 0u;
    const void *src = which ? a.v : a.k;
    const int64_t stride = which ? a.v_stride : a.k_stride;
    const int64_t row0 = s.row0 + s.n - (s.kv - lo);                 // row of position lo
    const int items = D >> 4, t0 = tid / items, step = W / items;    // a thread keeps its place in the head
    const Item it = item_of(a, tid % items, !which && a.rot > 0);

    float x[NP][8], y[NP][8];
    float big = 0.f;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int t = t0 + i * step;
        if (t < n_new) {
            float cs[16];
            load_item<TYPE>(src, (row0 + t) * stride + (int64_t)head * D, it, x[i], y[i]);
            load_angles(a, it, lo + t, cs);
            rotate(it, cs, x[i], y[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e) big = amax3(big, x[i][e], y[i][e]);
        }
    }
    uint32_t m = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(big));   // bits of numbers, then infinity, then NaN
    if (W > 32) {
        if ((tid & 31) == 0) part[tid >> 5] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < W / 32; ++w) m = max(m, part[w]);
    } else {
        __syncwarp();                                                // every lane has read the old scale
    }
    const uint32_t byte = max(old, block_scale_byte(m));
    if (tid == 0) *scale = (uint8_t)byte;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int t = t0 + i * step;
        if (t < n_new) {
            uint8_t *to = codes + (int64_t)(lo - base + t) * D;
            const uint2 p = encode8(x[i], byte), q = encode8(y[i], byte);
            if (it.c1 == it.c0 + 8) {
                *reinterpret_cast<uint4 *>(to + it.c0) = make_uint4(p.x, p.y, q.x, q.y);
            } else {
                *reinterpret_cast<uint2 *>(to + it.c0) = p;
                *reinterpret_cast<uint2 *>(to + it.c1) = q;
            }
        }
    }
    if (lo > base && byte != old && byte != 255u) {
        // the block's earlier codes at the larger scale: exact but where they become subnormal
        const int down = (int)byte - (int)old;
        const float f = down > 126 ? 0.f : __uint_as_float((uint32_t)(127 - down) << 23);
        for (int i = tid; i < (lo - base) * D / 8; i += W) {
            uint2 *p = reinterpret_cast<uint2 *>(codes) + i;
            const uint2 w = *p;
            const float2 a0 = e4m3x2_to_f32(w.x), a1 = e4m3x2_to_f32(w.x >> 16), b0 = e4m3x2_to_f32(w.y),
                         b1 = e4m3x2_to_f32(w.y >> 16);
            *p = make_uint2(e4m3x4(a0.x * f, a0.y * f, a1.x * f, a1.y * f), e4m3x4(b0.x * f, b0.y * f, b1.x * f, b1.y * f));
        }
    }
}

template <int TYPE, int W, int NP>
cudaError_t launch_units(AppendArgs &a, cudaStream_t s) {
    const int threads = W == 32 ? 128 : W, kUnits = W == 32 ? 4 : 1;
    // a whole block a query row while the rows do not fill the GPU, else a warp (4096 rows of 32 heads: 21.4 us, with
    // 64 threads a row 22.9)
    a.rows_per_block = a.c.rows < 1024 ? 1 : threads / 32;
    const int64_t q_blocks = a.q ? (a.c.rows + a.rows_per_block - 1) / a.rows_per_block : 0;
    const int64_t units = (int64_t)a.slots * 2 * a.c.KH;
    kv_append_kernel<TYPE, W, NP><<<(unsigned)(q_blocks + (units + kUnits - 1) / kUnits), threads, 0, s>>>(a);
    return cudaGetLastError();
}

template <int TYPE>
cudaError_t launch_typed(AppendArgs &a, cudaStream_t s) {
    // a warp a unit while a sequence adds at most 4 tokens (4 x 8 items), else a block that holds a page in two items a thread
    const int items = a.c.pt * a.c.D >> 4;
    if (a.c.max_rows <= 4) return launch_units<TYPE, 32, 1>(a, s);
    if (items <= 256) return launch_units<TYPE, 128, 2>(a, s);
    return items <= 512 ? launch_units<TYPE, 256, 2>(a, s) : launch_units<TYPE, 512, 2>(a, s);
}

}  // namespace

cudaError_t launch_kv_append(AppendArgs a, cudaStream_t s) {
    // A sequence of n tokens touches at most (n + pt - 2) / pt + 1 pages, all of
    // them together at most rows / pt + 2 batch: slots are laid out a fixed
    // number a sequence where that is no more, else found by a prefix sum.
    const int64_t span = ((int64_t)a.c.max_rows + a.c.pt - 2) / a.c.pt + 1;
    const int64_t tight = a.c.rows / a.c.pt + 2ll * a.c.batch;
    const bool direct = span * a.c.batch <= tight;
    a.span = direct ? (int32_t)span : 0;
    const int64_t slots = direct ? span * a.c.batch : tight;
    if (slots * 2 * a.c.KH + a.c.rows > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    a.slots = (int32_t)slots;
    return a.type == ENGRAM_T_BF16 ? launch_typed<ENGRAM_T_BF16>(a, s)
           : a.type == ENGRAM_T_F16 ? launch_typed<ENGRAM_T_F16>(a, s)
                                    : launch_typed<ENGRAM_T_F32>(a, s);
}

}  // namespace engram
