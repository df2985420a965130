// append.cu -- keys and values into the paged 8-bit cache, rotated on the way
// (engram_kv_append).
//
// A unit is one (sequence, page, head, K or V) that the call touches: its new
// tokens are read once into registers and rotated, their largest |value| and
// the block's earlier scale give the block's scale, and the codes go out; the
// page's earlier codes are read and encoded again only when the scale grew.
// One group of threads owns a unit, so nothing is shared between units and no
// order matters.  Further blocks rotate the queries, one row each.
// Bound by memory for prompts and by launch and load latency for single tokens.
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

// Eight elements from dim0 of the head at `base`, rotated to position pos.
template <int TYPE>
__device__ __forceinline__ void load_rotated(const AppendArgs &a, const void *p, int64_t base, int dim0, int64_t pos,
                                             bool turn, float (&x)[8]) {
    load8<TYPE>(p, base + dim0, x);
    if (!turn || dim0 >= a.rot) return;
    const float *cs = a.rope + pos * a.rot;                        // rot / 2 pairs
    if (a.interleaved) {
        float t[8];
        load8<ENGRAM_T_F32>(cs, dim0, t);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float c = t[2 * e], s = t[2 * e + 1], u = x[2 * e], w = x[2 * e + 1];
            x[2 * e] = __fsub_rn(__fmul_rn(u, c), __fmul_rn(w, s));
            x[2 * e + 1] = __fadd_rn(__fmul_rn(w, c), __fmul_rn(u, s));
        }
    } else {
        const int half = a.rot >> 1;
        const bool upper = dim0 >= half;
        const int d = upper ? dim0 - half : dim0;
        float y[8], t[8], t2[8];
        load8<TYPE>(p, base + (upper ? d : d + half), y);
        load8<ENGRAM_T_F32>(cs, 2 * d, t);
        load8<ENGRAM_T_F32>(cs, 2 * d + 8, t2);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float c = e < 4 ? t[2 * e] : t2[2 * e - 8], s = e < 4 ? t[2 * e + 1] : t2[2 * e - 7];
            x[e] = upper ? __fadd_rn(__fmul_rn(x[e], c), __fmul_rn(y[e], s))
                         : __fsub_rn(__fmul_rn(x[e], c), __fmul_rn(y[e], s));
        }
    }
}

// One row of queries.  A thread writes what it read (both halves of its pairs), so q_out may be q.
template <int TYPE>
__device__ __forceinline__ void query_row(const AppendArgs &a, int r) {
    const int b = sequence_of_row(a.c, r);
    if (b >= a.c.batch) return;
    const Seq s = sequence(a.c, b);
    if (r < s.row0 || r >= s.row0 + s.n) return;
    int fp, f;
    const bool known = pages_touched(a, s, fp, f) > 0;
    const int64_t pos = (int64_t)s.kv - s.n + (r - s.row0);
    const int D = a.c.D;
    const int half = a.rot >> 1, pairs = a.interleaved ? 0 : half >> 3, plain = (D - (a.interleaved ? 0 : a.rot)) >> 3;
    const int items = a.H * (pairs + plain);
    for (int i = threadIdx.x; i < items; i += blockDim.x) {
        const int h = i / (pairs + plain), j = i % (pairs + plain);
        const int64_t in = (int64_t)r * a.q_stride + (int64_t)h * D, to = (int64_t)r * a.q_out_stride + (int64_t)h * D;
        float x[8], y[8];
        if (pos < 0 || !known) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = 0.f;
            store8<TYPE>(a.q_out, to + (j < pairs ? 8 * j : (a.interleaved ? 0 : a.rot) + 8 * (j - pairs)), x);
            if (j < pairs) store8<TYPE>(a.q_out, to + half + 8 * j, x);
        } else if (j < pairs) {
            load_rotated<TYPE>(a, a.q, in, 8 * j, pos, true, x);
            load_rotated<TYPE>(a, a.q, in, half + 8 * j, pos, true, y);
            store8<TYPE>(a.q_out, to + 8 * j, x);
            store8<TYPE>(a.q_out, to + half + 8 * j, y);
        } else {
            const int d = (a.interleaved ? 0 : a.rot) + 8 * (j - pairs);
            load_rotated<TYPE>(a, a.q, in, d, pos, a.rot > 0, x);
            store8<TYPE>(a.q_out, to + d, x);
        }
    }
}

// W threads a unit (32: a warp, four units a block; 256: a block); NP passes of
// W / (D / 8) tokens stay in registers, longer units are read a second time (from L1 or L2).
template <int TYPE, int W, int NP>
__global__ void __launch_bounds__(W == 32 ? 128 : W) kv_append_kernel(const AppendArgs a) {
    __shared__ uint32_t part[W / 32];
    const int q_blocks = a.q ? a.c.rows : 0;
    if ((int)blockIdx.x < q_blocks) {
        query_row<TYPE>(a, blockIdx.x);
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
    const int lo = max(first, base), hi = min(s.kv, base + a.c.pt);   // the unit's new positions
    const int id = page_of(a.c, b, page);
    if (id < 0) return;
    uint8_t *codes = (which ? a.c.v : a.c.k) + id * a.c.page_stride + ((int64_t)head << a.c.pt_log2) * D;
    uint8_t *scale = (which ? a.c.v_scales : a.c.k_scales) + (int64_t)id * KH + head;
    const uint32_t old = lo > base ? *scale : 0u;
    const void *src = which ? a.v : a.k;
    const int64_t stride = which ? a.v_stride : a.k_stride;
    const int64_t row0 = s.row0 + s.n - (s.kv - lo);                 // row of position lo
    const int tpt = D >> 3, t0 = tid / tpt, dim0 = (tid % tpt) * 8, step = W / tpt;
    const bool turn = !which && a.rot > 0, one = hi - lo <= NP * step;

    float x[NP][8];
    uint32_t m = 0u;
    for (int c = 0; c < hi - lo; c += NP * step) {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int t = c + t0 + i * step;
            if (t < hi - lo) {
                load_rotated<TYPE>(a, src, (row0 + t) * stride + (int64_t)head * D, dim0, lo + t, turn, x[i]);
#pragma unroll
                for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(x[i][e]) & 0x7FFFFFFFu);
            }
        }
    }
    m = __reduce_max_sync(0xFFFFFFFFu, m);
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
    for (int c = 0; c < hi - lo; c += NP * step) {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int t = c + t0 + i * step;
            if (t < hi - lo) {
                if (!one)
                    load_rotated<TYPE>(a, src, (row0 + t) * stride + (int64_t)head * D, dim0, lo + t, turn, x[i]);
                *reinterpret_cast<uint2 *>(codes + (int64_t)(lo - base + t) * D + dim0) = encode8(x[i], byte);
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

template <int TYPE>
cudaError_t launch_typed(AppendArgs &a, cudaStream_t s) {
    const int64_t units = (int64_t)a.slots * 2 * a.c.KH;
    const int64_t q_blocks = a.q ? a.c.rows : 0;
    // a warp a unit while a sequence adds at most a few tokens, a block a unit for prompts
    if (a.c.max_rows <= 4) {
        kv_append_kernel<TYPE, 32, 2><<<(unsigned)(q_blocks + (units + 3) / 4), 128, 0, s>>>(a);
    } else {
        kv_append_kernel<TYPE, 256, 4><<<(unsigned)(q_blocks + units), 256, 0, s>>>(a);
    }
    return cudaGetLastError();
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
