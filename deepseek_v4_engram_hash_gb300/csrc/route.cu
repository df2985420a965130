// route.cu -- tokens to experts (engram_route): scores, groups, the top_k, their
// weights, and the lists of pairs by expert.
//
// A warp takes a token; lane l holds the experts l, l + 32, ...  A choice is the
// largest key (a float's bits, ordered as integers) by one warp-wide maximum of
// integers and the lowest index that has it by one minimum.  Scores are formed in 32 bits; where two that a choice
// depends on lie closer than their error (kTol, about one row in a thousand of 256
// sigmoid scores), the row is chosen again on scores in 64 bits.
//
// Lists: counts of a block's experts, then positions from the counts of the blocks
// before it (two kernels; one where a block takes all tokens).  A warp's tokens are consecutive and walked in order,
// and a token's choices are different experts, so a counter an expert and warp needs no atomics and the lists
// are in rising order.
//
// Bound by latency: one token is a chain of load, exponential and top_k + 1 maxima.
#include "experts.cuh"

namespace engram {

namespace {

constexpr int kWarps = 16, kThreads = kWarps * 32;
constexpr int kOneBlock = 64;                        // tokens up to which one block does all
constexpr int kBlocks = 152;                         // blocks at most of the others
constexpr unsigned kAll = 0xFFFFFFFFu;
// A 32-bit score is within 3e-7 max(1, |c|) of the 64-bit one: exp and the quotient are off by 2^-22 of s <= 1 at most,
// the sum with the bias by 2^-24 |c|; a softmax adds 2^-24 |l - max| e^(l - max) <= 2^-25.  Two of them, and sums of two, differ by twice that.
constexpr float kTol = 1e-6f;

int route_blocks(int tokens) {
    if (tokens <= kOneBlock) return 1;
    const int b = (tokens + kWarps - 1) / kWarps;
    return b < kBlocks ? b : kBlocks;
}

__device__ __forceinline__ float load_logit(const RouteArgs &a, int64_t i) {
    if (a.type == ENGRAM_T_F32) return __ldg(static_cast<const float *>(a.logits) + i);
    const uint32_t u = __ldg(static_cast<const uint16_t *>(a.logits) + i);
    return a.type == ENGRAM_T_BF16 ? __uint_as_float(u << 16) : __half2float(__ushort_as_half((unsigned short)u));
}

// Keys ordered as the numbers are; 0, below all of them, means not to be chosen.  (+ 0 makes -0 the same as 0.)
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    return u ^ ((int)u < 0 ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
    return __uint_as_float((int)k < 0 ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ uint64_t key_of(double x) {
    const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
    return u ^ ((long long)u < 0 ? ~0ull : 1ull << 63);
}
__device__ __forceinline__ double of_key(uint64_t k) {
    return __longlong_as_double((long long)((long long)k < 0 ? k ^ (1ull << 63) : ~k));
}
__device__ __forceinline__ uint32_t warp_max(uint32_t k) { return __reduce_max_sync(kAll, k); }
__device__ __forceinline__ uint64_t warp_max(uint64_t k) {
    const uint32_t hi = __reduce_max_sync(kAll, (uint32_t)(k >> 32));
    const uint32_t lo = __reduce_max_sync(kAll, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
    return (uint64_t)hi << 32 | lo;
}

template <class Key> struct Real;
template <> struct Real<uint32_t> { using type = float; };
template <> struct Real<uint64_t> { using type = double; };

// Largest key of the warp and the lowest expert that has it (key 0: none left).
template <class Key, int NV>
__device__ __forceinline__ Key best_of(const Key (&key)[NV], int lane, int &e) {
    Key m = 0;
    int at = 0;
#pragma unroll
    for (int v = 0; v < NV; ++v)
        if (key[v] > m) m = key[v], at = v;          // the lowest of equal ones
    const Key top = warp_max(m);
    e = (int)__reduce_min_sync(kAll, m == top ? (unsigned)(at * 32 + lane) : 0xFFFFFFFFu);
    return top;
}

// Whether two scores that order experts e and f by their 32-bit values are too near to do so: not if they are equal for being
// formed of the same numbers.
__device__ __forceinline__ bool unsure(const RouteArgs &a, int64_t row, float x, float y, int e, int f) {
    if (x - y > kTol * fmaxf(1.f, fabsf(x))) return false;
    return !(load_logit(a, row * a.stride + e) == load_logit(a, row * a.stride + f) && a.bias[e] == a.bias[f]);
}

// The row's choices from `key` (consumed), with `group` the values that order groups (without a bias and of two: the scores).
// Lane j gets id j (-1: none).  CHECK: false where 32 bits leave a doubt.
template <bool CHECK, class Key, int NV>
__device__ __forceinline__ bool choose(const RouteArgs &a, int64_t row, Key (&key)[NV], const Key (&group)[NV], bool exact,
                                       int lane, int &id) {
    using T = typename Real<Key>::type;
    const engram_router &r = a.r;
    bool sure = true;
    if (r.top_groups < r.n_groups) {
        const int size = r.n_experts / r.n_groups;
        Key mine = 0;                                // lane g: group g's sum
        for (int g = 0; g < r.n_groups; ++g) {
            const int lo = g * size, hi = lo + size;
            Key in[NV];
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int e = v * 32 + lane;
                in[v] = e >= lo && e < hi ? group[v] : Key(0);
            }
            int e;
            const Key first = best_of(in, lane, e);
            Key sum = first;
            if (r.group_best == 2 && first) {
#pragma unroll
                for (int v = 0; v < NV; ++v)
                    if (v * 32 + lane == e) in[v] = 0;
                const Key second = best_of(in, lane, e);
                if (second) sum = key_of(of_key(first) + of_key(second));
            }
            if (lane == g) mine = sum;
        }
        unsigned kept = 0;
        T last = 0;
        for (int i = 0; i <= r.top_groups; ++i) {
            const Key top = warp_max(mine);
            const int g = (int)__reduce_min_sync(kAll, mine == top ? (unsigned)lane : 0xFFFFFFFFu);
            if (i == r.top_groups) {
                // single logits and equal infinities need no care
                if (CHECK && top && !(exact && r.group_best == 1) && last - of_key(top) <= (T)(2 * kTol) * fmax((T)1, fabs(last)))
                    sure = false;
                break;
            }
            if (!top) break;                         // masked groups alone are left
            last = of_key(top);
            kept |= 1u << g;
            if (lane == g) mine = 0;
        }
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (!(kept >> min(31, (v * 32 + lane) / size) & 1)) key[v] = 0;
    }
    id = -1;
    int before = -1;
    T last = 0;
    for (int j = 0; j <= r.top_k; ++j) {
        int e;
        const Key top = best_of(key, lane, e);
        if (!top) break;
        if (CHECK && !exact && before >= 0 && unsure(a, row, (float)last, (float)of_key(top), before, e)) sure = false;
        if (j == r.top_k) break;
        last = of_key(top);
        before = e;
        if (lane == j) id = e;
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (v * 32 + lane == e) key[v] = 0;
    }
    return sure;
}

// The same on scores in 64 bits.
template <int NV>
__device__ __noinline__ void choose_again(const RouteArgs &a, int64_t row, int lane, int &id) {
    uint64_t key[NV], group[NV];
    double s[NV], top = -INFINITY, sum = 0;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int e = v * 32 + lane;
        s[v] = e < a.r.n_experts ? (double)load_logit(a, row * a.stride + e) : -INFINITY;
        if (s[v] != s[v]) s[v] = -INFINITY;
        top = fmax(top, s[v]);
    }
    const bool soft = a.r.score == ENGRAM_SCORE_SOFTMAX;
    if (soft) {
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmax(top, __shfl_xor_sync(kAll, top, o));
#pragma unroll
        for (int v = 0; v < NV; ++v) sum += s[v] == -INFINITY ? 0. : exp(s[v] - top);
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int e = v * 32 + lane;
        const bool masked = s[v] == -INFINITY;
        const double p = soft ? exp(s[v] - top) / sum : 1. / (1. + exp(-s[v]));
        key[v] = masked ? 0 : key_of(a.bias ? p + (double)a.bias[e] : s[v]);
        group[v] = masked ? 0 : a.bias || a.r.group_best == 1 ? key[v] : key_of(p);
    }
    choose<false>(a, row, key, group, true, lane, id);
}

// Token `row`: its ids and weights, one choice a lane.
template <int NV>
__device__ __forceinline__ int route_row(const RouteArgs &a, int64_t row, int lane) {
    const engram_router &r = a.r;
    const bool soft = r.score == ENGRAM_SCORE_SOFTMAX;
    float l[NV], top = -INFINITY, sum = 0.f;
    bool nan = false;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int e = v * 32 + lane;
        l[v] = e < r.n_experts ? load_logit(a, row * a.stride + e) : -INFINITY;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        nan |= l[v] != l[v] || (soft && l[v] == INFINITY);
        if (l[v] != l[v]) l[v] = -INFINITY;
        top = fmaxf(top, l[v]);
    }
    nan = __any_sync(kAll, nan);
    if (soft) {
        top = of_key(__reduce_max_sync(kAll, key_of(top)));
#pragma unroll
        for (int v = 0; v < NV; ++v) sum += l[v] == -INFINITY ? 0.f : expf(l[v] - top);
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    }
    const bool scores = a.bias || (r.top_groups < r.n_groups && r.group_best == 2);
    uint32_t key[NV], group[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int e = v * 32 + lane;
        const bool masked = l[v] == -INFINITY;
        float p = 0.f;
        if (scores && !masked) p = soft ? expf(l[v] - top) / sum : 1.f / (1.f + expf(-l[v]));
        key[v] = masked ? 0u : key_of(a.bias ? p + __ldg(a.bias + e) : l[v]);
        group[v] = masked ? 0u : a.bias || r.group_best == 1 ? key[v] : key_of(p);
    }
    int id;
    // a row with infinite scores that are equal is as sure as another (a NaN of inf - inf)
    if (!choose<true>(a, row, key, group, !a.bias, lane, id)) choose_again<NV>(a, row, lane, id);
    float s = 0.f;
    if (id >= 0) {
        const float x = load_logit(a, row * a.stride + id);
        s = soft ? expf(x - top) / sum : 1.f / (1.f + expf(-x));
    }
    if (r.renormalise) {
        float t = s;
#pragma unroll
        for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(kAll, t, o);
        s = s / (t + 1e-20f);
    }
    if (lane < r.top_k) {
        a.ids[row * r.top_k + lane] = id;
        a.weights[row * r.top_k + lane] = nan ? __int_as_float(0x7FFFFFFF) : id < 0 ? 0.f : s * r.scale;
    }
    return id;
}

// Tokens of warp `w` of block b.
__device__ __forceinline__ void warp_tokens(const RouteArgs &a, int b, int blocks, int w, int64_t &lo, int64_t &hi) {
    const int64_t n = (int64_t)blocks * kWarps, i = (int64_t)b * kWarps + w;
    lo = a.tokens * i / n;
    hi = a.tokens * (i + 1) / n;
}

// Exclusive sums over `n` values of v[], all threads of the block; v[n] gets the total.  part: 32 ints.
__device__ __forceinline__ void block_scan(int *v, int n, int *part) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int carry = 0;
    for (int i0 = 0; i0 < n; i0 += kThreads) {
        const int i = i0 + tid, x = i < n ? v[i] : 0;
        int s = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kAll, s, o);
            if (lane >= o) s += y;
        }
        if (lane == 31) part[warp] = s;
        __syncthreads();
        int before = carry, total = carry;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before += part[w];
            total += part[w];
        }
        if (i < n) v[i] = before + s - x;
        carry = total;
        __syncthreads();
    }
    if (tid == 0) v[n] = carry;
    __syncthreads();
}

// Counts of the warp's pairs by expert.
__device__ __forceinline__ void count_row(const RouteArgs &a, int *mine, int id, int lane) {
    if (id >= 0) ++mine[id];                         // a token's choices are different experts
    __syncwarp();
}

// counts: [kWarps][E] of the block's warps, turned into the first position of each; first: position of the block's first pair
// of each expert.  Then the warp's pairs to their places.
__device__ __forceinline__ void place_pairs(const RouteArgs &a, int *counts, const int *first, int64_t lo, int64_t hi) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, E = a.r.n_experts, k = a.r.top_k;
    for (int e = tid; e < E; e += kThreads) {
        int at = first[e];
        for (int w = 0; w < kWarps; ++w) {
            const int n = counts[w * E + e];
            counts[w * E + e] = at;
            at += n;
        }
    }
    __syncthreads();
    int *mine = counts + warp * E;
    for (int64_t t = lo; t < hi; ++t) {
        const int id = lane < k ? a.ids[t * k + lane] : -1;
        if (id >= 0) a.pairs[mine[id]++] = (int)(t * k + lane);
        __syncwarp();
    }
}

// One block: everything.  Several: ids, weights and the block's counts (ws).
template <int NV>
__global__ void __launch_bounds__(kThreads) route_kernel(const RouteArgs a) {
    extern __shared__ int smem[];
    __shared__ int part[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, E = a.r.n_experts;
    int *counts = smem, *mine = counts + warp * E, *first = counts + kWarps * E;
    int64_t lo, hi;
    warp_tokens(a, blockIdx.x, gridDim.x, warp, lo, hi);
    if (a.offsets)
        for (int e = lane; e < E; e += 32) mine[e] = 0;
    __syncwarp();
    for (int64_t t = lo; t < hi; ++t) {
        const int id = route_row<NV>(a, t, lane);
        if (a.offsets) count_row(a, mine, id, lane);
    }
    if (!a.offsets) return;
    __syncthreads();
    if (gridDim.x > 1) {
        for (int e = tid; e < E; e += kThreads) {
            int n = 0;
            for (int w = 0; w < kWarps; ++w) n += counts[w * E + e];
            a.ws[(int64_t)blockIdx.x * E + e] = n;
        }
        return;
    }
    for (int e = tid; e < E; e += kThreads) {
        int n = 0;
        for (int w = 0; w < kWarps; ++w) n += counts[w * E + e];
        first[e] = n;
    }
    __syncthreads();
    block_scan(first, E, part);
    for (int e = tid; e <= E; e += kThreads) a.offsets[e] = first[e];
    place_pairs(a, counts, first, lo, hi);
}

__global__ void __launch_bounds__(kThreads) route_lists_kernel(const RouteArgs a) {
    extern __shared__ int smem[];
    __shared__ int part[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, E = a.r.n_experts, k = a.r.top_k;
    int *counts = smem, *mine = counts + warp * E, *first = counts + kWarps * E, *before = first + E + 1;
    int64_t lo, hi;
    warp_tokens(a, blockIdx.x, gridDim.x, warp, lo, hi);
    for (int e = lane; e < E; e += 32) mine[e] = 0;
    __syncwarp();
    for (int64_t t = lo; t < hi; ++t) count_row(a, mine, lane < k ? a.ids[t * k + lane] : -1, lane);
    for (int e = tid; e < E; e += kThreads) {
        int n = 0, sum = 0;
#pragma unroll 8
        for (int b = 0; b < (int)gridDim.x; ++b) {
            const int c = a.ws[(int64_t)b * E + e];
            n += b < (int)blockIdx.x ? c : 0;
            sum += c;
        }
        first[e] = sum;
        before[e] = n;
    }
    __syncthreads();
    block_scan(first, E, part);
    if (blockIdx.x == 0)
        for (int e = tid; e <= E; e += kThreads) a.offsets[e] = first[e];
    __syncthreads();
    for (int e = tid; e < E; e += kThreads) first[e] += before[e];
    __syncthreads();
    place_pairs(a, counts, first, lo, hi);
}

constexpr size_t smem_bytes(int E) { return ((size_t)(kWarps + 2) * E + 2) * sizeof(int); }

// Once a device: dynamic shared memory for the most experts.
cudaError_t allow_smem(void (*kernel)(const RouteArgs), bool (&done)[64]) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (done[dev]) return cudaSuccess;
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes(kMaxExperts));
    done[dev] = e == cudaSuccess;
    return e;
}

template <int NV>
cudaError_t launch_rows(const RouteArgs &a, int blocks, size_t smem, cudaStream_t s) {
    static bool wide[64] = {};
    const cudaError_t e = allow_smem(route_kernel<NV>, wide);
    if (e != cudaSuccess) return e;
    route_kernel<NV><<<blocks, kThreads, smem, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

size_t route_workspace_ints(int n_experts, int tokens) {
    const int b = route_blocks(tokens);
    return b > 1 ? (size_t)b * n_experts : 0;
}

cudaError_t launch_route(const RouteArgs &a, cudaStream_t s) {
    const int blocks = route_blocks(a.tokens), E = a.r.n_experts;
    const size_t smem = smem_bytes(E);
    cudaError_t e;
    if (E <= 32)
        e = launch_rows<1>(a, blocks, smem, s);
    else if (E <= 64)
        e = launch_rows<2>(a, blocks, smem, s);
    else if (E <= 128)
        e = launch_rows<4>(a, blocks, smem, s);
    else if (E <= 256)
        e = launch_rows<8>(a, blocks, smem, s);
    else if (E <= 512)
        e = launch_rows<16>(a, blocks, smem, s);
    else
        e = launch_rows<32>(a, blocks, smem, s);
    if (e != cudaSuccess || blocks == 1 || !a.offsets) return e;
    static bool wide[64] = {};
    e = allow_smem(route_lists_kernel, wide);
    if (e != cudaSuccess) return e;
    route_lists_kernel<<<blocks, kThreads, smem, s>>>(a);
    return cudaGetLastError();
}

}  // namespace engram
