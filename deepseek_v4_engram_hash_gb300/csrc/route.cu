// route.cu -- tokens to experts (engram_route): scores, groups, the top_k, their
// weights, and the lists of pairs by expert.
//
// A warp takes a token; lane l holds c = ceil(n_experts / 32) consecutive experts from l c on.  A
// lane sorts its experts (up to eight) by their keys, a float's bits ordered as integers; a choice is the largest first key by one
// warp-wide maximum of integers, the lowest lane that has it by a vote, and a step of that lane's list.  The sort is of 32-bit words that hold
// a key's upper 29 bits and its place, wherever that tells all that a choice needs.  Groups that are a power of two
// of lanes (8 groups of 256 experts: four) find their two largest all at once by exchanges.  Scores are formed in 32 bits;
// where two that a choice depends on lie closer than their error (tol_of, about one row in some hundreds of 256
// sigmoid scores), those in question are formed again in 64 bits, one a lane (all of a row's took its warp 15 us: so for softmax beside a bias).
//
// Lists: counts of a block's experts, then positions from the counts of the blocks
// before it (two kernels; one where a block takes all tokens).  A warp's tokens are consecutive and walked in order,
// and a token's choices are different experts, so a counter an expert and warp needs no atomics and the lists
// are in rising order.  Each block of the second kernel reads all blocks' counts (155 KB of 152 x 256, 24 MB from L2 in all) and counts its own
// tokens again before it places them: a third of a long prompt's time.
//
// Bound by latency and instructions: one token is a chain of load, exponential and top_k + 1 maxima, 6.0 us; 4096 tokens of 256 experts in 8
// groups, 8 choices, 24 us; 16384 of them 32 us, of which the lists' kernel is 10 and the rare rows in 64 bits, whose warps are the last, about 5 (up to
// 39 us with inputs of which more rows are in doubt).
#include "experts.cuh"

#include <mutex>

namespace engram {

namespace {

constexpr int kOneBlock = 32;                        // tokens up to which one block does all
constexpr int kBlocks = 152;                         // blocks at most of the others
constexpr unsigned kAll = 0xFFFFFFFFu;
// A 32-bit score that orders experts is within 4e-7 max(1, |c|) of the 64-bit one.  e = 2^(-l log2 e) is off by 2^-22 + 2^-23 |l| of itself, which
// moves s = 1 / (1 + e) by s (1 - s) of that, under 2^-23; 1 + e and the reciprocal (1 ulp) by 2^-24 + 2^-23 of s; the sum with the
// bias by 2^-24 |c|.  Two of them differ by twice that, 8e-7, and where keys lose their last three bits, all to the same side, by 7 2^-23 |c| =
// 8.4e-7 more: 1.7e-6.  Sums of two by twice as much.
constexpr float kTol = 2e-6f;
// The same for rows of NV experts a lane.  Softmax beside a bias, in units of u = 2^-24: of two p = e^(l - max) / sum, which are together at most 1, the
// exponentials, the differences' rounding and the products are off by 6 u in all; of the divisor, by which the two move apart by at most its own
// error, the terms by 4 u and by |l - max| u each, under 5 u of 1024 terms together, the sum by NV - 1 additions in a lane and 5
// exchanges, u each, and the reciprocal by u; the sums with the biases by u max(1, |c|) each: NV + 22 in all, and 14 for the keys' lost bits where
// NV is at most 8.  kTol is 33 of them.  (Without a bias the divisor is common to all that is compared.)
template <int NV>
__device__ __forceinline__ float tol_of(const RouteArgs &a) {
    return a.bias && a.r.score == ENGRAM_SCORE_SOFTMAX ? kTol + (NV + 4) * 0x1p-24f : kTol;
}

// Warps a block: 32 with 64 registers; rows of many experts take 16 with 128.
int route_warps(int n_experts) { return n_experts <= 256 ? 32 : 16; }
int route_blocks(int n_experts, int tokens) {
    if (tokens <= kOneBlock) return 1;
    const int w = route_warps(n_experts) / 4, b = (tokens + w - 1) / w;   // a few tokens do not wait for each other in a warp
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
    return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
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

// How lanes hold a row's experts, and groups their lanes.
struct Shape {
    int c;                              // experts a lane
    int size;                           // experts a group
    int lanes;                          // lanes a group where that is a power of two, else 0
};
__device__ __forceinline__ Shape shape_of(const engram_router &r) {
    Shape s;
    s.c = (r.n_experts + 31) / 32;
    s.size = r.n_experts / r.n_groups;
    s.lanes = s.size / s.c;
    if (s.lanes * s.c != s.size || (s.lanes & (s.lanes - 1))) s.lanes = 0;
    return s;
}

template <class Key>
__device__ __forceinline__ void two_best(Key &first, Key &second, Key x, Key y) {   // of (first, second) and (x, y), both ordered
    const Key low = first < x ? first : x;
    first = first < x ? x : first;
    second = second < y ? y : second;
    second = second < low ? low : second;
}

template <class Key>
__device__ __forceinline__ Key sum_of(int best, Key first, Key second) {
    return best == 2 && second ? key_of(of_key(first) + of_key(second)) : first;
}
// The two largest of this warp's (first, second)s.
template <class Key>
__device__ __forceinline__ void two_best_of_lanes(Key &first, Key &second, int lanes) {
    for (int o = 1; o < lanes; o <<= 1) {
        const Key x = __shfl_xor_sync(kAll, first, o), y = __shfl_xor_sync(kAll, second, o);
        two_best(first, second, x, y);
    }
}
// The larger of the two numbers' sizes: it bounds the error of their sum, which may be smaller.
template <class Key>
__device__ __forceinline__ float part_of(int best, Key first, Key second) {
    const float x = first ? fabsf((float)of_key(first)) : 0.f;
    return best == 2 && second ? fmaxf(x, fabsf((float)of_key(second))) : x;
}
// Groups that are no whole lanes: lane g gets group g's sum, and its larger part.
template <class Key, int NV>
__device__ __forceinline__ Key group_sums(const RouteArgs &a, const Shape &sh, const Key (&group)[NV], int lane, float &part) {
    Key mine = 0;
    part = 0.f;
    for (int g = 0; g < a.r.n_groups; ++g) {
        const int lo = g * sh.size - lane * sh.c, hi = lo + sh.size;   // of this lane's experts
        Key first = 0, second = 0;
#pragma unroll
        for (int v = 0; v < NV; ++v) two_best(first, second, v >= lo && v < hi ? group[v] : Key(0), Key(0));
        two_best_of_lanes(first, second, 32);
        if (lane == g) mine = sum_of(a.r.group_best, first, second), part = part_of(a.r.group_best, first, second);
    }
    return mine;
}
// The top_groups of the groups' sums `mine` (lane g: group g's).
template <class Key>
__device__ __forceinline__ unsigned keep_groups(const RouteArgs &a, Key mine, int lane) {
    unsigned kept = 0;
    for (int i = 0; i < a.r.top_groups; ++i) {
        const Key top = warp_max(mine);
        if (!top) break;                             // masked groups alone are left
        const int g = __ffs(__ballot_sync(kAll, mine == top)) - 1;
        kept |= 1u << g;
        mine = lane == g ? Key(0) : mine;
    }
    return kept;
}
// Whether 32 bits tell that the groups `kept` are those: the least that any of them can be is above the most that any other can.
__device__ __forceinline__ bool sure_of_groups(uint32_t mine, float part, unsigned kept, float tol, int lane) {
    const float x = of_key(mine), err = 2 * tol * fmaxf(1.f, part);
    const bool in = kept >> lane & 1;
    const uint32_t most = __reduce_max_sync(kAll, mine && !in ? key_of(x + err) : 0u);
    return !most || __reduce_min_sync(kAll, mine && in ? key_of(x - err) : 0xFFFFFFFFu) > most;
}
template <class Key, int NV>
__device__ __forceinline__ void mask_groups(const Shape &sh, unsigned kept, int lane, Key (&key)[NV]) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
        if (!(kept >> min(31, (lane * sh.c + v) / sh.size) & 1)) key[v] = 0;
}

// Whether two experts' scores are formed of the same numbers.
__device__ __forceinline__ bool same_numbers(const RouteArgs &a, int64_t row, int e, int f) {
    return load_logit(a, row * a.stride + e) == load_logit(a, row * a.stride + f) && a.bias[e] == a.bias[f];
}

// The top_k of the keys of which a lane's largest that is left is `m`, of its expert `at`; next(): the lane takes it out.  Lane j gets
// id j (-1: none).  CHECK: false where 32 bits leave a doubt about the order of two choices, or of the last and any that is left (`least`: the
// largest of those) -- not where two are equal for being formed of the same numbers.
template <bool CHECK, class Key, class Next>
__device__ __forceinline__ bool choose(const RouteArgs &a, const Shape &sh, int64_t row, Key &m, int &at, Next next, bool exact,
                                       float tol, int lane, int &id, Key &least) {
    const int k = a.r.top_k;
    id = -1;
    Key mine = 0, last = 0;
    int last_id = 0;
    least = 0;
    for (int j = 0;; ++j) {
        const Key top = warp_max(m);
        if (!top) break;
        if (j == k) {
            least = top;
            break;
        }
        const bool from = m == top;
        const unsigned who = __ballot_sync(kAll, from);
        const int first = __ffs(who) - 1;                // lower lanes hold lower experts
        last = top;
        last_id = __shfl_sync(kAll, lane * sh.c + at, first);
        id = lane == j ? last_id : id;
        mine = lane == j ? top : mine;
        next(lane == first);
    }
    if (!CHECK || exact) return true;
    const Key after = __shfl_down_sync(kAll, mine, 1);
    const int other = __shfl_down_sync(kAll, id, 1);
    bool doubt = false;
    if (lane < k - 1 && mine && after) {
        const float x = (float)of_key(mine), y = (float)of_key(after);
        doubt = x - y <= tol * fmaxf(1.f, fabsf(x)) && !same_numbers(a, row, id, other);
    }
    // Behind the last choice the key that stands first may be of the same numbers, and another behind that of larger ones.
    const float x = (float)of_key(last);
    const Key from = key_of(x - tol * fmaxf(1.f, fabsf(x)));
    while (__any_sync(kAll, m >= from)) {
        const bool near = m >= from;
        if (near) doubt |= !same_numbers(a, row, last_id, lane * sh.c + at);
        next(near);
    }
    return !__any_sync(kAll, doubt);
}
// The same on keys in registers, unsorted.
template <bool CHECK, class Key, int NV>
__device__ __forceinline__ bool choose_of(const RouteArgs &a, const Shape &sh, int64_t row, const Key (&key)[NV], bool exact, int lane,
                                          int &id, Key &least) {
    unsigned taken = 0;
    int at = 0;
    Key m = 0;
    auto next = [&](bool mine) {
        if (!mine) return;
        taken |= 1u << at;
        m = 0;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const Key x = taken >> v & 1 ? Key(0) : key[v];
            if (x > m) m = x, at = v;                // the lowest of equal ones
        }
    };
#pragma unroll
    for (int v = 0; v < NV; ++v)
        if (key[v] > m) m = key[v], at = v;
    return choose<CHECK>(a, sh, row, m, at, next, exact, tol_of<NV>(a), lane, id, least);
}

// Up to 32 experts, marked in `want` bit by bit of a lane, to one a lane in rising order; -1 behind the last.  False: more.
__device__ __forceinline__ bool one_a_lane(const Shape &sh, unsigned want, int lane, int &e) {
    int upto = __popc(want);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(kAll, upto, o);
        if (lane >= o) upto += x;
    }
    const int total = __shfl_sync(kAll, upto, 31);
    e = -1;
    if (total > 32) return false;
#pragma unroll 1
    for (int i = 0; i < total; ++i) {
        // the lane whose marks reach past i
        const int from = __ffs(__ballot_sync(kAll, upto > i)) - 1;
        const int x = __shfl_sync(kAll, lane * sh.c + __ffs(want) - 1, from);
        if (lane == i) e = x;
        if (lane == from) want &= want - 1;
    }
    return true;
}
// c of expert e in 64 bits (p without a bias), softmax without its divisor: for rows whose order it does not change.
__device__ __forceinline__ double score64(const RouteArgs &a, int64_t row, int e, float top) {
    const double x = (double)load_logit(a, row * a.stride + e);
    const double p = a.r.score == ENGRAM_SCORE_SOFTMAX ? exp(x - (double)top) : 1. / (1. + exp(-x));
    return a.bias ? p + (double)a.bias[e] : p;
}

// Logits of token `row` as a lane holds them; -inf where there is no expert.  wide: NV of them lie side by side in aligned 16 bytes.
template <int NV>
__device__ __forceinline__ void load_row(const RouteArgs &a, int c, bool wide, int64_t row, int lane, float (&l)[NV]) {
    const int64_t at = row * a.stride + lane * c;
    if (NV >= 4 && wide && a.type == ENGRAM_T_F32) {
#pragma unroll
        for (int v = 0; v + 3 < NV; v += 4) {
            const float4 x = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(a.logits) + at + v));
            l[v] = x.x, l[v + 1] = x.y, l[v + 2] = x.z, l[v + 3] = x.w;
        }
    } else if (NV >= 8 && wide) {
#pragma unroll
        for (int v = 0; v + 7 < NV; v += 8) {
            float x[8];
            const uint4 raw = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.logits) + at + v));
            if (a.type == ENGRAM_T_BF16)
                load8<ENGRAM_T_BF16>(&raw, 0, x);
            else
                load8<ENGRAM_T_F16>(&raw, 0, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) l[v + i] = x[i];
        }
    } else {
#pragma unroll
        for (int v = 0; v < NV; ++v)
            l[v] = v < c && lane * c + v < a.r.n_experts ? load_logit(a, at + v) : -INFINITY;
    }
}
template <int NV>
__device__ __forceinline__ bool wide_rows(const RouteArgs &a) {
    const int size = a.type == ENGRAM_T_F32 ? 4 : 2;
    return a.r.n_experts == 32 * NV && NV * size % 16 == 0 && a.stride * size % 16 == 0 && reinterpret_cast<uintptr_t>(a.logits) % 16 == 0;
}

// s of a logit; top and sum: a softmax's.
__device__ __forceinline__ float score32(bool soft, float x, float top, float sum) {
    return soft ? __fdividef(expf(x - top), sum) : __fdividef(1.f, 1.f + expf(-x));
}
__device__ __forceinline__ float reciprocal(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float exp_of(float x) {   // 2^(x log2 e); 0 below 2^-126
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.44269504f));
    return r;
}
// The same, of few instructions, to order by (see kTol); of sum its reciprocal.
__device__ __forceinline__ float quick_score(bool soft, float x, float top, float per_sum) {
    return soft ? exp_of(x - top) * per_sum : reciprocal(1.f + exp_of(-x));
}
// The value that orders groups, of a key.
__device__ __forceinline__ uint32_t group_key32(const RouteArgs &a, bool soft, uint32_t key, float top, float per_sum) {
    return !key || a.bias || a.r.group_best == 1 ? key : key_of(quick_score(soft, of_key(key), top, per_sum));
}
// Keys of the logits l; 0 for masked ones (-inf, NaN).
template <int NV>
__device__ __forceinline__ void keys_of(const RouteArgs &a, bool soft, const float (&l)[NV], const float (&bias)[NV], float top, float per_sum,
                                        uint32_t (&key)[NV]) {
    if (!a.bias) {
#pragma unroll
        for (int v = 0; v < NV; ++v) key[v] = key_of(l[v]);
    } else if (soft) {
#pragma unroll
        for (int v = 0; v < NV; ++v) key[v] = key_of(quick_score(true, l[v], top, per_sum) + bias[v]);
    } else {
#pragma unroll
        for (int v = 0; v < NV; ++v) key[v] = key_of(quick_score(false, l[v], top, per_sum) + bias[v]);
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) key[v] = l[v] > -INFINITY ? key[v] : 0u;
}

// What follows is called for about one row in some thousands; it forms the row's numbers anew, so that they stay in registers
// elsewhere.
// The 32-bit keys of row `row`.
template <int NV>
__device__ __forceinline__ void keys_again(const RouteArgs &a, const Shape &sh, int64_t row, int lane, float top, float per_sum,
                                           uint32_t (&key)[NV]) {
    float l[NV], bias[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int e = lane * sh.c + v;
        const bool real = v < sh.c && e < a.r.n_experts;
        l[v] = real ? load_logit(a, row * a.stride + e) : -INFINITY;
        bias[v] = real && a.bias ? a.bias[e] : 0.f;
    }
    keys_of(a, a.r.score == ENGRAM_SCORE_SOFTMAX, l, bias, top, per_sum, key);
}
// The row's choices on all its scores in 64 bits.
template <int NV>
__device__ __noinline__ int choose_all(const RouteArgs &a, int64_t row, int lane) {
    const Shape sh = shape_of(a.r);
    uint64_t key[NV], group[NV], least = 0;
    double s[NV], top = -INFINITY, sum = 0;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int e = lane * sh.c + v;
        s[v] = v < sh.c && e < a.r.n_experts ? (double)load_logit(a, row * a.stride + e) : -INFINITY;
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
        const bool masked = s[v] == -INFINITY;
        const double p = soft ? exp(s[v] - top) / sum : 1. / (1. + exp(-s[v]));
        key[v] = masked ? 0 : key_of(a.bias ? p + (double)a.bias[lane * sh.c + v] : s[v]);
        group[v] = masked ? 0 : a.bias || a.r.group_best == 1 ? key[v] : key_of(p);
    }
    float part;
    int id;
    if (a.r.top_groups < a.r.n_groups)
        mask_groups(sh, keep_groups(a, group_sums(a, sh, group, lane, part), lane), lane, key);
    choose_of<false>(a, sh, row, key, true, lane, id, least);
    return id;
}
// The groups that stay, by 64-bit scores of each group's experts that may be among its two largest.  0: too many of them.
template <int NV>
__device__ __noinline__ unsigned groups_again(const RouteArgs &a, int64_t row, int lane, float top, float per_sum) {
    const Shape sh = shape_of(a.r);
    const engram_router &r = a.r;
    uint32_t key[NV];
    keys_again(a, sh, row, lane, top, per_sum, key);
#pragma unroll
    for (int v = 0; v < NV; ++v) key[v] = group_key32(a, r.score == ENGRAM_SCORE_SOFTMAX, key[v], top, per_sum);
    unsigned want = 0;
    // of keys at lo .. hi - 1 those that may be among the group's two largest, of which the 32-bit ones are first and second
    auto mark = [&](int lo, int hi, uint32_t first, uint32_t second) {
        const uint32_t low = second && r.group_best == 2 ? second : first;
        if (!low) return;
        const float x = of_key(low), from = x - kTol * fmaxf(1.f, fabsf(x));
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (v >= lo && v < hi && key[v] && of_key(key[v]) >= from) want |= 1u << v;
    };
    if (sh.lanes) {
        uint32_t first = 0, second = 0;
#pragma unroll
        for (int v = 0; v < NV; ++v) two_best(first, second, key[v], 0u);
        two_best_of_lanes(first, second, sh.lanes);
        mark(0, NV, first, second);
    } else {
#pragma unroll 1
        for (int g = 0; g < r.n_groups; ++g) {
            const int lo = g * sh.size - lane * sh.c, hi = lo + sh.size;
            uint32_t first = 0, second = 0;
#pragma unroll
            for (int v = 0; v < NV; ++v) two_best(first, second, v >= lo && v < hi ? key[v] : 0u, 0u);
            two_best_of_lanes(first, second, 32);
            mark(lo, hi, first, second);
        }
    }
    int e;
    if (!one_a_lane(sh, want, lane, e)) return 0;
    const uint64_t mine = e >= 0 ? key_of(score64(a, row, e, top)) : 0;
    uint64_t sums = 0;                               // lane g: group g's
#pragma unroll 1
    for (int g = 0; g < r.n_groups; ++g) {
        uint64_t x = e >= 0 && e / sh.size == g ? mine : 0;
        const uint64_t first = warp_max(x);
        if (lane == __ffs(__ballot_sync(kAll, x == first)) - 1) x = 0;
        const uint64_t second = warp_max(x);
        if (lane == g) sums = sum_of(r.group_best, first, second);
    }
    return keep_groups(a, sums, lane);
}
// The choices among the groups `kept`, by 64-bit scores of the experts that may be among them: from `least`, the 32-bit key behind the
// last choice, on.  -2: too many.
template <int NV>
__device__ __noinline__ int experts_again(const RouteArgs &a, int64_t row, int lane, float top, float per_sum, unsigned kept, uint32_t least) {
    const Shape sh = shape_of(a.r);
    uint32_t key[NV];
    keys_again(a, sh, row, lane, top, per_sum, key);
    if (a.r.top_groups < a.r.n_groups) mask_groups(sh, kept, lane, key);
    const float x = of_key(least), from = least ? x - kTol * fmaxf(1.f, fabsf(x)) : -INFINITY;   // 0: none is left behind them
    unsigned want = 0;
#pragma unroll
    for (int v = 0; v < NV; ++v)
        if (key[v] && of_key(key[v]) >= from) want |= 1u << v;
    int e, id = -1;
    if (!one_a_lane(sh, want, lane, e)) return -2;
    uint64_t mine = e >= 0 ? key_of(score64(a, row, e, top)) : 0;
#pragma unroll 1
    for (int j = 0; j < a.r.top_k; ++j) {
        const uint64_t most = warp_max(mine);
        if (!most) break;
        const int g = __ffs(__ballot_sync(kAll, mine == most)) - 1, f = __shfl_sync(kAll, e, g);
        if (lane == j) id = f;
        if (lane == g) mine = 0;
    }
    return id;
}

// A lane's keys with their places (the lower the larger), in falling order: an odd-even merge of powers of two.
template <int NV>
__device__ __forceinline__ void sort_falling(uint64_t (&s)[NV]) {
#pragma unroll
    for (int p = 1; p < NV; p <<= 1)
#pragma unroll
        for (int k = p; k > 0; k >>= 1)
#pragma unroll
            for (int j = k % p; j + k < NV; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if (i + j + k < NV && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                        const uint64_t x = s[i + j], y = s[i + j + k];
                        const bool swap = x < y;
                        s[i + j] = swap ? y : x;
                        s[i + j + k] = swap ? x : y;
                    }
}

__device__ __forceinline__ void sort_falling(uint32_t (&s)[1]) {}
template <int NV>
__device__ __forceinline__ void sort_falling(uint32_t (&s)[NV]) {
#pragma unroll
    for (int p = 1; p < NV; p <<= 1)
#pragma unroll
        for (int k = p; k > 0; k >>= 1)
#pragma unroll
            for (int j = k % p; j + k < NV; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if (i + j + k < NV && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                        const uint32_t x = s[i + j], y = s[i + j + k];
                        s[i + j] = max(x, y);
                        s[i + j + k] = min(x, y);
                    }
}

// Token `row` with the logits l: its ids and weights, one choice a lane.  PACKED: a key's last bits give way to its place in the lane (scores with a
// bias, for which kTol allows; logits of 16 bits, which leave them alone), so that a lane sorts words of 32 bits: half the instructions.
template <int NV, bool PACKED>
__device__ __forceinline__ int route_row(const RouteArgs &a, const Shape &sh, const float (&bias)[NV], float (&l)[NV], int64_t row,
                                         int lane) {
    const engram_router &r = a.r;
    const bool soft = r.score == ENGRAM_SCORE_SOFTMAX, grouped = r.top_groups < r.n_groups, exact = !a.bias;
    float top = -INFINITY, sum = 0.f, per_sum = 0.f;
    bool nan = false;
#pragma unroll
    for (int v = 0; v < NV; ++v) nan |= l[v] != l[v];
    if (soft) {
#pragma unroll
        for (int v = 0; v < NV; ++v) top = fmaxf(top, l[v]);     // NaN gives way
        top = of_key(__reduce_max_sync(kAll, key_of(top)));
        nan |= top == INFINITY;
#pragma unroll
        for (int v = 0; v < NV; ++v) sum += l[v] > -INFINITY ? expf(l[v] - top) : 0.f;
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
        per_sum = 1.f / sum;
    }
    nan = __any_sync(kAll, nan);
    uint32_t key[NV], least = 0;
    keys_of(a, soft, l, bias, top, per_sum, key);
    // a softmax beside a bias needs its divisor in 64 bits, too: all scores
    bool all = false;
    unsigned kept = 0xFFFFFFFFu;
    auto settle_groups = [&](uint32_t mine, float part) {
        kept = keep_groups(a, mine, lane);
        // (logits alone are ordered exactly)
        if ((exact && r.group_best == 1) || sure_of_groups(mine, part, kept, tol_of<NV>(a), lane)) return;
        all = (soft && a.bias) || !(kept = groups_again<NV>(a, row, lane, top, per_sum));
    };
    if (grouped && (!sh.lanes || NV > 8)) {
        uint32_t group[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) group[v] = group_key32(a, soft, key[v], top, per_sum);
        float part;
        const uint32_t mine = group_sums(a, sh, group, lane, part);
        settle_groups(mine, part);
        mask_groups(sh, kept, lane, key);
    }
    int id;
    bool chosen;
    if (PACKED) {
        constexpr uint32_t kPlace = NV <= 8 ? NV - 1 : 0;
        uint32_t s[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) s[v] = key[v] ? (key[v] & ~kPlace) | (kPlace - v) : 0u;
        sort_falling(s);
        if (grouped && sh.lanes) {
            // (a 16-bit logit's key has its last bits all 0, or all 1 if it is negative)
            auto value = [&](uint32_t k) { return exact && k && (int)k >= 0 ? k | kPlace : k & ~kPlace; };
            uint32_t first = group_key32(a, soft, value(s[0]), top, per_sum);
            uint32_t second = NV > 1 ? group_key32(a, soft, value(s[NV > 1]), top, per_sum) : 0u;
            two_best_of_lanes(first, second, sh.lanes);
            const uint32_t mine = __shfl_sync(kAll, sum_of(r.group_best, first, second), lane * sh.lanes & 31);
            const float part = __shfl_sync(kAll, part_of(r.group_best, first, second), lane * sh.lanes & 31);
            settle_groups(lane < r.n_groups ? mine : 0u, part);
            const bool out = !(kept >> min(31, lane / sh.lanes) & 1);
#pragma unroll
            for (int v = 0; v < NV; ++v) s[v] = out ? 0u : s[v];
        }
        uint32_t m = s[0] & ~kPlace;                 // equal ones: the lowest lane's, and in a lane the lowest place's
        int at = kPlace - (s[0] & kPlace);
        auto next = [&](bool mine) {
#pragma unroll
            for (int v = 0; v < NV; ++v) s[v] = mine ? v + 1 < NV ? s[(v + 1) % NV] : 0u : s[v];
            m = s[0] & ~kPlace;
            at = kPlace - (s[0] & kPlace);
        };
        chosen = choose<true>(a, sh, row, m, at, next, exact, tol_of<NV>(a), lane, id, least);
    } else if (NV <= 8) {
        uint64_t s[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) s[v] = (uint64_t)key[v] << 32 | (uint32_t)(NV - 1 - v);
        sort_falling(s);
        if (grouped && sh.lanes) {
            uint32_t first = group_key32(a, soft, (uint32_t)(s[0] >> 32), top, per_sum);
            uint32_t second = NV > 1 ? group_key32(a, soft, (uint32_t)(s[NV > 1] >> 32), top, per_sum) : 0u;
            two_best_of_lanes(first, second, sh.lanes);
            const uint32_t mine = __shfl_sync(kAll, sum_of(r.group_best, first, second), lane * sh.lanes & 31);
            const float part = __shfl_sync(kAll, part_of(r.group_best, first, second), lane * sh.lanes & 31);
            settle_groups(lane < r.n_groups ? mine : 0u, part);
            const bool out = !(kept >> min(31, lane / sh.lanes) & 1);
#pragma unroll
            for (int v = 0; v < NV; ++v) s[v] = out ? (uint32_t)s[v] : s[v];
        }
        // keys in order, their places four bits each
        uint32_t order = 0;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            key[v] = (uint32_t)(s[v] >> 32);
            order |= (NV - 1 - (uint32_t)s[v]) << (4 * v);
        }
        uint32_t m = key[0];
        int at = order & 15;
        auto next = [&](bool mine) {
#pragma unroll
            for (int v = 0; v < NV; ++v) key[v] = mine ? v + 1 < NV ? key[(v + 1) % NV] : 0 : key[v];
            order = mine ? order >> 4 : order;
            m = key[0];
            at = order & 15;
        };
        chosen = choose<true>(a, sh, row, m, at, next, exact, tol_of<NV>(a), lane, id, least);
    } else {
        chosen = choose_of<true>(a, sh, row, key, exact, lane, id, least);
    }
    if (!chosen && !all) {
        if (soft)
            all = true;
        else
            all = (id = experts_again<NV>(a, row, lane, top, per_sum, kept, least)) == -2;
    }
    if (all) id = choose_all<NV>(a, row, lane);
    float s = id >= 0 ? score32(soft, load_logit(a, row * a.stride + id), top, sum) : 0.f;
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

// ---- four tokens a warp ----
// Eight lanes a token, C consecutive experts a lane: what takes all lanes' attention above (maxima, votes) is paid once for four tokens.
// A key gives five bits to its place, so more rows than above are in doubt; those are formed again as above.
// Two scores, x the one of the larger size, are told apart by this: 8e-7 max(1, |x|) (see kTol), and C units of its last place (keys lose their
// last bits towards minus infinity, so of two negative ones the smaller's unit counts, which may be twice the other's).  Half of it bounds the
// error of a value in the middle of those that its key may stand for.
template <int C>
__device__ __forceinline__ float quad_tol(float x) {
    return fmaf(__uint_as_float(__float_as_uint(x) & 0x7F800000u), C * 0x1p-23f, 1e-6f * fmaxf(1.f, fabsf(x)));
}
template <int NV>
__device__ __noinline__ int row_again(const RouteArgs &a, int64_t row, int lane) {
    const Shape sh = shape_of(a.r);
    float l[NV], bias[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) bias[v] = a.bias ? __ldg(a.bias + lane * NV + v) : 0.f;
    load_row<NV>(a, NV, wide_rows<NV>(a), row, lane, l);
    return route_row<NV, true>(a, sh, bias, l, row, lane);
}
// Whether `a` has such rows (64, 128 or 256 experts, sigmoid, groups of whole lanes, up to 8 choices, keys that may lose bits, aligned) and enough of
// them, four a warp in all blocks: 16384 tokens of 256 experts, without lists, 21.2 us for 30.2; 4096 tokens some 4 more.
inline bool quads_fit(const RouteArgs &a, int blocks, int C) {
    const int size = a.type == ENGRAM_T_F32 ? 4 : 2;
    return a.tokens >= 64 * blocks && blocks > 1 && a.r.n_experts == 8 * C && a.r.n_groups <= 8 && 8 % a.r.n_groups == 0 &&
           a.r.top_k <= 8 && a.r.score == ENGRAM_SCORE_SIGMOID && (a.bias || a.type != ENGRAM_T_F32) && a.stride * size % 16 == 0 && reinterpret_cast<uintptr_t>(a.logits) % 16 == 0;
}
// Tokens t .. t + 3 (before hi); bias: [C / 4][8 lanes][4] in shared memory.  A lane's choice: lane j of a token's eight, choice j.
template <int C>
__device__ __forceinline__ int route_quad(const RouteArgs &a, const float4 *bias, int64_t t, int64_t hi, int lane) {
    constexpr uint32_t kPlace = C - 1;
    const engram_router &r = a.r;
    const int sub = lane & 7, seg = lane >> 3, k = r.top_k;
    const int64_t row = t + seg < hi ? t + seg : hi - 1;
    const bool exact = !a.bias;
    uint32_t key[C];
    bool nan = false;
    {
        const int64_t at = row * a.stride + sub * C;
#pragma unroll
        for (int v = 0; v < C; v += 8) {
            float l[8];
            if (a.type == ENGRAM_T_F32) {
                const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(a.logits) + at + v);
                const float4 x = __ldg(p), y = __ldg(p + 1);
                l[0] = x.x, l[1] = x.y, l[2] = x.z, l[3] = x.w, l[4] = y.x, l[5] = y.y, l[6] = y.z, l[7] = y.w;
            } else {
                const uint4 raw = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.logits) + at + v));
                if (a.type == ENGRAM_T_BF16)
                    load8<ENGRAM_T_BF16>(&raw, 0, l);
                else
                    load8<ENGRAM_T_F16>(&raw, 0, l);
            }
            float b[8] = {};
            if (a.bias) {
                const float4 x = bias[v / 4 * 8 + sub], y = bias[(v / 4 + 1) * 8 + sub];
                b[0] = x.x, b[1] = x.y, b[2] = x.z, b[3] = x.w, b[4] = y.x, b[5] = y.y, b[6] = y.z, b[7] = y.w;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                nan |= l[i] != l[i];
                const uint32_t u = key_of(a.bias ? quick_score(false, l[i], 0.f, 0.f) + b[i] : l[i]);
                key[v + i] = l[i] > -INFINITY ? (u & ~kPlace) | (kPlace - (v + i)) : 0u;
            }
        }
    }
    nan = (__ballot_sync(kAll, nan) >> (8 * seg) & 0xFF) != 0;
    uint32_t m = 0, second = 0;                      // the lane's largest two
#pragma unroll
    for (int v = 0; v < C; ++v) {
        second = max(second, min(m, key[v]));
        m = max(m, key[v]);
    }
    bool doubt = false, doubt_group = false;
    unsigned groups = 0xFF;                          // this token's lanes that stay
    if (r.top_groups < r.n_groups) {
        const int lanes = 8 / r.n_groups;
        // (a 16-bit logit's key has its last bits all 0, or all 1 if it is negative)
        auto value = [&](uint32_t x) { return !x ? 0u : !exact ? (x & ~kPlace) | C / 2 : (int)x >= 0 ? x | kPlace : x & ~kPlace; };
        uint32_t x1 = group_key32(a, false, value(m), 0.f, 0.f), x2 = group_key32(a, false, value(second), 0.f, 0.f);
        two_best_of_lanes(x1, x2, lanes);
        const uint32_t mine = sum_of(r.group_best, x1, x2);
        // of equal sums the lower group; a lane asks for those of the token's other lanes
        int before = 0;
#pragma unroll
        for (int o = 1; o < 8; ++o) {
            const uint32_t other = __shfl_xor_sync(kAll, mine, o);
            if ((sub ^ o) / lanes != sub / lanes) before += other > mine || (other == mine && (sub ^ o) < sub);
        }
        const bool kept = before < r.top_groups * lanes;
        if (!(exact && r.group_best == 1)) {         // logits alone are ordered exactly
            const bool both = r.group_best == 2 && x2;
            const float s = of_key(mine), err = mine ? 0.5f * (quad_tol<C>(of_key(x1)) + (both ? quad_tol<C>(of_key(x2)) : 0.f)) : 0.f;
            float least = mine && kept ? s - err : INFINITY, most = mine && !kept ? s + err : -INFINITY;
#pragma unroll
            for (int o = 4; o; o >>= 1) {
                least = fminf(least, __shfl_xor_sync(kAll, least, o));
                most = fmaxf(most, __shfl_xor_sync(kAll, most, o));
            }
            doubt_group = least <= most;
        }
        m = kept ? m : 0u;
        groups = __ballot_sync(kAll, kept) >> (8 * seg) & 0xFF;
    }
    // from m to the largest key below it: of the differences from m modulo 2^32 the largest, for they are larger for those below m (0 is one)
    // than for others
    auto next_key = [&](uint32_t m) {
        uint32_t next = 0u - m;
#pragma unroll
        for (int v = 0; v < C; v += 2) next = __vimax3_u32(next, key[v] - m, key[v + 1] - m);
        return next;
    };
    int id = -1;
    uint32_t mine = 0, least = 0;
#pragma unroll 1
    for (int j = 0; j <= k; ++j) {
        const uint32_t x = m & ~kPlace;
        uint32_t top = x;
#pragma unroll
        for (int o = 4; o; o >>= 1) top = max(top, __shfl_xor_sync(kAll, top, o));
        const int first = __ffs(__ballot_sync(kAll, x == top) >> (8 * seg) & 0xFF) - 1;   // lower lanes hold lower experts
        const int e = __shfl_sync(kAll, sub * C + (int)(kPlace - (m & kPlace)), 8 * seg + first);
        if (j == k) {
            least = top;
        } else if (sub == j && top) {
            id = e, mine = top;
        }
        if (j == k) break;
        const uint32_t next = next_key(m);
        m = sub == first && top ? m + next : m;
    }
    if (!exact) {                                    // as in choose()
        const uint32_t after = __shfl_down_sync(kAll, mine, 1);
        const int other = __shfl_down_sync(kAll, id, 1);
        if (sub < k - 1 && mine && after) {
            const float x = of_key(mine), y = of_key(after);
            doubt = x - y <= quad_tol<C>(fmaxf(fabsf(x), fabsf(y))) && !same_numbers(a, row, id, other);
        }
        const uint32_t last = __shfl_sync(kAll, mine, 8 * seg + k - 1);
        const float x = of_key(last);                // (of those that are near enough none is of a larger size than the inner sum)
        const uint32_t from = last ? key_of(x - quad_tol<C>(fabsf(x) + quad_tol<C>(x))) : 0xFFFFFFFFu;
        while (__any_sync(kAll, m >= from)) {
            const int last_id = __shfl_sync(kAll, id, 8 * seg + k - 1);
            if (m >= from) {
                doubt |= !same_numbers(a, row, last_id, sub * C + (int)(kPlace - (m & kPlace)));
                m += next_key(m);
            }
        }
    }
    const bool real = t + seg < hi;
    unsigned doubts = __ballot_sync(kAll, (doubt || doubt_group) && real);
#pragma unroll 1
    while (doubts) {
        const int at = (__ffs(doubts) - 1) >> 3;
        doubts &= ~(0xFFu << (8 * at));
        // the token's groups as the others have them, a bit a group
        const unsigned lanes_in = __shfl_sync(kAll, groups, 8 * at);
        unsigned kept = 0;
        for (int g = 0; g < r.n_groups; ++g) kept |= (lanes_in >> (g * 8 / r.n_groups) & 1) << g;
        const uint32_t from = __shfl_sync(kAll, least, 8 * at);
        const bool same = !__shfl_sync(kAll, (int)doubt_group, 8 * at) || groups_again<C / 4>(a, t + at, lane, 0.f, 0.f) == kept;
        if (same && !__any_sync(kAll, doubt && seg == at)) continue;
        int again = same ? experts_again<C / 4>(a, t + at, lane, 0.f, 0.f, kept, from) : -2;
        if (__any_sync(kAll, again == -2)) again = row_again<C / 4>(a, t + at, lane);
        __syncwarp();
        again = __shfl_sync(kAll, again, sub);
        if (seg == at) id = sub < k ? again : -1;
    }
    float s = id >= 0 ? score32(false, load_logit(a, row * a.stride + id), 0.f, 0.f) : 0.f;
    if (r.renormalise) {
        float u = s;
#pragma unroll
        for (int o = 4; o; o >>= 1) u += __shfl_xor_sync(kAll, u, o);
        s = s / (u + 1e-20f);
    }
    if (real && sub < k) {
        a.ids[row * k + sub] = id;
        a.weights[row * k + sub] = nan ? __int_as_float(0x7FFFFFFF) : id < 0 ? 0.f : s * r.scale;
    }
    return real ? id : -1;
}

// Tokens of warp `w` of block b.
__device__ __forceinline__ void warp_tokens(const RouteArgs &a, int b, int blocks, int w, int64_t &lo, int64_t &hi) {
    const int warps = blockDim.x >> 5;
    const int64_t first = (int64_t)a.tokens * b / blocks, n = (int64_t)a.tokens * (b + 1) / blocks - first;
    lo = first + n * w / warps;
    hi = first + n * (w + 1) / warps;
}

// Exclusive sums over `n` values of v[], all threads of the block; v[n] gets the total.  part: 32 ints.
__device__ __forceinline__ void block_scan(int *v, int n, int *part) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    int carry = 0;
    for (int i0 = 0; i0 < n; i0 += (int)blockDim.x) {
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
        for (int w = 0; w < warps; ++w) {
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

// Choices of four tokens from t on, one a lane.
__device__ __forceinline__ void four_rows(const RouteArgs &a, int64_t t, int64_t hi, int lane, int (&id)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) id[i] = lane < a.r.top_k && t + i < hi ? a.ids[(t + i) * a.r.top_k + lane] : -1;
}

// counts: [warps][E] of the block's warps, turned into the first position of each; first: position of the block's first pair
// of each expert.  Then the warp's pairs to their places.
__device__ __forceinline__ void place_pairs(const RouteArgs &a, int *counts, const int *first, int64_t lo, int64_t hi) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5, E = a.r.n_experts, k = a.r.top_k;
    for (int e = tid; e < E; e += blockDim.x) {
        int at = first[e];
        for (int w = 0; w < warps; ++w) {
            const int n = counts[w * E + e];
            counts[w * E + e] = at;
            at += n;
        }
    }
    __syncthreads();
    int *mine = counts + warp * E;
    for (int64_t t = lo; t < hi; t += 4) {
        int id[4];
        four_rows(a, t, hi, lane, id);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (id[i] >= 0) a.pairs[mine[id[i]]++] = (int)((t + i) * k + lane);
            __syncwarp();
        }
    }
}

// One block: everything.  Several: ids, weights and the block's counts (ws).
template <int NV, bool PACKED>
__global__ void __launch_bounds__(NV <= 8 ? 1024 : 512) route_kernel(const __grid_constant__ RouteArgs a) {
    extern __shared__ int smem[];
    __shared__ int part[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5, E = a.r.n_experts;
    int *counts = smem, *mine = counts + warp * E, *first = counts + warps * E;
    int64_t lo, hi;
    warp_tokens(a, blockIdx.x, gridDim.x, warp, lo, hi);
    if (a.offsets)
        for (int e = lane; e < E; e += 32) mine[e] = 0;
    __syncwarp();
    const Shape sh = shape_of(a.r);
    const bool wide = wide_rows<NV>(a);
    float bias[NV], next[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v)
        bias[v] = a.bias && v < sh.c && lane * sh.c + v < E ? __ldg(a.bias + lane * sh.c + v) : 0.f;
    if (lo < hi) load_row<NV>(a, sh.c, wide, lo, lane, next);
    for (int64_t t = lo; t < hi; ++t) {
        float l[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) l[v] = next[v];
        if (t + 1 < hi) load_row<NV>(a, sh.c, wide, t + 1, lane, next);
        const int id = route_row<NV, PACKED>(a, sh, bias, l, t, lane);
        if (a.offsets) count_row(a, mine, id, lane);
    }
    if (!a.offsets) return;
    __syncthreads();
    if (gridDim.x > 1) {
        for (int e = tid; e < E; e += blockDim.x) {
            int n = 0;
            for (int w = 0; w < warps; ++w) n += counts[w * E + e];
            a.ws[(int64_t)blockIdx.x * E + e] = n;
        }
        return;
    }
    for (int e = tid; e < E; e += blockDim.x) {
        int n = 0;
        for (int w = 0; w < warps; ++w) n += counts[w * E + e];
        first[e] = n;
    }
    __syncthreads();
    block_scan(first, E, part);
    for (int e = tid; e <= E; e += blockDim.x) a.offsets[e] = first[e];
    place_pairs(a, counts, first, lo, hi);
}

// Several blocks, four tokens a warp: as route_kernel.
template <int C>
__global__ void __launch_bounds__(512) route_quads_kernel(const __grid_constant__ RouteArgs a) {
    extern __shared__ int smem[];
    __shared__ float4 bias[2 * C];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5, E = 8 * C;
    int *counts = smem, *mine = counts + warp * E;
    int64_t lo, hi;
    warp_tokens(a, blockIdx.x, gridDim.x, warp, lo, hi);
    if (a.offsets)
        for (int e = lane; e < E; e += 32) mine[e] = 0;
    if (a.bias)
        for (int e = tid; e < E; e += blockDim.x)
            reinterpret_cast<float *>(bias)[((e % C) / 4 * 8 + e / C) * 4 + e % 4] = __ldg(a.bias + e);
    __syncthreads();
    for (int64_t t = lo; t < hi; t += 4) {
        const int id = route_quad<C>(a, bias, t, hi, lane);
        if (!a.offsets) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) count_row(a, mine, lane >> 3 == i ? id : -1, lane);
    }
    if (!a.offsets) return;
    __syncthreads();
    for (int e = tid; e < E; e += blockDim.x) {
        int n = 0;
        for (int w = 0; w < warps; ++w) n += counts[w * E + e];
        a.ws[(int64_t)blockIdx.x * E + e] = n;
    }
}

__global__ void __launch_bounds__(1024) route_lists_kernel(const RouteArgs a) {
    extern __shared__ int smem[];
    __shared__ int part[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5, E = a.r.n_experts;
    int *counts = smem, *mine = counts + warp * E, *first = counts + warps * E, *before = first + E + 1;
    int64_t lo, hi;
    warp_tokens(a, blockIdx.x, gridDim.x, warp, lo, hi);
    for (int e = lane; e < E; e += 32) mine[e] = 0;
    for (int e = tid; e < E; e += blockDim.x) first[e] = before[e] = 0;
    __syncthreads();
    griddep_wait();
    int id[4];
    four_rows(a, lo, hi, lane, id);
    // the blocks' counts of an expert, by as many threads as there are for each
    const int parts = max(1, (int)blockDim.x / E), blocks = gridDim.x;
    for (int i = tid; i < parts * E; i += blockDim.x) {
        const int e = i % E, part_no = i / E;
        int n = 0, sum = 0;
#pragma unroll 19
        for (int b = blocks * part_no / parts; b < blocks * (part_no + 1) / parts; ++b) {
            const int c = a.ws[(int64_t)b * E + e];
            n += b < (int)blockIdx.x ? c : 0;
            sum += c;
        }
        atomicAdd(first + e, sum);                   // whole numbers: in any order
        atomicAdd(before + e, n);
    }
    for (int64_t t = lo; t < hi; t += 4) {
        if (t > lo) four_rows(a, t, hi, lane, id);
#pragma unroll
        for (int i = 0; i < 4; ++i) count_row(a, mine, id[i], lane);
    }
    __syncthreads();
    block_scan(first, E, part);
    if (blockIdx.x == 0)
        for (int e = tid; e <= E; e += blockDim.x) a.offsets[e] = first[e];
    __syncthreads();
    for (int e = tid; e < E; e += blockDim.x) first[e] += before[e];
    __syncthreads();
    place_pairs(a, counts, first, lo, hi);
}

size_t smem_bytes(int E, int warps) { return ((size_t)(warps + 2) * E + 2) * sizeof(int); }

// Once a device: dynamic shared memory for the most experts.
cudaError_t allow_smem(void (*kernel)(const RouteArgs), bool (&done)[64]) {
    static std::mutex mutex;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mutex);
    if (done[dev]) return cudaSuccess;
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes(kMaxExperts, 32));
    done[dev] = e == cudaSuccess;
    return e;
}

template <int NV, bool PACKED>
cudaError_t launch_kernel(const RouteArgs &a, int blocks, int warps, cudaStream_t s) {
    static bool wide[64] = {};
    const cudaError_t e = allow_smem(route_kernel<NV, PACKED>, wide);
    if (e != cudaSuccess) return e;
    route_kernel<NV, PACKED><<<blocks, 32 * warps, a.offsets ? smem_bytes(a.r.n_experts, warps) : 0, s>>>(a);
    return cudaGetLastError();
}
template <int C>
cudaError_t launch_quads(const RouteArgs &a, int blocks, cudaStream_t s) {
    static bool wide[64] = {};
    const cudaError_t e = allow_smem(route_quads_kernel<C>, wide);
    if (e != cudaSuccess) return e;
    route_quads_kernel<C><<<blocks, 512, a.offsets ? smem_bytes(a.r.n_experts, 16) : 0, s>>>(a);
    return cudaGetLastError();
}
template <int NV>
cudaError_t launch_rows(const RouteArgs &a, int blocks, int warps, cudaStream_t s) {
    if (NV >= 2 && NV <= 8 && quads_fit(a, blocks, 4 * NV)) return launch_quads<(NV >= 2 && NV <= 8 ? 4 * NV : 8)>(a, blocks, s);
    if (NV <= 8 && (a.bias || a.type != ENGRAM_T_F32)) return launch_kernel<NV, NV <= 8>(a, blocks, warps, s);
    return launch_kernel<NV, false>(a, blocks, warps, s);
}

}  // namespace

size_t route_workspace_ints(int n_experts, int tokens) {
    const int b = route_blocks(n_experts, tokens);
    return b > 1 ? (size_t)b * n_experts : 0;
}

cudaError_t launch_route(const RouteArgs &a, cudaStream_t s) {
    const int E = a.r.n_experts, blocks = route_blocks(E, a.tokens);
    // no more warps than tokens, but the eight that make short work of the lists
    const int most = route_warps(E), each = (a.tokens + blocks - 1) / blocks, warps = each > most ? most : each < 8 ? 8 : each;
    cudaError_t e;
    if (E <= 32)
        e = launch_rows<1>(a, blocks, warps, s);
    else if (E <= 64)
        e = launch_rows<2>(a, blocks, warps, s);
    else if (E <= 128)
        e = launch_rows<4>(a, blocks, warps, s);
    else if (E <= 256)
        e = launch_rows<8>(a, blocks, warps, s);
    else if (E <= 512)
        e = launch_rows<16>(a, blocks, warps, s);
    else
        e = launch_rows<32>(a, blocks, warps, s);
    if (e != cudaSuccess || blocks == 1 || !a.offsets) return e;
    static bool wide[64] = {};
    e = allow_smem(route_lists_kernel, wide);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    // a block's tokens do not depend on its warps; the more blocks, the more threads share their counts
    const int list_warps = blocks > 32 ? 32 : warps;
    cfg.blockDim = dim3(32 * list_warps);
    cfg.dynamicSmemBytes = smem_bytes(E, list_warps);
    cfg.stream = s;
    cudaLaunchAttribute la[1];
    la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    la[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = la;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, route_lists_kernel, a);
}

}  // namespace engram
