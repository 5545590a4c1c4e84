// route_topk.cu -- top-k routing from router logits, and its gradient.
//
// Forward, for every token t with logits z[e]:
//   s_e = softmax(z)_e or 1 / (1 + exp(-z_e));   c_e = s_e + bias_e  (balance bias)
//   group value = sum of the two largest c of the group (of one where it has one)
//   ids = the k largest c among the topk_group groups of largest value, in
//         descending order, ties to the lowest index
//   w_i = s_ids[i] (divided by their sum when renormalised) * scale
//   gates[t, :] = 0 but for gates[t, ids[i]] = w_i
// Experts whose logit is -inf (or NaN) are never chosen; a token without k
// choosable experts has ids -1 and weights 0 behind them.
//
// One warp per token; a lane holds NJ = ceil(E / 32) neighbouring experts in
// registers, so the lowest lane of a tie is the lowest index.  The choice is made
// on order-preserving integer keys: one redux.max, one ballot per chosen expert.
//
// The choice is that of scores in 64 bits.  Scores in fp32 can order two experts wrongly whose true
// values differ by less than their rounding, so every gap that decides something
// (between neighbours of the k + 1 best, at the border of the chosen groups) is
// compared with a bound on that rounding; a token with a gap below it is
// chosen again from scores in 64 bits (a few tokens in a thousand).  The bound is absolute, so
// scores that lie close together are doubtful for most tokens: groups without a bias over
// saturated scores (32749 x 256, 8 groups, sigmoid: 48 us for normal logits of deviation 1.5,
// 135 at 4, 182 at 10; softmax 53, 56, 144; with a bias of 0.2 all of them 45 to 51).  Without
// bias and groups the scores grow with the logits, which are compared as they are.
//
// The renormalised weights are formed relative to the largest chosen logit: no
// sum of theirs underflows, however low the chosen logits are.
//
// Bound: reading the logits and writing the gates, T * E * (2 or 4) + T * E * 4 bytes, is
// the floor (10.6 us at 32749 tokens x 256 fp32 logits); the instructions of the choice take
// longer: 45 us there, 8 of 256 experts in 4 of 8 groups, 76 % of the issue slots
// (51 us before keys named their expert, 88 us with groups compared one by one).
// The gradient writes as many values as there are logits.  It reads the whole rows for plain
// softmax weights only, else the chosen logits: 16381 x 256 fp32, sigmoid, renormalised, 8 a
// token, then moves 22 MB, 3.4 us, and takes 8.1 us (with whole rows read the floor is 5.3).
// Every lane's zeros wait for the chain id -> logit -> exp -> sums.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>

#include "common.cuh"
#include "launch.h"

namespace bffn {

namespace {

constexpr int kTkWarps = 4;      // tokens per block
constexpr int kTkMaxE = 256;

__device__ __forceinline__ float tk_f32(float v) { return v; }
__device__ __forceinline__ float tk_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void tk_put(float* p, float v) { *p = v; }
__device__ __forceinline__ void tk_put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

template <int BYTES> struct TkVec;
template <> struct TkVec<2> { using type = uint16_t; };
template <> struct TkVec<4> { using type = uint32_t; };
template <> struct TkVec<8> { using type = uint2; };
template <> struct TkVec<16> { using type = uint4; };

// The lane's NJ neighbouring elements of a row of E (missing ones: `missing`).
// Rows of exactly 32 * NJ elements, NJ a power of two, are read in vectors (every
// lane's part is then aligned to its size, the row's base being 16-byte aligned).
template <int NJ, typename T>
__device__ __forceinline__ void tk_load(const T* row, int E, int lane, float missing, float (&v)[NJ]) {
    constexpr int kBytes = NJ * (int)sizeof(T);
    constexpr int kVec = kBytes < 16 ? kBytes : 16;
    if constexpr ((NJ & (NJ - 1)) == 0) {
        if (E == 32 * NJ) {
            using V = typename TkVec<kVec>::type;
            constexpr int kPer = kVec / (int)sizeof(T);
            alignas(16) T buf[NJ];
#pragma unroll
            for (int i = 0; i < kBytes / kVec; ++i)
                reinterpret_cast<V*>(buf)[i] = reinterpret_cast<const V*>(row + lane * NJ)[i];
            static_assert(kPer * (kBytes / kVec) == NJ, "whole vectors");
#pragma unroll
            for (int j = 0; j < NJ; ++j) v[j] = tk_f32(buf[j]);
            return;
        }
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const int e = lane * NJ + j;
        v[j] = e < E ? tk_f32(row[e]) : missing;
    }
}

template <int NJ, typename T>
__device__ __forceinline__ void tk_store(T* row, int E, int lane, const float (&v)[NJ]) {
    constexpr int kBytes = NJ * (int)sizeof(T);
    constexpr int kVec = kBytes < 16 ? kBytes : 16;
    if constexpr ((NJ & (NJ - 1)) == 0) {
        if (E == 32 * NJ) {
            using V = typename TkVec<kVec>::type;
            alignas(16) T buf[NJ];
#pragma unroll
            for (int j = 0; j < NJ; ++j) tk_put(buf + j, v[j]);
#pragma unroll
            for (int i = 0; i < kBytes / kVec; ++i)
                reinterpret_cast<V*>(row + lane * NJ)[i] = reinterpret_cast<const V*>(buf)[i];
            return;
        }
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const int e = lane * NJ + j;
        if (e < E) tk_put(row + e, v[j]);
    }
}

// Order-preserving integer keys, 0 for "not choosable" (below every number's key).
struct Key32 {
    using Real = float;
    using Bits = uint32_t;
    __device__ static Bits of(float v) {
        const uint32_t u = __float_as_uint(v);
        return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    }
    __device__ static float value(Bits k) {
        return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
    }
    __device__ static Bits warp_max(Bits k) { return __reduce_max_sync(0xffffffffu, k); }
};
struct Key64 {
    using Real = double;
    using Bits = unsigned long long;
    __device__ static Bits of(double v) {
        const unsigned long long u = (unsigned long long)__double_as_longlong(v);
        return (u >> 63) ? ~u : (u | (1ull << 63));
    }
    __device__ static double value(Bits k) {
        return __longlong_as_double((long long)((k >> 63) ? (k & ~(1ull << 63)) : ~k));
    }
    __device__ static Bits warp_max(Bits k) {
        const uint32_t hi = (uint32_t)(k >> 32);
        const uint32_t mh = __reduce_max_sync(0xffffffffu, hi);
        const uint32_t ml = __reduce_max_sync(0xffffffffu, hi == mh ? (uint32_t)k : 0u);
        return ((Bits)mh << 32) | ml;
    }
};

// Scores for the choice.  In fp32 from the fast exponential and division: off by less than
// 1e-6 (s <= 1, and the exponent's error of 2^-24 |z| comes in times s (1 - s) or s), a
// quarter of the gap at which the choice is made again in 64 bits.
__device__ __forceinline__ float tk_exp(float v) { return __expf(v); }
__device__ __forceinline__ double tk_exp(double v) { return exp(v); }
__device__ __forceinline__ float tk_sigmoid(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }
__device__ __forceinline__ double tk_sigmoid(double z) { return 1.0 / (1.0 + exp(-z)); }

template <typename R>
__device__ __forceinline__ R tk_warp_sum(R v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

struct TkArgs {
    const float* bias;     // [E] or nullptr
    int T, E, k;
    int sigmoid;           // scores: 1 sigmoid, 0 softmax
    int n_group, topk_group, per;   // experts per group = E / n_group
    int lane_groups;       // groups are whole lanes, a power of two of them
    int renorm;
    float scale;
    float* gates;          // [T, E] or nullptr
    int32_t* ids;          // [T, k]
    float* weights;        // [T, k]
};

// Keys of the choice from the logits (softmax: the largest is m), in K::Real arithmetic.
template <int NJ, class K>
__device__ __forceinline__ void tk_choice_keys(const TkArgs& a, const float (&z)[NJ], const float* brow, int lane,
                                               typename K::Bits (&key)[NJ], float m) {
    using R = typename K::Real;
    R s[NJ];
    if (a.sigmoid) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) s[j] = tk_sigmoid((R)z[j]);
    } else {
        R part = R(0);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            s[j] = z[j] > -INFINITY ? tk_exp((R)z[j] - (R)m) : R(0);
            part += s[j];
        }
        const R total = tk_warp_sum(part);
        const R inv = total > R(0) ? R(1) / total : R(0);
#pragma unroll
        for (int j = 0; j < NJ; ++j) s[j] *= inv;
    }
    float b[NJ];
    if (brow != nullptr) {
        tk_load<NJ>(brow, a.E, lane, 0.f, b);
    } else {
#pragma unroll
        for (int j = 0; j < NJ; ++j) b[j] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const R c = s[j] + (R)b[j];
        key[j] = (z[j] > -INFINITY && c > -INFINITY) ? K::of(c) : typename K::Bits(0);
    }
}

// How much larger the two parts of a group's value are than the value itself (0 unless their
// signs differ): their rounding stays while they cancel, so the doubtful gap grows with the
// most of it in any group.
__device__ __forceinline__ float tk_cancelled(float v1, float v2) {
    return (v1 > 0.f) != (v2 > 0.f) ? 2.f * fminf(fabsf(v1), fabsf(v2)) : 0.f;
}
__device__ __forceinline__ float tk_warp_most(float v) {   // (of numbers >= 0)
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
}

// tk_keep_groups for groups that are whole lanes, a power of two of them (32 / n_group, as with
// 32 NJ experts in a power of two of groups): the two largest keys of a group meet in
// butterflies.  Same result.
template <int NJ>
__device__ __forceinline__ bool tk_keep_lane_groups(const TkArgs& a, int lane, uint32_t (&key)[NJ]) {
    uint32_t b1 = 0, b2 = 0;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        b2 = max(b2, min(b1, key[j]));
        b1 = max(b1, key[j]);
    }
    const int L = 32 / a.n_group;   // lanes per group
    for (int o = 1; o < L; o <<= 1) {
        const uint32_t c1 = __shfl_xor_sync(0xffffffffu, b1, o), c2 = __shfl_xor_sync(0xffffffffu, b2, o);
        b2 = max(min(b1, c1), max(b2, c2));
        b1 = max(b1, c1);
    }
    // the group's value, in its first lane
    uint32_t gv = 0;
    float lost = 0.f;
    if (b1 != 0 && (lane & (L - 1)) == 0) {
        const float v1 = Key32::value(b1), v2 = b2 != 0 ? Key32::value(b2) : 0.f;
        gv = Key32::of(v1 + v2);
        lost = tk_cancelled(v1, v2);
    }
    lost = tk_warp_most(lost);
    uint32_t kept = 0;   // lanes of the kept groups
    const uint32_t lanes = L == 32 ? 0xffffffffu : (1u << L) - 1u;
    float last = 0.f;
    bool close = false;
    for (int n = 0; n <= a.topk_group && n < a.n_group; ++n) {
        const uint32_t m = Key32::warp_max(gv);
        if (m == 0) break;
        const float v = Key32::value(m);
        if (n == a.topk_group) {
            close = !(last - v > 8e-6f * (1.f + fabsf(v) + lost));
            break;
        }
        const int src = __ffs(__ballot_sync(0xffffffffu, gv == m)) - 1;
        if (lane == src) gv = 0;
        kept |= lanes << src;
        last = v;
    }
    if (!(kept >> lane & 1u)) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) key[j] = 0;
    }
    return close;
}

// Of the groups of `per` neighbouring experts, keep the topk_group of largest
// value: keys outside them become 0.  Returns whether the border between kept and
// dropped groups is nearer than the rounding of fp32 scores.
template <int NJ, class K>
__device__ __forceinline__ bool tk_keep_groups(const TkArgs& a, int lane, typename K::Bits (&key)[NJ],
                                               typename K::Bits* srow) {
    using Bits = typename K::Bits;
    using R = typename K::Real;
    // srow: the warp's row of keys; every group's value from it, lane g + 32 i for group g + 32 i
#pragma unroll
    for (int j = 0; j < NJ; ++j) srow[lane * NJ + j] = key[j];
    __syncwarp();
    constexpr int kMaxPerLane = kTkMaxE / 32;
    Bits gv[kMaxPerLane];
    float lost = 0.f;
    const int G = a.n_group, per = a.per;
#pragma unroll
    for (int i = 0; i < kMaxPerLane; ++i) {
        gv[i] = 0;
        const int g = lane + 32 * i;
        if (g < G) {
            Bits b1 = 0, b2 = 0;   // the two largest
            for (int q = 0; q < per; ++q) {
                const Bits v = srow[g * per + q];
                b2 = v > b1 ? b1 : (v > b2 ? v : b2);
                b1 = v > b1 ? v : b1;
            }
            if (b1 != 0) {
                const R v1 = K::value(b1), v2 = b2 != 0 ? K::value(b2) : R(0);
                gv[i] = K::of(v1 + v2);
                lost = fmaxf(lost, tk_cancelled((float)v1, (float)v2));
            }
        }
    }
    lost = tk_warp_most(lost);
    uint32_t kept = 0;    // bit i: group lane + 32 i is kept
    bool close = false;
    R last = R(0);
    for (int n = 0; n <= a.topk_group && n < G; ++n) {
        Bits best = 0;
        int bi = 0;
#pragma unroll
        for (int i = 0; i < kMaxPerLane; ++i)
            if (!(kept >> i & 1u) && gv[i] > best) { best = gv[i]; bi = i; }
        const Bits m = K::warp_max(best);
        if (m == 0) break;
        const R v = K::value(m);
        if (n == a.topk_group) {
            close = !(last - v > R(8e-6f) * (R(1) + fabs(v) + R(lost)));
            break;
        }
        // lowest index of a tie: lowest i first, then the lowest lane
        const int mi = __reduce_min_sync(0xffffffffu, best == m ? bi : 255);
        const uint32_t who = __ballot_sync(0xffffffffu, best == m && bi == mi);
        if (lane == __ffs(who) - 1) kept |= 1u << bi;
        last = v;
    }
    // the kept groups as bits that every lane can read (the keys' row is done with)
    __syncwarp();
    uint32_t* bits = reinterpret_cast<uint32_t*>(srow);
#pragma unroll
    for (int i = 0; i < kMaxPerLane; ++i) {
        const uint32_t word = __ballot_sync(0xffffffffu, kept >> i & 1u);
        if (lane == 0) bits[i] = word;
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const int e = lane * NJ + j;
        if (e < a.E) {
            const int g = e / per;
            if (!(bits[g >> 5] >> (g & 31) & 1u)) key[j] = 0;
        }
    }
    __syncwarp();
    return close;
}

// The k best keys: lane i gets the i-th one's expert (-1: none).  Returns whether
// two neighbours of the k + 1 best are nearer than the rounding of fp32 scores
// without being equal in logit and bias (check: only then; keys that are the
// logits themselves are exact).
template <int NJ, class K>
__device__ __forceinline__ bool tk_pick(const TkArgs& a, const float (&z)[NJ], int lane, typename K::Bits (&key)[NJ],
                                        bool check, int& my_id) {
    using Bits = typename K::Bits;
    using R = typename K::Real;
    my_id = -1;
    bool close = false;
    R last = R(0);
    int last_id = -1;
    for (int n = 0; n < a.k + (check ? 1 : 0); ++n) {
        Bits best = 0;
        int bj = 0;
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            if (key[j] > best) { best = key[j]; bj = j; }
        const Bits m = K::warp_max(best);
        if (m == 0) break;
        const uint32_t who = __ballot_sync(0xffffffffu, best == m);
        const int src = __ffs(who) - 1;
        const int id = src * NJ + __shfl_sync(0xffffffffu, bj, src);
        if (check) {
            const R v = K::value(m);
            if (n > 0 && last - v <= R(4e-6f) * (R(1) + fabs(v))) {
                // equal inputs have equal scores: a tie, not a doubt
                float zi = 0.f, zl = 0.f;
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    if (lane * NJ + j == id) zi = z[j];
                    if (lane * NJ + j == last_id) zl = z[j];
                }
                zi = __shfl_sync(0xffffffffu, zi, id / NJ);
                zl = __shfl_sync(0xffffffffu, zl, last_id / NJ);
                const bool same_b = a.bias == nullptr || __ldg(a.bias + id) == __ldg(a.bias + last_id);
                if (!(zi == zl && same_b)) close = true;
            }
            last = v;
            last_id = id;
        }
        if (n < a.k && lane == n) my_id = id;
        if (lane == src) {
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                if (j == bj) key[j] = 0;
        }
    }
    return close;
}

// tk_pick for scored keys, quicker: the three lowest bits of a key give way to the place of
// the expert in its lane, so that the warp's maximum names it.  That moves a value by less
// than 2^-20 of itself, which the doubtful gap covers; a tie orders by that place first, so
// every gap that small is doubtful here and the row is picked again by tk_pick.
template <int NJ>
__device__ __forceinline__ bool tk_pick_quick(const TkArgs& a, int lane, const uint32_t (&key)[NJ], int& my_id) {
    uint32_t k3[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) k3[j] = key[j] != 0 ? (key[j] & ~7u) | (uint32_t)(7 - j) : 0u;
    my_id = -1;
    float last = INFINITY;
    for (int n = 0; n <= a.k; ++n) {
        uint32_t best = k3[0];
#pragma unroll
        for (int j = 1; j < NJ; ++j) best = max(best, k3[j]);
        const uint32_t m = Key32::warp_max(best);
        if (m == 0) break;
        const float v = Key32::value(m);
        if (!(last - v > 6e-6f * (1.f + fabsf(v)))) return true;
        if (n == a.k) break;
        last = v;
        const int src = __ffs(__ballot_sync(0xffffffffu, best == m)) - 1;
        if (lane == n) my_id = src * NJ + 7 - (int)(m & 7u);
        const uint32_t mine = lane == src ? m : 0xffffffffu;
#pragma unroll
        for (int j = 0; j < NJ; ++j) k3[j] = k3[j] == mine ? 0u : k3[j];
    }
    return false;
}

template <int NJ, class K>
__device__ __forceinline__ bool tk_choose(const TkArgs& a, const float (&z)[NJ], int lane, void* srow, bool scored,
                                          int& my_id, float m) {
    typename K::Bits key[NJ];
    bool close = false;
    if (scored) {
        tk_choice_keys<NJ, K>(a, z, a.bias, lane, key, m);
        if (a.n_group > 1) {
            if constexpr (sizeof(typename K::Bits) == 4) {
                if (a.lane_groups) close = tk_keep_lane_groups<NJ>(a, lane, key);
                else close = tk_keep_groups<NJ, K>(a, lane, key, static_cast<typename K::Bits*>(srow));
            } else {
                close = tk_keep_groups<NJ, K>(a, lane, key, static_cast<typename K::Bits*>(srow));
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < NJ; ++j)   // (adding 0 makes -0 a +0: equal logits have equal keys)
            key[j] = z[j] > -INFINITY ? K::of(z[j] + 0.f) : typename K::Bits(0);
    }
    if constexpr (sizeof(typename K::Bits) == 4) {
        if (scored && !close && !tk_pick_quick<NJ>(a, lane, key, my_id)) return false;
    }
    const bool c2 = tk_pick<NJ, K>(a, z, lane, key, scored, my_id);
    return close || c2;
}

template <int NJ, typename T>
__global__ void __launch_bounds__(kTkWarps * 32) route_topk_kernel(const T* __restrict__ logits, const TkArgs a) {
    __shared__ alignas(16) unsigned long long stage[kTkWarps][kTkMaxE];   // a row of keys, then of gates
    griddep_wait();
    griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long t = (long long)blockIdx.x * kTkWarps + warp;
    if (t >= a.T) return;
    const T* row = logits + (size_t)t * a.E;
    float z[NJ];
    tk_load<NJ>(row, a.E, lane, -INFINITY, z);
#pragma unroll
    for (int j = 0; j < NJ; ++j) z[j] = z[j] == z[j] ? fminf(z[j], FLT_MAX) : -INFINITY;   // NaN: not choosable

    const bool scored = a.bias != nullptr || a.n_group > 1;
    float m = 0.f, sum = 0.f;
    if (!a.sigmoid && (scored || !a.renorm)) {   // softmax: its maximum and, for the weights, its sum
        uint32_t mk = 0;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const uint32_t kj = z[j] > -INFINITY ? Key32::of(z[j]) : 0u;
            mk = kj > mk ? kj : mk;
        }
        mk = Key32::warp_max(mk);
        m = mk != 0 ? Key32::value(mk) : 0.f;
        if (!a.renorm) {   // (not the choice's sum: the same logits have the same weights however they are chosen)
            float part = 0.f;
#pragma unroll
            for (int j = 0; j < NJ; ++j) part += z[j] > -INFINITY ? expf(z[j] - m) : 0.f;
            sum = tk_warp_sum(part);
        }
    }
    int id;
    if (tk_choose<NJ, Key32>(a, z, lane, stage[warp], scored, id, m))
        tk_choose<NJ, Key64>(a, z, lane, stage[warp], scored, id, m);

    // weights, in lane i for the i-th choice
    const bool have = id >= 0;
    float zi = -INFINITY;
    if (have) {
        const float v = tk_f32(row[id]);
        zi = fminf(v, FLT_MAX);
    }
    float w = 0.f;
    if (a.renorm) {
        const uint32_t mk = Key32::warp_max(have ? Key32::of(zi) : 0u);
        const float mm = mk != 0 ? Key32::value(mk) : 0.f;   // largest chosen logit
        if (have) {
            if (!a.sigmoid) w = expf(zi - mm);
            else w = mm < 0.f ? expf(zi - mm) / (1.f + expf(zi)) : 1.f / (1.f + expf(-zi));
        }
        const float total = tk_warp_sum(w);
        if (have) w = w / total * a.scale;
    } else if (have) {
        w = (a.sigmoid ? 1.f / (1.f + expf(-zi)) : expf(zi - m) / sum) * a.scale;
    }
    if (lane < a.k) {
        a.ids[(size_t)t * a.k + lane] = id;
        a.weights[(size_t)t * a.k + lane] = w;
    }
    if (a.gates == nullptr) return;
    // the dense row: zeros and the chosen weights meet in shared memory (rows of float4)
    float* srow = reinterpret_cast<float*>(stage[warp]);
    constexpr int kQuads = (NJ * 32 + 127) / 128;
#pragma unroll
    for (int i = 0; i < kQuads; ++i) reinterpret_cast<float4*>(srow)[i * 32 + lane] = make_float4(0.f, 0.f, 0.f, 0.f);
    __syncwarp();
    if (have) srow[id] = w;
    __syncwarp();
    float* grow = a.gates + (size_t)t * a.E;
    if ((a.E & 3) == 0) {   // (every row is then 16-byte aligned)
#pragma unroll
        for (int i = 0; i < kQuads; ++i)
            if ((i * 32 + lane) * 4 < a.E)
                reinterpret_cast<float4*>(grow)[i * 32 + lane] = reinterpret_cast<const float4*>(srow)[i * 32 + lane];
    } else {
        for (int e = lane; e < a.E; e += 32) grow[e] = srow[e];
    }
}

// The gradient of the weights with respect to the logits, the choice held fixed.
// With S = sum of the chosen scores and a = scale:
//   renormalised:  ds_i = a (dw_i - sum_j dw_j s_j / S) / S      else  ds_i = a dw_i
//   sigmoid:       dz_e = ds_e s_e (1 - s_e)      softmax: dz_e = s_e (ds_e - sum_j ds_j s_j)
// (an expert listed twice adds both its terms).  Renormalised softmax weights are
// the softmax over the chosen logits alone, so with p_i = s_i / S it is
// dz_i = a p_i (dw_i - sum_j dw_j p_j): nothing outside the chosen logits is read.
// One warp per token, the chosen experts in lanes 0 .. k-1; only softmax scores that
// are not renormalised need the whole row of logits.  Bound: writing d_logits (and
// reading the logits where the whole row counts).
template <int NJ, typename T>
__global__ void __launch_bounds__(kTkWarps * 32) route_topk_backward_kernel(
    const T* __restrict__ logits, const int32_t* __restrict__ ids, const float* __restrict__ d_weights, int T_, int E,
    int k, int sigmoid, int renorm, float scale, T* __restrict__ d_logits) {
    __shared__ alignas(16) float stage[kTkWarps][kTkMaxE];
    griddep_wait();
    griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long t = (long long)blockIdx.x * kTkWarps + warp;
    if (t >= T_) return;
    const T* row = logits + (size_t)t * E;
    int id = -1;
    float dw = 0.f, zi = -INFINITY;
    if (lane < k) {
        id = ids[(size_t)t * k + lane];
        if ((unsigned)id >= (unsigned)E) id = -1;
        if (id >= 0) {
            dw = d_weights[(size_t)t * k + lane] * scale;
            zi = tk_f32(row[id]);
            zi = zi == zi ? fminf(zi, FLT_MAX) : -INFINITY;   // (as the forward reads it)
            if (!(zi > -INFINITY)) {   // an expert that cannot be chosen has no weight
                id = -1;
                dw = 0.f;
            }
        }
    }
    const bool have = id >= 0;
    const bool whole = !sigmoid && !renorm;
    float z[NJ], m = 0.f, inv = 0.f;
    if (whole) {
        tk_load<NJ>(row, E, lane, -INFINITY, z);
        uint32_t mk = 0;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            z[j] = z[j] == z[j] ? fminf(z[j], FLT_MAX) : -INFINITY;
            const uint32_t kj = z[j] > -INFINITY ? Key32::of(z[j]) : 0u;
            mk = kj > mk ? kj : mk;
        }
        mk = Key32::warp_max(mk);
        m = mk != 0 ? Key32::value(mk) : 0.f;
        float part = 0.f;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            z[j] = z[j] > -INFINITY ? expf(z[j] - m) : 0.f;
            part += z[j];
        }
        const float total = tk_warp_sum(part);
        inv = total > 0.f ? 1.f / total : 0.f;
    }
    // v: what the lane's chosen expert receives; dot: what softmax takes from every expert
    float v = 0.f, dot = 0.f;
    if (renorm) {
        const uint32_t mk = Key32::warp_max(have ? Key32::of(zi) : 0u);
        const float mm = mk != 0 ? Key32::value(mk) : 0.f;
        const float sg = 1.f / (1.f + expf(-zi));
        float r = 0.f;
        if (have) r = !sigmoid ? expf(zi - mm) : (mm < 0.f ? expf(zi - mm) / (1.f + expf(zi)) : sg);
        const float S = tk_warp_sum(r);
        const float p = have ? r / S : 0.f;
        const float mean = tk_warp_sum(dw * p);
        v = have ? p * (dw - mean) * (sigmoid ? 1.f / (1.f + expf(zi)) : 1.f) : 0.f;   // 1 - s = 1 / (1 + e^z)
    } else if (sigmoid) {
        const float sg = 1.f / (1.f + expf(-zi));
        v = have ? dw * sg * (1.f / (1.f + expf(zi))) : 0.f;
    } else {
        const float s = have ? expf(zi - m) * inv : 0.f;
        dot = tk_warp_sum(dw * s);
        v = dw;
    }
    float* srow = stage[warp];
#pragma unroll
    for (int j = 0; j < NJ; ++j) srow[lane * NJ + j] = 0.f;
    __syncwarp();
    // an expert listed twice adds up in the order of the list
    const uint32_t same = __match_any_sync(0xffffffffu, have ? id : -1 - lane);
    if (__any_sync(0xffffffffu, __popc(same) > 1)) {
        for (int i = 0; i < k; ++i) {
            if (lane == i && have) srow[id] += v;
            __syncwarp();
        }
    } else if (have) {
        srow[id] = v;
    }
    __syncwarp();
    float d[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        d[j] = srow[lane * NJ + j];
        if (whole) d[j] = z[j] * inv * (d[j] - dot);
    }
    tk_store<NJ>(d_logits + (size_t)t * E, E, lane, d);
}

template <typename T, typename F>
cudaError_t tk_dispatch(int E, F&& f) {
    switch ((E + 31) / 32) {
        case 1: return f(std::integral_constant<int, 1>{});
        case 2: return f(std::integral_constant<int, 2>{});
        case 3: return f(std::integral_constant<int, 3>{});
        case 4: return f(std::integral_constant<int, 4>{});
        case 5: return f(std::integral_constant<int, 5>{});
        case 6: return f(std::integral_constant<int, 6>{});
        case 7: return f(std::integral_constant<int, 7>{});
        default: return f(std::integral_constant<int, 8>{});
    }
}

template <typename... KArgs, typename... Args>
cudaError_t tk_launch(void (*kern)(KArgs...), int T, cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(((long long)T + kTkWarps - 1) / kTkWarps));
    cfg.blockDim = dim3(kTkWarps * 32);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <typename T>
cudaError_t route_topk_t(const void* logits, const TkArgs& a, cudaStream_t s) {
    return tk_dispatch<T>(a.E, [&](auto nj) {
        return tk_launch(route_topk_kernel<decltype(nj)::value, T>, a.T, s, static_cast<const T*>(logits), a);
    });
}

template <typename T>
cudaError_t route_topk_backward_t(const void* logits, const int32_t* ids, const float* d_weights, int T_, int E, int k,
                                  int sigmoid, int renorm, float scale, void* d_logits, cudaStream_t s) {
    return tk_dispatch<T>(E, [&](auto nj) {
        return tk_launch(route_topk_backward_kernel<decltype(nj)::value, T>, T_, s, static_cast<const T*>(logits), ids,
                         d_weights, T_, E, k, sigmoid, renorm, scale, static_cast<T*>(d_logits));
    });
}

}  // namespace

cudaError_t launch_route_topk(const void* logits, bool bf16, const float* bias, int T, int E, int k, bool sigmoid,
                              int n_group, int topk_group, bool renorm, float scale, float* gates, int32_t* ids,
                              float* weights, cudaStream_t s) {
    TkArgs a;
    a.bias = bias;
    a.T = T;
    a.E = E;
    a.k = k;
    a.sigmoid = sigmoid;
    a.n_group = topk_group == n_group ? 1 : n_group;   // every group kept: no groups
    a.topk_group = topk_group;
    a.per = E / n_group;
    a.lane_groups = E % 32 == 0 && n_group <= 32 && (n_group & (n_group - 1)) == 0;
    a.renorm = renorm;
    a.scale = scale;
    a.gates = gates;
    a.ids = ids;
    a.weights = weights;
    return bf16 ? route_topk_t<__nv_bfloat16>(logits, a, s) : route_topk_t<float>(logits, a, s);
}

cudaError_t launch_route_topk_backward(const void* logits, bool bf16, const int32_t* ids, const float* d_weights, int T,
                                       int E, int k, bool sigmoid, bool renorm, float scale, void* d_logits,
                                       cudaStream_t s) {
    return bf16 ? route_topk_backward_t<__nv_bfloat16>(logits, ids, d_weights, T, E, k, sigmoid, renorm, scale,
                                                       d_logits, s)
                : route_topk_backward_t<float>(logits, ids, d_weights, T, E, k, sigmoid, renorm, scale, d_logits, s);
}

}  // namespace bffn
