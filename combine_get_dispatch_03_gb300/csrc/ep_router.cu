// ep_router.cu -- the router in front of a dispatch: every token's experts and their weights, and its gradient (sm_103a).
//
//   forward    s = softmax(l) or sigmoid(l);  key = s + bias;  of G groups of E / G experts the L with the largest sums of
//              their two largest keys stay;  the K largest keys in descending order, ties to the lowest expert;
//              w = scale * s, or scale * s / sum of the chosen s
//   gradient   dl from dw.  With normalised weights u = w / scale only the chosen logits have one:
//                softmax  dl = scale * u * (dw - sum dw u)        sigmoid  dl = scale * u * (dw - sum dw u) * (1 - s)
//              else  sigmoid  dl = scale * dw * s * (1 - s) of the chosen,  softmax  dl_e = p_e * (scale * dw_e - sum scale dw p)
//
// A warp owns a token; its lanes hold neighbouring experts.  The K-th largest of the lanes' largest keys is a bound that at
// least K keys reach, few more do, and no chosen key lies below: those that reach it are given a lane each, which counts
// the ones before it.  Where more than 32 reach it (ties), the keys are taken one by one (choose_in_turn).
//
// Which experts are chosen must not hang on the rounding of s.  Without bias the keys are the logits themselves; groups
// are compared by their scores.  32-bit scores decide unless two that are compared lie closer than their error
// (kSigmoidError): such keys are computed again in 64 bits, a lane each, of those that reached the bound or may decide between
// groups.  Beside a softmax a bias feels the sum of all exponentials: there the whole token is computed again (choose_exactly),
// a percent of the tokens.
//
// Instructions bound it, not memory (an ncu capture: 1249 a token with bias and groups, 618 and 657 without): 32768 tokens of 256 fp32
// logits, K 8, whose bytes take 5.4 us, take 24 us with sigmoid, 26 with softmax, 36 with a bias, 46 to 49 with 8 groups, 70 with
// softmax and bias (bf16 the same: 24, 25, with 8 groups 47); 4096 tokens 6 to 10 us, with softmax and bias 25; a decode step of 32
// tokens 2.  K rounds of a maximum over the warp took 42 us without bias and 90 with bias and groups.  Groups that begin inside a
// lane's experts (160 experts in 8) go through shared memory, 70 to 90 us.
//
// The gradient writes every logit, and reads them all only for a softmax that is not normalised: 18.7 us, bf16 17.5, where the
// bytes take 10.4 and 5.4.  The other forms read the chosen logits: normalised softmax 13.7 us, bf16 10.0, sigmoid 14.3 and 10.7, not
// normalised 13.6 and 8.3, where the bytes (33.5 MB written in fp32, 8.4 in sectors of 32 bytes of the chosen, 3.1 of indices
// and weights) take 6.7 and 4.2.  Not memory bounds them but a token's two loads, its indices and then their logits, with
// nothing of the warp's next token on its way.
#include "ep_act.cuh"
#include "ep_groups.cuh"
#include "ep_handle.h"
#include "ep_trace.h"

namespace ep {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / kWarpSize;
constexpr int kMaxGroups = 32;
// The error of a comparison of two keys, as a part of the token's largest score.  Sigmoid: 2^-22.3 a key from the
// exponential, the reciprocal and two roundings.  Softmax: at most 28 roundings of 2^-24 more in its sum, which a bias feels.
constexpr float kSigmoidError = 1e-6f, kSoftmaxError = 2e-6f;
constexpr float kFlushError = 2.4e-38f;  // 2^-125: sigmoids below 2^-126 are flushed to 0
constexpr float kSumError = 2.4e-7f;  // 2^-22 of the keys themselves, from adding the bias or a second key

struct RouterParams {
    const void* logits;
    const float* bias;
    const uint8_t* token_mask;
    int64_t* topk_idx;
    float* topk_weights;
    const int64_t* chosen;      // gradient: topk_idx
    const float* d_weights;
    void* d_logits;
    int32_t* status;
    int64_t tokens;
    int32_t experts, topk, groups, kept, softmax, normalize, vector;
    float scale;
};

// Order-preserving 64-bit key; 0 for what cannot be chosen (NaN, -inf).
__device__ __forceinline__ uint64_t ordered64(double v) {
    if (!(v > -INFINITY)) return 0;
    const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
    return u >> 63 ? ~u : u | (1ull << 63);
}

__device__ __forceinline__ double unordered64(uint64_t k) {
    if (k == 0) return -INFINITY;
    return __longlong_as_double(static_cast<long long>(k >> 63 ? k & ~(1ull << 63) : ~k));
}

// exp(v) to 2^-22.  Past e^88 and e^-104 (0) it stays there: keys that become equal so are looked at in 64 bits.
__device__ __forceinline__ float exp_fast(float v) { return exp_fp32(fminf(fmaxf(v, -104.0f), 88.0f)); }

__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// A logit: NaN counts as -inf (it cannot be chosen and has no weight), +inf as the largest finite value.
template <typename T>
__device__ __forceinline__ float logit(const void* p, int64_t at) {
    float v;
    if constexpr (sizeof(T) == 4) v = __ldg(static_cast<const float*>(p) + at);
    else v = __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(p) + at)) << 16);
    return v != v ? -INFINITY : fminf(v, 3.402823466e38f);
}

// An expert's bias: -inf for NaN; of finite size, 2^100 at most, so that sums of two keys and their errors stay finite.
__device__ __forceinline__ float bias_of(const RouterParams& p, int expert) {
    const float b = __ldg(p.bias + expert);
    return b > -INFINITY ? fminf(fmaxf(b, -0x1p100f), 0x1p100f) : -INFINITY;
}

// Experts [lane * V, lane * V + V) of a token; -inf past the last, for NaN, and the largest finite value for +inf.
template <typename T, int V>
__device__ __forceinline__ void load_row(const RouterParams& p, int64_t token, float (&l)[V]) {
    const int first = lane_id() * V;
    constexpr int kVec = 16 / sizeof(T);
    if constexpr (V >= kVec) {
        if (p.vector) {  // rows are 16-byte aligned: pieces of kVec experts are there or not
            const int4* row = reinterpret_cast<const int4*>(static_cast<const uint8_t*>(p.logits) + (token * p.experts + first) * sizeof(T));
#pragma unroll
            for (int i = 0; i < V / kVec; ++i) {
                int4 q = make_int4(0, 0, 0, 0);
                const bool in = first + i * kVec < p.experts;
                if (in) q = ld_stream_ordered_v4(row + i);
                float f[kVec];
                if constexpr (sizeof(T) == 4) {
                    f[0] = __int_as_float(q.x), f[1] = __int_as_float(q.y), f[2] = __int_as_float(q.z), f[3] = __int_as_float(q.w);
                } else {
                    unpack8(q, f);
                }
#pragma unroll
                for (int j = 0; j < kVec; ++j) l[i * kVec + j] = in ? fminf(fmaxf(f[j], -INFINITY), 3.402823466e38f) : -INFINITY;  // fmaxf drops NaN
            }
            return;
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) l[v] = first + v < p.experts ? logit<T>(p.logits, token * p.experts + first + v) : -INFINITY;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = kWarpSize / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kFullMask, v, o);
    return v;
}

// The largest logit (-inf without any) and the sum of exp(l - largest).
template <int V>
__device__ __forceinline__ void softmax_stats(const float (&l)[V], float* most, float* sum) {
    float m = l[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = fmaxf(m, l[v]);
    m = warp_max(m);
    const float base = m > -INFINITY ? m : 0.0f;
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int v = 0; v < V; ++v) s[v & 3] += l[v] > -INFINITY ? exp_fast(l[v] - base) : 0.0f;
    *most = base;
    *sum = warp_sum((s[0] + s[1]) + (s[2] + s[3]));
}

__device__ __forceinline__ uint64_t warp_max64(uint64_t v) {
    const uint32_t high = __reduce_max_sync(kFullMask, static_cast<uint32_t>(v >> 32));
    const uint32_t low = __reduce_max_sync(kFullMask, v >> 32 == high ? static_cast<uint32_t>(v) : 0u);
    return static_cast<uint64_t>(high) << 32 | low;
}

// a >= b: the two largest of four.
__device__ __forceinline__ void join_two(uint64_t& a, uint64_t& b, uint64_t c, uint64_t d) {
    b = c > a ? (a > d ? a : d) : (b > c ? b : c);
    a = c > a ? c : a;
}

// The token's choice with keys in 64 bits.  Returns lane k's expert (-1: none) for k < topk.  The lanes' experts are worked
// on side by side: FP64 instructions are slow, and each alone waits for the one before.
template <typename T, int V>
__device__ __noinline__ int choose_exactly(const RouterParams& p, int64_t token) {
    uint64_t key[V];
    const int first = lane_id() * V;
    double most = 0.0, inv_sum = 1.0;
    if (p.softmax) {
        float top = -INFINITY;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (first + v < p.experts) top = fmaxf(top, logit<T>(p.logits, token * p.experts + first + v));
        top = warp_max(top);
        most = top > -INFINITY ? top : 0.0;
        double sum = 0.0;
#pragma unroll 8
        for (int v = 0; v < V; ++v) {
            const float l = first + v < p.experts ? logit<T>(p.logits, token * p.experts + first + v) : -INFINITY;
            sum += exp(static_cast<double>(l) - most);
        }
        for (int o = kWarpSize / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(kFullMask, sum, o);
        inv_sum = sum > 0.0 ? sum : 1.0;
    }
#pragma unroll 8
    for (int v = 0; v < V; ++v) {
        const float l = first + v < p.experts ? logit<T>(p.logits, token * p.experts + first + v) : -INFINITY;
        const double e = exp(p.softmax ? static_cast<double>(l) - most : -static_cast<double>(l));
        double s = p.softmax ? e / inv_sum : 1.0 / (1.0 + e);
        if (p.bias && first + v < p.experts) s += static_cast<double>(bias_of(p, first + v));
        key[v] = l > -INFINITY ? ordered64(s) : 0;
    }
    if (p.groups > 1) {
        const int size = p.experts / p.groups, lanes = size / V;
        uint64_t mine = 0;  // lane g: the score of group g
        if (lanes * V == size && (lanes & (lanes - 1)) == 0) {  // a group is a power of two of whole lanes
            uint64_t a = 0, b = 0;
#pragma unroll
            for (int v = 0; v < V; ++v) join_two(a, b, key[v], 0);
            for (int o = 1; o < lanes; o <<= 1) {
                const uint64_t c = __shfl_xor_sync(kFullMask, a, o), d = __shfl_xor_sync(kFullMask, b, o);
                join_two(a, b, c, d);
            }
            const uint64_t score = size == 1 ? a : ordered64(unordered64(a) + unordered64(b));
            mine = __shfl_sync(kFullMask, score, min(lane_id() * lanes, kWarpSize - 1));
        } else {
            for (int g = 0; g < p.groups; ++g) {
                uint64_t a = 0, b = 0;
                for (int v = 0; v < V; ++v)
                    if (first + v < p.experts && (first + v) / size == g) join_two(a, b, key[v], 0);
                for (int o = kWarpSize / 2; o > 0; o >>= 1) {
                    const uint64_t c = __shfl_xor_sync(kFullMask, a, o), d = __shfl_xor_sync(kFullMask, b, o);
                    join_two(a, b, c, d);
                }
                if (lane_id() == g) mine = size == 1 ? a : ordered64(unordered64(a) + unordered64(b));
            }
        }
        int better = 0;
        for (int g = 0; g < p.groups; ++g) {
            const uint64_t other = __shfl_sync(kFullMask, mine, g);
            better += other > mine || (other == mine && g < lane_id());
        }
        const unsigned stay = __ballot_sync(kFullMask, lane_id() < p.groups && better < p.kept);
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (first + v < p.experts && !(stay >> ((first + v) / size) & 1)) key[v] = 0;
    }
    int chosen = -1;
#pragma unroll 1
    for (int k = 0; k < p.topk; ++k) {
        uint64_t best = 0;
        int at = 0;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (key[v] > best) best = key[v], at = v;
        const uint64_t top = warp_max64(best);
        if (top == 0) break;
        const int lane = __ffs(__ballot_sync(kFullMask, best == top)) - 1;
        const int expert = __shfl_sync(kFullMask, first + at, lane);
        if (lane_id() == k) chosen = expert;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (lane_id() == lane && v == at) key[v] = 0;
    }
    return chosen;
}

// The score of the group of this lane's number (lane g < groups), from the warp's keys: two largest, added up.  *second: the
// smaller; *magnitude: their sizes added up, by which their roundings and the sum's go (the sum itself may be of two that cancel).
template <int V>
__device__ __forceinline__ float group_score(const RouterParams& p, const float (&key)[V], float* scratch, float* second, float* magnitude) {
    const int size = p.experts / p.groups;
    float a = -INFINITY, b = -INFINITY;
    const int lanes = size / V;
    if (lanes * V == size && (lanes & (lanes - 1)) == 0) {  // a group is a power of two of whole lanes
#pragma unroll
        for (int v = 0; v < V; ++v) {
            b = fmaxf(b, fminf(a, key[v]));
            a = fmaxf(a, key[v]);
        }
        for (int o = 1; o < lanes; o <<= 1) {
            const float c = __shfl_xor_sync(kFullMask, a, o), d = __shfl_xor_sync(kFullMask, b, o);
            b = fmaxf(fminf(a, c), fmaxf(b, d));
            a = fmaxf(a, c);
        }
        const int from = min(lane_id() * lanes, kWarpSize - 1);
        a = __shfl_sync(kFullMask, a, from);
        b = __shfl_sync(kFullMask, b, from);
    } else {
        __syncwarp();
#pragma unroll
        for (int v = 0; v < V; ++v) scratch[lane_id() * V + v] = key[v];
        __syncwarp();
        if (lane_id() < p.groups)
            for (int i = 0; i < size; ++i) {
                const float k = scratch[lane_id() * size + i];
                b = fmaxf(b, fminf(a, k));
                a = fmaxf(a, k);
            }
    }
    *second = size == 1 ? a : b;
    *magnitude = size == 1 ? fabsf(a) : fabsf(a) + fabsf(b);
    return size == 1 ? a : a + b;
}

// Whether a key's order in 64 bits hangs on its own logit alone: not on a softmax's sum, which a bias is added beside.
__device__ __forceinline__ bool alone(const RouterParams& p) { return !p.softmax || p.bias == nullptr; }

// A key in 64 bits, then; of a softmax times its sum.  One copy of it: code that few tokens run is fetched from memory when
// they do.
__device__ __noinline__ double key64(const RouterParams& p, float l, int expert, float most) {
    const double e = exp(p.softmax ? static_cast<double>(l) - most : -static_cast<double>(l));
    if (p.softmax) return e;
    return 1.0 / (1.0 + e) + (p.bias ? static_cast<double>(bias_of(p, expert)) : 0.0);
}

// How far apart two keys must lie for 32 bits to tell them; `error` is that of their scores.
__device__ __forceinline__ float key_error(float error, float a, float b) { return error + kSumError * (fabsf(a) + fabsf(b)); }

// sigmoid(l) * exp(-top) for l <= top < 0; 0 where sigmoid(l) is 0 in 64 bits too.
__device__ __forceinline__ float low_sigmoid(float l, float top) { return l < -709.78f ? 0.0f : expf(l - top) / (1.0f + expf(l)); }

struct Chosen {
    int expert;  // lane k's, -1: none
    bool close;  // 32 bits may have it wrong
};

// The K largest keys one by one, each the maximum of the lanes' largest, the lowest lane's and expert's of equal ones.
template <typename T, int V>
__device__ __noinline__ Chosen choose_in_turn(const RouterParams& p, int64_t token, float (&key)[V], float error, bool scored) {
    const int first = lane_id() * V;
    Chosen r = {-1, false};
    float chosen_key = -INFINITY, last = -INFINITY;
#pragma unroll 1
    for (int k = 0; k < p.topk; ++k) {
        float best = key[0];
        int at = 0;
        for (int v = 1; v < V; ++v)
            if (key[v] > best) best = key[v], at = v;
        const float top = warp_max(best);
        last = top;
        if (!(top > -INFINITY)) break;
        const int lane = __ffs(__ballot_sync(kFullMask, best == top)) - 1;
        const int expert = __shfl_sync(kFullMask, first + at, lane);
        if (lane_id() == k) r.expert = expert, chosen_key = top;
        if (lane_id() == lane) key[at] = -INFINITY;
    }
    if (!scored) return r;
    // Neighbours in the order, and who is left next to the last: too close, unless they tie because their inputs are the same.
    float lc = 0.0f, bc = 0.0f;
    if (r.expert >= 0) {
        lc = logit<T>(p.logits, token * p.experts + r.expert);
        if (p.bias) bc = p.bias[r.expert];
    }
    const float after = __shfl_down_sync(kFullMask, chosen_key, 1);
    const float l_after = __shfl_down_sync(kFullMask, lc, 1), b_after = __shfl_down_sync(kFullMask, bc, 1);
    bool near = r.expert >= 0 && lane_id() < p.topk - 1 && lane_id() < kWarpSize - 1 && after > -INFINITY &&
                chosen_key - after <= key_error(error, chosen_key, after) && !(lc == l_after && bc == b_after);
    if (last > -INFINITY) {  // all K are there
        const float l_last = __shfl_sync(kFullMask, lc, p.topk - 1), b_last = __shfl_sync(kFullMask, bc, p.topk - 1);
        for (int v = 0; v < V; ++v)
            if (key[v] > -INFINITY && last - key[v] <= key_error(error, last, key[v]))
                near |= !(logit<T>(p.logits, token * p.experts + first + v) == l_last && (p.bias == nullptr || p.bias[first + v] == b_last));
    }
    r.close = __any_sync(kFullMask, near);
    return r;
}

// What a warp knows of the keys that reach the bound: of each its key, expert and logit, in order of experts, and the keys in
// descending order.
struct Reach {
    float2 key_expert[kWarpSize];
    float logit[kWarpSize];
    float2 sorted[kWarpSize];  // key, which (as bits)
};

// The scored tokens' keys, s + bias, of the groups that stay; *error: of a score.  Whether 32 bits may have the groups wrong.
template <int V>
__device__ __forceinline__ bool make_keys(const RouterParams& p, const float (&l)[V], float most, float sum, float* scratch,
                                          Reach& reach, float (&key)[V], float* error) {
    const int first = lane_id() * V;
    const float inv = 1.0f / sum;
    float top = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const bool in = l[v] > -INFINITY;
        const float e = exp_fast(p.softmax ? l[v] - most : -l[v]);
        const float s = p.softmax ? e * inv : reciprocal(1.0f + e);
        top = fmaxf(top, in ? s : 0.0f);
        key[v] = in ? (p.bias ? s + bias_of(p, first + v) : s) : -INFINITY;
    }
    *error = fmaf(p.softmax ? kSoftmaxError : kSigmoidError, warp_max(top), kFlushError);
    if (p.groups == 1) return false;
    const int size = p.experts / p.groups;
    float second, magnitude;
    const float score = group_score<V>(p, key, scratch, &second, &magnitude);
    int better = 0;
    for (int g = 0; g < p.groups; ++g) {
        const float other = __shfl_sync(kFullMask, score, g);
        better += other > score || (other == score && g < lane_id());
    }
    const bool there = lane_id() < p.groups, in = there && better < p.kept;
    unsigned stay = __ballot_sync(kFullMask, in);
    // A score lies in [low, high] in 64 bits: the least that one that stays can have, the most of one that does not.
    const float own = score > -INFINITY ? *error + kSumError * magnitude : 0.0f;
    const float low = score - own, high = score + own;
    const float last = -warp_max(in ? -low : -INFINITY), next = warp_max(there && !in ? high : -INFINITY);
    bool close = next > -INFINITY && last <= next;
    if (close && alone(p) && size % V == 0) {
        // Groups around the border compete again, by what their largest members are worth in 64 bits, a lane each.
        const bool rival = there && low <= next && high >= last;
        const unsigned rivals = __ballot_sync(kFullMask, rival), above = __ballot_sync(kFullMask, in && !rival);
        const int mine = first < p.experts ? first / size : 0;
        const float least = __shfl_sync(kFullMask, second - 2.0f * key_error(*error, second, second), mine);
        int all = 0;
        __syncwarp();
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const bool member = first < p.experts && (rivals >> mine & 1) && key[v] > -INFINITY && key[v] >= least;
            const unsigned members = __ballot_sync(kFullMask, member);
            const int at = all + __popc(members & lanemask_lt());
            if (member && at < kWarpSize) reach.key_expert[at] = make_float2(l[v], __int_as_float(first + v));
            all += __popc(members);
        }
        __syncwarp();
        if (all <= kWarpSize) {
            const float2 c = lane_id() < all ? reach.key_expert[lane_id()] : make_float2(0.0f, 0.0f);
            const int expert = __float_as_int(c.y);
            const uint64_t exact = lane_id() < all ? ordered64(key64(p, c.x, expert, most)) : 0;
            uint64_t sum = 0;  // lane g: the score of rival g
            for (unsigned left = rivals; left; left &= left - 1) {
                const int g = __ffs(left) - 1;
                uint64_t k = lane_id() < all && expert / size == g ? exact : 0;
                const uint64_t a = warp_max64(k);
                if (lane_id() == __ffs(__ballot_sync(kFullMask, k == a)) - 1) k = 0;
                const uint64_t b = warp_max64(k);
                if (lane_id() == g) sum = size == 1 ? a : ordered64(unordered64(a) + unordered64(b));
            }
            int ahead = 0;
            for (unsigned left = rivals; left; left &= left - 1) {
                const int g = __ffs(left) - 1;
                const uint64_t other = __shfl_sync(kFullMask, sum, g);
                ahead += other > sum || (other == sum && g < lane_id());
            }
            stay = above | __ballot_sync(kFullMask, rival && ahead < p.kept - __popc(above));
            close = false;
        }
    }
    if (size % V == 0) {
        if (first < p.experts && !(stay >> (first / size) & 1))
#pragma unroll
            for (int v = 0; v < V; ++v) key[v] = -INFINITY;
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (first + v < p.experts && !(stay >> ((first + v) / size) & 1)) key[v] = -INFINITY;
    }
    return close;
}

// kScored: with bias or groups; otherwise the scores' order is the logits'.
template <typename T, int V, bool kScored>
__device__ __forceinline__ void route_token(const RouterParams& p, int64_t token, const float (&l)[V], float* scratch, Reach& reach) {
    const int first = lane_id() * V;
    const int64_t out = token * p.topk;
    if (p.token_mask && p.token_mask[token] == 0) {
        if (lane_id() < p.topk) p.topk_idx[out + lane_id()] = -1, p.topk_weights[out + lane_id()] = 0.0f;
        return;
    }
    float most = 0.0f, sum = 1.0f;
    if (p.softmax && (kScored || !p.normalize)) softmax_stats<V>(l, &most, &sum);
    float key[V];
    float error = 0.0f;
    bool close = false;
    if constexpr (kScored) {
        close = make_keys<V>(p, l, most, sum, scratch, reach, key, &error);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) key[v] = l[v];
    }
    // the K-th largest of the lanes' largest keys: at least K keys reach it
    float mine = key[0];
#pragma unroll
    for (int v = 1; v < V; ++v) mine = fmaxf(mine, key[v]);
    float bound;
    int reached = 0;
    do {
        bound = warp_max(mine);
        const bool is = mine == bound;
        reached += __popc(__ballot_sync(kFullMask, is));
        mine = is ? -INFINITY : mine;
    } while (reached < p.topk && bound > -INFINITY);
    // who reaches it, with the room that 32 bits need
    if (kScored) bound -= 2.0f * key_error(error, bound, bound);
    bound = fmaxf(bound, -3.402823466e38f);
    int count = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) count += key[v] >= bound;
    int at = count;
#pragma unroll
    for (int o = 1; o < kWarpSize; o <<= 1) {
        const int other = __shfl_up_sync(kFullMask, at, o);
        if (lane_id() >= o) at += other;
    }
    const int all = __shfl_sync(kFullMask, at, kWarpSize - 1);
    at -= count;
    int expert = -1, rank = kWarpSize;
    float lc = -INFINITY;
    if (!close && all <= kWarpSize) {
        __syncwarp();  // the last token's have been read
        if (count)
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (key[v] >= bound) {
                    reach.key_expert[at] = make_float2(key[v], __int_as_float(first + v));
                    if (kScored) reach.logit[at] = l[v];
                    ++at;
                }
        __syncwarp();
        const bool there = lane_id() < all;
        float k = -INFINITY;
        if (there) {
            const float2 c = reach.key_expert[lane_id()];
            k = c.x, expert = __float_as_int(c.y);
            lc = kScored ? reach.logit[lane_id()] : k;
        }
        int before = 0;
        for (int j = 0; j < all; ++j) {  // in order of experts
            const float other = reach.key_expert[j].x;
            before += other > k || (other == k && j < lane_id());
        }
        if (there) rank = before;
        if constexpr (kScored) {
            // Neighbours in the order of which one at least is chosen: too close, unless they tie because their inputs are the
            // same.  Then the next one is looked at: where equal inputs lie on both sides of the last place, it is what
            // may belong before them.
            if (there) reach.sorted[rank] = make_float2(k, __int_as_float(lane_id()));
            __syncwarp();
            bool near = false;
            for (int r = rank < p.topk ? rank + 1 : all; r < all && !near; ++r) {
                const float2 next = reach.sorted[r];
                if (k - next.x > key_error(error, k, next.x)) break;
                const int j = __float_as_int(next.y), e = __float_as_int(reach.key_expert[j].y);
                near = reach.logit[j] != lc || (p.bias && p.bias[e] != p.bias[expert]);
            }
            __syncwarp();
            if (__any_sync(kFullMask, near)) {
                if (!alone(p)) {
                    close = true;
                } else {
                    const double exact = there ? key64(p, lc, expert, most) : 0.0;
                    before = 0;
                    for (int j = 0; j < all; ++j) {
                        const double other = __shfl_sync(kFullMask, exact, j);
                        before += other > exact || (other == exact && j < lane_id());
                    }
                    if (there) rank = before;
                }
            }
        }
    }
    if (close || all > kWarpSize) {
        if (!close) {
            float copy[V];
#pragma unroll
            for (int v = 0; v < V; ++v) copy[v] = key[v];
            const Chosen r = choose_in_turn<T, V>(p, token, copy, error, kScored);
            expert = r.expert;
            close = r.close;
        }
        if (close) expert = choose_exactly<T, V>(p, token);
        rank = lane_id();
        lc = expert >= 0 ? logit<T>(p.logits, token * p.experts + expert) : -INFINITY;
    }

    const bool chosen = expert >= 0 && rank < p.topk;
    float s = 0.0f;
    if (p.softmax) {
        float base = most;
        if (p.normalize) base = warp_max(chosen ? lc : -INFINITY);  // the sum cancels
        if (chosen) s = expf(lc - base);
        if (chosen && !p.normalize) s /= sum;
    } else {
        // normalised, the largest score cancels: without it none is lost where all lie below what fp32 holds
        const float top = p.normalize ? warp_max(chosen ? lc : -INFINITY) : 0.0f;
        if (chosen) s = top < 0.0f ? low_sigmoid(lc, top) : 1.0f / (1.0f + expf(-lc));
    }
    float w = s * p.scale;
    if (p.normalize) {
        const float total = warp_sum(s);
        w = total > 0.0f ? s / total * p.scale : 0.0f;
    }
    if (chosen) {
        p.topk_idx[out + rank] = expert;
        p.topk_weights[out + rank] = w;
    }
    const int found = __popc(__ballot_sync(kFullMask, chosen));
    if (lane_id() >= found && lane_id() < p.topk) p.topk_idx[out + lane_id()] = -1, p.topk_weights[out + lane_id()] = 0.0f;
}

template <typename T, int V, bool kScored>
__global__ void __launch_bounds__(kThreads, V <= 8 ? 4 : V <= 16 ? 2 : 1) router_kernel(const RouterParams p) {
    extern __shared__ float scratch[];  // a warp's keys, where groups cut across lanes
    __shared__ Reach reach[kWarps];
    pdl_enter();
    const int64_t warps = static_cast<int64_t>(gridDim.x) * kWarps;
    int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / kWarpSize;
    if (t >= p.tokens) return;
    // the next token's logits are on their way while one is worked on
    float next[V];
    load_row<T, V>(p, t, next);
    for (; t < p.tokens; t += warps) {
        float l[V];
#pragma unroll
        for (int v = 0; v < V; ++v) l[v] = next[v];
        if (t + warps < p.tokens) load_row<T, V>(p, t + warps, next);
        route_token<T, V, kScored>(p, t, l, scratch + threadIdx.x / kWarpSize * (kWarpSize * V), reach[threadIdx.x / kWarpSize]);
    }
}

template <typename T>
__device__ __forceinline__ void store_logit(void* p, int64_t at, float v) {
    if constexpr (sizeof(T) == 4) static_cast<float*>(p)[at] = v;
    else static_cast<__nv_bfloat16*>(p)[at] = __float2bfloat16_rn(v);
}

template <typename T, int V>
__device__ __forceinline__ void store_row(const RouterParams& p, int64_t token, const float (&d)[V]) {
    const int first = lane_id() * V;
    constexpr int kVec = 16 / sizeof(T);
    if constexpr (V >= kVec) {
        if (p.vector) {
            int4* row = reinterpret_cast<int4*>(static_cast<uint8_t*>(p.d_logits) + (token * p.experts + first) * sizeof(T));
#pragma unroll
            for (int i = 0; i < V / kVec; ++i) {
                if (first + i * kVec >= p.experts) break;
                float f[kVec];
#pragma unroll
                for (int j = 0; j < kVec; ++j) f[j] = d[i * kVec + j];
                if constexpr (sizeof(T) == 4)
                    st_stream_v4(row + i, make_int4(__float_as_int(f[0]), __float_as_int(f[1]), __float_as_int(f[2]), __float_as_int(f[3])));
                else
                    st_stream_v4(row + i, pack8_bf16(f));
            }
            return;
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (first + v < p.experts) store_logit<T>(p.d_logits, token * p.experts + first + v, d[v]);
}

template <typename T, int V>
__device__ __forceinline__ void route_gradient(const RouterParams& p, int64_t token) {
    const int64_t in = token * p.topk + lane_id();
    const int64_t raw = lane_id() < p.topk ? p.chosen[in] : -1;
    if (raw < -1 || raw >= p.experts) report(p.status, EP_ERR_BAD_EXPERT);
    const int chosen = raw >= 0 && raw < p.experts ? static_cast<int>(raw) : -1;
    const bool mine = chosen >= 0;
    const float lc = mine ? logit<T>(p.logits, token * p.experts + chosen) : -INFINITY;
    const float dw = mine ? p.d_weights[in] * p.scale : 0.0f;
    float d[V];
    float own = 0.0f, base = 0.0f;  // the chosen logit's gradient in two parts: its slot's, and what every logit of the token gets
    if (p.softmax && !p.normalize) {
        load_row<T, V>(p, token, d);
        float most, sum;
        softmax_stats<V>(d, &most, &sum);
        const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
        const float u = mine && lc > -INFINITY ? expf(lc - most) * inv : 0.0f;
        own = dw * u;
        const float dot = warp_sum(own);
        base = -u * dot;
#pragma unroll
        for (int v = 0; v < V; ++v) d[v] = d[v] > -INFINITY ? -(exp_fast(d[v] - most) * inv) * dot : 0.0f;
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) d[v] = 0.0f;
        float s = 0.0f, rest = 1.0f;  // rest: 1 - s
        const float top = p.softmax || p.normalize ? warp_max(lc) : 0.0f;
        if (p.softmax) {
            if (mine && lc > -INFINITY) s = expf(lc - top);
        } else if (mine) {
            const float e = expf(-fabsf(lc)), small = e / (1.0f + e), large = 1.0f / (1.0f + e);
            s = top < 0.0f ? low_sigmoid(lc, top) : lc >= 0.0f ? large : small;
            rest = lc >= 0.0f ? small : large;
        }
        if (p.normalize) {
            const float total = warp_sum(s);
            const float u = total > 0.0f ? s / total : 0.0f;
            own = u * (dw - warp_sum(dw * u)) * rest;
        } else {
            own = dw * s * rest;
        }
    }
    store_row<T, V>(p, token, d);
    // the chosen ones: the same expert twice gets both
    const unsigned same = __match_any_sync(kFullMask, chosen);
    float total = own;
    if (__any_sync(kFullMask, mine && (same & (same - 1)))) {
        total = 0.0f;
        for (int k = 0; k < p.topk; ++k) {
            const float other = __shfl_sync(kFullMask, own, k);
            if (same >> k & 1) total += other;
        }
    }
    __syncwarp();  // after the row's stores
    if (mine) store_logit<T>(p.d_logits, token * p.experts + chosen, base + total);
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) router_grad_kernel(const RouterParams p) {
    pdl_enter();
    const int64_t warps = static_cast<int64_t>(gridDim.x) * kWarps;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / kWarpSize; t < p.tokens; t += warps)
        route_gradient<T, V>(p, t);
}

constexpr int ctas_per_sm(int per_lane) { return per_lane <= 8 ? 4 : per_lane <= 16 ? 2 : 1; }  // of the forward pass: one resident wave
constexpr int kCtasPerSm = 4;  // that any variant can have resident
constexpr int kWaves = 8;

template <bool kGrad, typename T, int V>
cudaError_t start(const ep_handle* h, const RouterParams& p, cudaStream_t stream) {
    const int64_t wanted = (p.tokens + kWarps - 1) / kWarps;
    const int64_t most = static_cast<int64_t>(h->plan.num_sms) * (kGrad ? kCtasPerSm * (h->plan.sm_limited ? 1 : kWaves) : ctas_per_sm(V));
    const dim3 grid(static_cast<unsigned>(wanted < most ? wanted : most));
    if constexpr (kGrad) return launch_kernel(router_grad_kernel<T, V>, grid, dim3(kThreads), 0, stream, 1, p);
    if (p.bias == nullptr && p.groups == 1)
        return launch_kernel(router_kernel<T, V, false>, grid, dim3(kThreads), 0, stream, 1, p);
    const int size = p.experts / p.groups, lanes = size / V;
    const bool cut = p.groups > 1 && (lanes * V != size || (lanes & (lanes - 1)) != 0);
    const size_t smem = cut ? sizeof(float) * kThreads * V : 0;
    if (smem > 40 * 1024) {
        const cudaError_t err = cudaFuncSetAttribute(router_kernel<T, V, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (err != cudaSuccess) return err;
    }
    return launch_kernel(router_kernel<T, V, true>, grid, dim3(kThreads), smem, stream, 1, p);
}

// Experts a lane: the fewest that hold all, so that few lanes are empty.  16384 tokens, sigmoid, without and with a bias: 264 experts
// at 16 a lane 19.6 and 30 us, at 64 108 and 303; 512 19.5 and 33, 72 and 238; 520 to 1024 (at 64) 58 to 67 and 117 to 149, 2048 75
// and 203.  At 32 a lane none is built.
template <bool kGrad, typename T>
cudaError_t start_type(const ep_handle* h, const RouterParams& p, cudaStream_t stream) {
    if (p.experts <= 32) return start<kGrad, T, 1>(h, p, stream);
    if (p.experts <= 128) return start<kGrad, T, 4>(h, p, stream);
    if (p.experts <= 256) return start<kGrad, T, 8>(h, p, stream);
    if (p.experts <= 512) return start<kGrad, T, 16>(h, p, stream);
    return start<kGrad, T, 64>(h, p, stream);
}

template <bool kGrad>
ep_status launch(const ep_handle* h, const RouterParams& p, ep_dtype dtype, cudaStream_t stream) {
    if (p.tokens == 0) return EP_OK;
    DeviceGuard guard(h->device);
    const cudaError_t err = dtype == EP_FP32 ? start_type<kGrad, float>(h, p, stream) : start_type<kGrad, __nv_bfloat16>(h, p, stream);
    if (err != cudaSuccess) return cuda_fail(err, "router launch");
    return EP_OK;
}

ep_status check(const ep_handle* h, int64_t num_tokens, const void* logits, ep_dtype dtype, int32_t score, float scale, RouterParams* p) {
    if (h == nullptr) return fail(EP_ERR_INVALID_ARG, "handle is NULL");
    EP_CHECK_ARG(num_tokens >= 0 && num_tokens <= INT32_MAX, "num_tokens %lld outside [0, 2^31)", static_cast<long long>(num_tokens));
    EP_CHECK_ARG(dtype == EP_FP32 || dtype == EP_BF16, "logits must be EP_FP32 or EP_BF16");
    EP_CHECK_ARG(score == EP_SCORE_SOFTMAX || score == EP_SCORE_SIGMOID, "score must be EP_SCORE_SOFTMAX or EP_SCORE_SIGMOID");
    EP_CHECK_ARG(scale == scale && scale - scale == 0.0f, "scale must be finite");
    EP_CHECK_ARG(num_tokens == 0 || (logits && (reinterpret_cast<uintptr_t>(logits) & (dtype == EP_FP32 ? 3u : 1u)) == 0),
                 "logits is NULL or misaligned");
    p->logits = logits;
    p->tokens = num_tokens;
    p->experts = h->cfg.num_experts;
    p->topk = h->cfg.num_topk;
    p->softmax = score == EP_SCORE_SOFTMAX;
    p->scale = scale;
    p->groups = p->kept = 1;
    p->status = h->status;
    p->vector = aligned16(logits) && p->experts % (dtype == EP_FP32 ? 4 : 8) == 0;
    return EP_OK;
}

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" {

ep_status ep_router(ep_handle* h, int64_t num_tokens, const void* logits, ep_dtype logits_dtype, const float* bias,
                    const uint8_t* token_mask, int32_t score, int32_t num_groups, int32_t kept_groups, int32_t normalize,
                    float scale, int64_t* topk_idx, float* topk_weights, ep_stream_t stream) {
    EP_TRACE();
    RouterParams p = {};
    const ep_status st = check(h, num_tokens, logits, logits_dtype, score, scale, &p);
    if (st != EP_OK) return st;
    EP_CHECK_ARG(num_groups >= 1 && num_groups <= kMaxGroups && p.experts % num_groups == 0,
                 "num_groups %d must divide num_experts %d and be at most %d", num_groups, p.experts, kMaxGroups);
    EP_CHECK_ARG(kept_groups >= 1 && kept_groups <= num_groups, "kept_groups %d outside [1, num_groups=%d]", kept_groups, num_groups);
    EP_CHECK_ARG(num_tokens == 0 || (topk_idx && topk_weights && aligned8(topk_idx) && aligned4(topk_weights)),
                 "topk_idx or topk_weights is NULL or misaligned");
    EP_CHECK_ARG(aligned4(bias), "misaligned bias");
    p.bias = bias;
    p.token_mask = token_mask;
    p.groups = kept_groups == num_groups ? 1 : num_groups;  // all stay
    p.kept = kept_groups;
    p.normalize = normalize != 0;
    p.topk_idx = topk_idx;
    p.topk_weights = topk_weights;
    return launch<false>(h, p, logits_dtype, stream);
}

ep_status ep_router_grad(ep_handle* h, int64_t num_tokens, const void* logits, ep_dtype logits_dtype, const int64_t* topk_idx,
                         const float* d_topk_weights, int32_t score, int32_t normalize, float scale, void* d_logits,
                         ep_stream_t stream) {
    EP_TRACE();
    RouterParams p = {};
    const ep_status st = check(h, num_tokens, logits, logits_dtype, score, scale, &p);
    if (st != EP_OK) return st;
    EP_CHECK_ARG(num_tokens == 0 || (topk_idx && d_topk_weights && aligned8(topk_idx) && aligned4(d_topk_weights)),
                 "topk_idx or d_topk_weights is NULL or misaligned");
    EP_CHECK_ARG(num_tokens == 0 || (d_logits && (reinterpret_cast<uintptr_t>(d_logits) & (logits_dtype == EP_FP32 ? 3u : 1u)) == 0),
                 "d_logits is NULL or misaligned");
    p.chosen = topk_idx;
    p.d_weights = d_topk_weights;
    p.normalize = normalize != 0;
    p.d_logits = d_logits;
    p.vector = p.vector && aligned16(d_logits);
    return launch<true>(h, p, logits_dtype, stream);
}

}  // extern "C"
