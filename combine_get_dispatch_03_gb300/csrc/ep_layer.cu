// ep_layer.cu -- a whole mixture-of-experts layer for a few tokens, in two kernels (sm_103a).
//
//   y[t] = sum_k w[t][k] * W_down[e] * (silu(W_gate[e] x[t]) * (W_up[e] x[t])) + bias_0[t] + bias_1[t],   e = topk_idx[t][k]
//
// With up to 64 tokens the weights of the experts that they hit are all there is to read, so the weights are the rows of the
// tensor cores' products (128 at a time) and the tokens their columns (16 to 64): every byte of weights goes from memory to
// shared memory by tensor map and into tcgen05.mma once, and no product has empty rows of weights.
//   up     a tile is 128 gate rows and the 128 up rows beside them, times x: in bf16 that of ALL tokens (no gather, the columns
//          of tokens that are not the expert's are dropped), in FP8 that of the expert's.  silu(gate) * up goes to a workspace
//          row of (expert, token).
//   down   a tile is 256 output channels of one expert, times its rows of the workspace; a CTA adds up the weighted
//          results of the experts it works on in shared memory, [token][256 channels] in fp32.
//
// The work of a kernel is one row of units (a tile's step of 128 bytes of the contraction) that the CTAs share evenly, so
// that none waits for a last wave: 8 experts of 7168 x 2048 are 128 tiles of the first kernel on 152 SMs.  A tile that
// crosses CTAs leaves partial sums in the workspace; the last CTA to arrive (a ticket) adds them up in the CTAs' order.
//
// The second kernel is launched beside the first (programmatic dependent launch; for up to 8 tokens both may fit an SM,
// both_on_an_sm()) and fills its shared memory with weights, which do not hang on the first kernel, before it waits for it.
//
// FP8 weights: e4m3 with one scale per 128 x 128.  The tokens stay bf16: a block of 128 channels is scaled by a power of two
// and split into two e4m3 values (split_e4m3()), columns of their own in the products, so that nothing of bf16's eight bits is
// lost but what lies 2^-17 below the block's largest value.  A block's sums are added, scaled and added up in fp32 registers.
//
// What bounds it (6754 GB/s copied; experts of 7168 x 2048): bf16, memory: 1 token of 8 experts 117 us, 6.0 TB/s, 8 tokens of 23 309,
// 6.6, 64 of 32 457, 6.2.  FP8, with half of the bytes, the two kernels' start and end (1 token 79 us, 4.5 TB/s; 8 of 23 180, 5.6),
// then the splitting and the adding up of blocks (64 tokens of 32 experts 343, 4.1).  Small experts, 1024 x 512: 17 to 20 us for one
// token, launches and the sums of parts.
#include "ep_act.cuh"
#include "ep_groups.cuh"
#include "ep_handle.h"
#include "ep_maps.h"
#include "ep_tc.cuh"
#include "ep_trace.h"

namespace ep {
namespace {

constexpr int kMaxTokens = 64;
constexpr int kTile = 128;                  // rows of weights of a product
constexpr int kOps = 2;                     // products of a unit: gate and up, or two times 128 channels
constexpr int kSwap = 4;                    // up: tokens whose gates and ups change hands at a time
constexpr uint32_t kRow = 128;              // bytes of the contraction in a stage
constexpr uint32_t kTileBytes = kTile * kRow;
constexpr int col_step(bool fp8) { return fp8 ? 8 : 16; }  // tokens come in steps of 16 columns of products, FP8 two columns a token
constexpr int kMaxStages = 8;
constexpr int kLeastUnits = 4;
constexpr int kSumWarps = 8;                // warps 4 to 11: accumulators to sums and out
constexpr int kScaleRing = 16;              // blocks whose token scales are kept: more than stages and accumulators
constexpr int kSmallTokens = 8;             // up to which both kernels fit an SM
constexpr int buffers(int tokens) { return tokens <= kSmallTokens ? 4 : 2; }  // accumulators
constexpr int kBatchPairs = 4;              // of tokens that a splitting warp has in hand, and as many on their way
// Warps 12 on, FP8: the tokens' values in two e4m3 parts, so many warps for a unit.
constexpr int split_group(int tokens) { return tokens <= kSmallTokens ? 1 : 2; }
constexpr int split_warps(int tokens) { return 4 * split_group(tokens); }
static_assert(kScaleRing > kMaxStages + 4 + 1, "a block's scales outlive it");
constexpr int layer_threads(bool fp8, int tokens) { return (4 + kSumWarps + (fp8 ? split_warps(tokens) : 0)) * kWarpSize; }

struct LayerParams {
    const int64_t* topk_idx;
    const float* topk_weights;
    const int32_t* rank_mask;
    const uint8_t* tokens_x;   // up: x rows; down: the workspace's rows (bf16)
    const float* w_scales;     // FP8
    uint8_t* act;              // [rows][width] bf16
    float* partial;            // of this kernel: [CTA][2][token][gate, up or channels][128]
    int32_t* tickets;          // [CTAs], 0
    const uint8_t* bias_0;
    const uint8_t* bias_1;
    uint8_t* out;
    int32_t* status;
    uint64_t wait_limit_ns;
    int32_t tokens, tokens_per_rank, topk, experts, local_experts, hidden, width;
    int32_t cols;              // tokens, rounded up to col_step()
    uint32_t op_cols;          // columns of tensor memory for a product: cols, FP8 twice that
    int32_t stages, ctas, small;  // small: the variant of up to kSmallTokens
    uint32_t stage_bytes, tmem_columns;
};

__host__ __device__ inline int part_words(int ctas) { return (ctas + kWarpSize - 1) / kWarpSize; }

struct LayerMaps {
    CUtensorMap w, x;
};

struct LayerControl {
    uint64_t full[kMaxStages];
    uint64_t empty[kMaxStages];
    uint64_t acc_full[4];
    uint64_t acc_empty[4];
    uint64_t drained;
    uint32_t tmem;
    int32_t abort_flag;
    int32_t last_arrival[2];
    int32_t hits;
    int64_t sums[20];
};

// Which experts the tokens hit, in shared memory.
struct Routing {
    uint64_t* tokens;   // [experts] bit t: token t
    int32_t* begin;     // [experts] first workspace row of a hit expert
    uint16_t* hit;      // hit experts in ascending order
    float* weight;      // down: [rows] the weight of a row's (expert, token)
    uint8_t* token;     // up, FP8: [rows] the token
};

__device__ __forceinline__ int count_bits(uint64_t m) { return __popcll(static_cast<long long>(m)); }
__device__ __forceinline__ int lowest_bit(uint64_t m) { return __ffsll(static_cast<long long>(m)) - 1; }

// The expert of a token's slot that names `e`, -1 for none: as in the low-latency dispatch, a masked rank neither sends nor receives.
__device__ __forceinline__ int slot_expert(const LayerParams& p, uint32_t masked, int64_t e, int token) {
    if (e < 0 || e >= p.experts) return -1;
    if (masked && ((masked >> (token / p.tokens_per_rank) | masked >> (static_cast<int>(e) / p.local_experts)) & 1)) return -1;
    return static_cast<int>(e);
}

template <int THREADS, bool kWeights, bool kTokenOf>
__device__ __forceinline__ void build_routing(const Routing& t, const LayerParams& p, LayerControl& ctl) {
    const int slots = p.tokens * p.topk;
    // a thread's first slot is on its way meanwhile, as the ranks' masks are
    const int64_t raw0 = static_cast<int>(threadIdx.x) < slots ? p.topk_idx[threadIdx.x] : -1;
    const uint32_t masked = __ballot_sync(kFullMask, lane_id() < p.experts / p.local_experts && p.rank_mask[lane_id()] != 0);
    for (int e = threadIdx.x; e < p.experts; e += THREADS) t.tokens[e] = 0;
    __syncthreads();
    for (int s = threadIdx.x; s < slots; s += THREADS) {
        const int64_t raw = s == static_cast<int>(threadIdx.x) ? raw0 : p.topk_idx[s];
        if (raw < -1 || raw >= p.experts) report(p.status, EP_ERR_BAD_EXPERT);
        const int e = slot_expert(p, masked, raw, s / p.topk);
        if (e >= 0) atomicOr(reinterpret_cast<unsigned long long*>(&t.tokens[e]), 1ull << (s / p.topk));
    }
    __syncthreads();
    const int per = (p.experts + THREADS - 1) / THREADS;
    const int first = threadIdx.x * per, last = min(first + per, p.experts);
    int64_t mine = 0, all = 0;  // hit experts in the upper half, rows in the lower
    for (int e = first; e < last; ++e)
        if (t.tokens[e]) mine += (1ll << 32) + count_bits(t.tokens[e]);
    int64_t at = block_prefix<THREADS>(mine, ctl.sums, &all);
    for (int e = first; e < last; ++e) {
        if (!t.tokens[e]) continue;
        t.hit[at >> 32] = static_cast<uint16_t>(e);
        t.begin[e] = static_cast<int32_t>(at);
        at += (1ll << 32) + count_bits(t.tokens[e]);
    }
    if (threadIdx.x == 0) ctl.hits = static_cast<int>(all >> 32);
    __syncthreads();
    if constexpr (kTokenOf) {
        for (int s = threadIdx.x; s < slots; s += THREADS) {
            const int token = s / p.topk;
            const int e = slot_expert(p, masked, s == static_cast<int>(threadIdx.x) ? raw0 : p.topk_idx[s], token);
            if (e >= 0) t.token[t.begin[e] + count_bits(t.tokens[e] & ((1ull << token) - 1))] = static_cast<uint8_t>(token);
        }
        __syncthreads();
    }
    if constexpr (kWeights) {
        // an expert that a token names twice counts with both weights
        for (int s = threadIdx.x; s < slots; s += THREADS) {
            const int token = s / p.topk;
            const int e = slot_expert(p, masked, p.topk_idx[s], token);
            if (e < 0) continue;
            bool before = false;
            float w = 0.0f;
            for (int q = token * p.topk; q < (token + 1) * p.topk; ++q) {
                if (p.topk_idx[q] != e) continue;
                before |= q < s;
                w += p.topk_weights[q];
            }
            if (!before) t.weight[t.begin[e] + count_bits(t.tokens[e] & ((1ull << token) - 1))] = w;
        }
        __syncthreads();
    }
}

// A CTA's share of a kernel's units, and whose share a unit is.
struct Shares {
    int64_t units;
    int ctas;
    __device__ __forceinline__ int64_t begin(int cta) const { return units * cta / ctas; }
    __device__ __forceinline__ int owner(int64_t unit) const { return static_cast<int>(((unit + 1) * ctas - 1) / units); }
};

// A CTA's units [first, last): steps of `steps` of the contraction of tiles, by expert and then `across` (up), or
// across and then by expert (down).
template <bool kDown>
struct Work {
    const Routing& t;
    Shares shares;
    int64_t first, last;
    int hits, across, steps;
};

// A unit: a tile and a step of its contraction.  Moves on without divisions, which a thread alone waits for long.
template <bool kDown>
struct Unit {
    const Work<kDown>& w;
    int64_t at;
    int step, hit, col;  // col: first gate row (up) or output channel (down) of the tile
    int expert;
    uint64_t tokens;

    __device__ __forceinline__ Unit(const Work<kDown>& work, int64_t unit) : w(work), at(unit) {
        if (!more()) return;
        const int tile = static_cast<int>(unit / w.steps);
        step = static_cast<int>(unit - static_cast<int64_t>(tile) * w.steps);
        hit = kDown ? tile % w.hits : tile / w.across;
        col = kDown ? tile / w.hits * (kOps * kTile) : tile % w.across * kTile;
        look();
    }
    __device__ __forceinline__ bool more() const { return at < w.last; }
    __device__ __forceinline__ void look() {
        expert = w.t.hit[hit];
        tokens = w.t.tokens[expert];
    }
    // n units on, at most a tile's
    __device__ __forceinline__ void move(int n) {
        at += n;
        step += n;
        while (step >= w.steps && more()) {
            step -= w.steps;
            if (kDown) {
                if (++hit == w.hits) hit = 0, col += kOps * kTile;
            } else {
                col += kTile;
                if (col >= w.across * kTile) col = 0, ++hit;
            }
            look();
        }
    }
};

// What the roles of a CTA share.
template <bool kDown>
struct LayerRoles {
    const LayerMaps& maps;
    const LayerParams& p;
    const Routing& t;
    const Work<kDown>& work;
    LayerControl& ctl;
    Waits waits;
    uint8_t* stages;
    float* scales;   // FP8: [kScaleRing][kTokens] of the tokens' blocks
    float* sums;     // down: [tokens][256]; up: [kSwap][gate, up][128]
    uint32_t* parts;  // down: [tokens][part_words] a bit for each CTA whose part has something for the token
};

constexpr uint32_t kABytes = kOps * kTileBytes;

template <bool kFp8>
__device__ __forceinline__ int round_cols(int n) { return (n + col_step(kFp8) - 1) / col_step(kFp8) * col_step(kFp8); }

// Tokens of a unit: the expert's, in the first kernel's bf16 form all; as columns of products.
template <bool kFp8, bool kDown>
__device__ __forceinline__ int unit_tokens(const LayerParams& p, const Unit<kDown>& u) {
    return kFp8 || kDown ? count_bits(u.tokens) : p.tokens;
}

template <bool kFp8, bool kDown>
__device__ __forceinline__ int unit_cols(const LayerParams& p, const Unit<kDown>& u) {
    return kFp8 || kDown ? round_cols<kFp8>(count_bits(u.tokens)) : p.cols;
}

// Weights of a unit into its stage.
template <bool kFp8, bool kDown>
__device__ __forceinline__ void load_weights(const LayerRoles<kDown>& x, const Unit<kDown>& u, int stage) {
    const int k0 = u.step * (kFp8 ? 128 : 64);
    uint8_t* a = x.stages + stage * x.p.stage_bytes;
    const uint32_t bar = smem_u32(&x.ctl.full[stage]);
    tma_load_3d<1>(a, &x.maps.w, k0, u.col, u.expert, bar);
    tma_load_3d<1>(a + kTileBytes, &x.maps.w, k0, (kDown ? kTile : x.p.width) + u.col, u.expert, bar);
}

// Bytes and copies of a unit's tokens, bf16.
template <bool kDown>
__device__ __forceinline__ uint32_t token_bytes(const LayerParams& p, const Unit<kDown>& u) {
    return unit_cols<false>(p, u) * kRow;
}

template <bool kDown>
__device__ __forceinline__ void load_tokens(const LayerRoles<kDown>& x, const Unit<kDown>& u, int stage) {
    uint8_t* b = x.stages + stage * x.p.stage_bytes + kABytes;
    const uint32_t bar = smem_u32(&x.ctl.full[stage]);
    const int first = kDown ? x.t.begin[u.expert] : 0;
    const int cols = unit_cols<false>(x.p, u);
    for (int c = 0; c < cols; c += col_step(false)) tma_load_2d<1>(b + c * kRow, &x.maps.x, u.step * 64, first + c, bar);
}

// One thread: the loads.
template <bool kFp8, bool kDown>
__device__ __forceinline__ void layer_loads(const LayerRoles<kDown>& x) {
    const LayerParams& p = x.p;
    LayerControl& ctl = x.ctl;
    const Work<kDown>& w = x.work;
    Unit<kDown> u(w, w.first);
    bool ok = true;
    int stage = 0, used = 0;
    uint32_t phase = 0;
    if constexpr (kDown) {
        // Weights for every stage, then the first kernel's results.
        Unit<kDown> v = u;
        int ahead = 0;
        for (; ahead < p.stages && u.more(); ++ahead, u.move(1)) {
            bar_arrive_expect_tx<1>(smem_u32(&ctl.full[ahead]), kABytes + (kFp8 ? 0 : token_bytes<kDown>(p, u)));
            load_weights<kFp8, kDown>(x, u, ahead);
        }
        asm volatile("griddepcontrol.wait;" ::: "memory");
        if constexpr (!kFp8)
            for (int i = 0; i < ahead; ++i, v.move(1)) load_tokens<kDown>(x, v, i);
        used = ahead;
        if (ahead == p.stages) phase = 1;
        else stage = ahead;
    }
    for (; u.more(); u.move(1)) {
        ok = wait_phase(&ctl.empty[stage], phase ^ 1, x.waits);
        if (!ok) break;
        bar_arrive_expect_tx<1>(smem_u32(&ctl.full[stage]), kABytes + (kFp8 ? 0 : token_bytes<kDown>(p, u)));
        load_weights<kFp8, kDown>(x, u, stage);
        if constexpr (!kFp8) load_tokens<kDown>(x, u, stage);
        ++used;
        if (++stage == p.stages) stage = 0, phase ^= 1;
    }
    // Copies and products in flight end before the memory goes away: the products have read every copy when the last stages
    // are free again; where some warp gave up, the copies that complete a stage, each wait with a limit, and a
    // hundred times what a copy takes for those of a stage that another warp left incomplete.
    for (int i = 0; i < p.stages && used > 0; ++i, --used) {
        if (stage == 0) phase ^= 1;
        stage = (stage == 0 ? p.stages : stage) - 1;
        if (ok) ok = wait_phase(&ctl.empty[stage], phase, x.waits);
        if (ok) continue;
        for (int k = 0; k < (1 << 8) && !mbar_try_wait(&ctl.full[stage], phase); ++k) {
        }
    }
    for (int k = 0; k < (1 << 12) && !mbar_try_wait(&ctl.drained, 0); ++k) {
    }
    if (ctl.abort_flag)
        for (const uint64_t begin = global_ns(); global_ns() - begin < 1000000;) __nanosleep(1000);
}

// One thread: the products.
template <bool kFp8, int kTokens, bool kDown>
__device__ __forceinline__ void layer_products(const LayerRoles<kDown>& x) {
    const LayerParams& p = x.p;
    LayerControl& ctl = x.ctl;
    const Work<kDown>& w = x.work;
    int stage = 0, buf = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool first = true;  // of an accumulator
    for (Unit<kDown> u(w, w.first); u.more(); u.move(1)) {
        if (!wait_phase(&ctl.full[stage], phase, x.waits)) break;
        if (first && !wait_phase(&ctl.acc_empty[buf], acc_phase ^ 1, x.waits)) break;
        tc_fence_after();
        const uint32_t cols = (kFp8 ? 2 : 1) * unit_cols<kFp8>(p, u);  // FP8: both parts' columns
        const uint32_t idesc = mma_desc(kFp8 ? 0 : 1, false, false, kTile, cols);
        const uint32_t a = smem_u32(x.stages) + stage * p.stage_bytes;
        const uint32_t d = ctl.tmem + buf * kOps * p.op_cols;
        const uint64_t db = smem_desc(a + kABytes, 16);
#pragma unroll
        for (int op = 0; op < kOps; ++op) {
            const uint64_t da = smem_desc(a + op * kTileBytes, 16);
#pragma unroll
            for (int i = 0; i < 4; ++i) tc_mma<1, kFp8>(d + op * p.op_cols, da + i * 2, db + i * 2, idesc, !first || i);
        }
        tc_commit<1>(&ctl.empty[stage]);
        first = false;
        if (kFp8 || u.step == w.steps - 1 || u.at == w.last - 1) {
            // this thread's own arrival passes on what it acquired with the stage: the tokens' scales
            bar_arrive<1>(smem_u32(&ctl.acc_full[buf]));
            tc_commit<1>(&ctl.acc_full[buf]);
            if (++buf == buffers(kTokens)) buf = 0, acc_phase ^= 1;
            first = true;
        }
        if (++stage == p.stages) stage = 0, phase ^= 1;
    }
    tc_commit<1>(&ctl.drained);
}

// Eight channels of a token times 2^m, as two e4m3 values each: the nearest, and the nearest to what is left.  Scaled so
// that the block's largest value lies in [128, 256), the second leaves at most 2^-10, 2^-17 of the largest; a bf16 value
// within 2^-9 of the largest is exact (4 + 4 bits).
__device__ __forceinline__ void split_e4m3(const float (&f)[8], float mult, uint2* high, uint2* low) {
    uint32_t h[2] = {0, 0}, l[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 v = __floats2half2_rn(f[2 * i] * mult, f[2 * i + 1] * mult);  // eight bits of eleven, to 2^-25
        const __nv_fp8x2_storage_t code = __nv_cvt_halfraw2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
        const __half2 rest = __hsub2(v, static_cast<__half2>(__nv_cvt_fp8x2_to_halfraw2(code, __NV_E4M3)));  // exact
        h[i / 2] |= static_cast<uint32_t>(code) << (i % 2 * 16);
        l[i / 2] |= static_cast<uint32_t>(__nv_cvt_halfraw2_to_fp8x2(rest, __NV_SATFINITE, __NV_E4M3)) << (i % 2 * 16);
    }
    *high = make_uint2(h[0], h[1]);
    *low = make_uint2(l[0], l[1]);
}

// FP8: the tokens' blocks of a unit, split, into the place and order in which a tensor-map load would put them: a row
// for each token's first part, then one for each second.  Groups of warps take units in turn, so that each has several units' time
// for a round trip to memory; half a warp has a token's 128 channels, and a batch's values are loaded before the one before it
// is worked on.  No more groups than stages: one that waits for a stage's use has filled a stage after the use before the last,
// so that the barrier's parity tells the two uses apart.
template <int kTokens, bool kDown>
__device__ __forceinline__ void layer_splits(const LayerRoles<kDown>& x, int warp) {
    constexpr int kGroup = split_group(kTokens);
    constexpr int kBatch = 2 * kBatchPairs;  // tokens
    const LayerParams& p = x.p;
    LayerControl& ctl = x.ctl;
    const Work<kDown>& w = x.work;
    const int64_t row_bytes = 2 * static_cast<int64_t>(kDown ? p.width : p.hidden);
    const int half = lane_id() >> 4, piece = lane_id() & 15;
    const int groups = min(split_warps(kTokens) / kGroup, p.stages), group = warp / kGroup;
    const int begin = warp % kGroup * kBatch;  // of a unit's tokens
    if (group >= groups) return;
    // what is loaded next: tokens [first, count) of a unit
    Unit<kDown> next(w, w.first + group);
    int next_first = 0, next_count = 0;
    int next_begin = 0;
    const uint8_t* next_at = nullptr;
    auto enter = [&] {
        next_first = begin;
        next_count = 0;
        if (!next.more()) return;
        next_count = count_bits(next.tokens);
        next_begin = x.t.begin[next.expert];
        next_at = p.tokens_x + next.step * 256 + piece * 16;
    };
    int4 ahead[kBatchPairs];
    auto fetch = [&] {
#pragma unroll
        for (int i = 0; i < kBatchPairs; ++i) {
            ahead[i] = make_int4(0, 0, 0, 0);
            const int q = next_first + 2 * i + half;
            if (q < next_count) {
                const int row = next_begin + q;
                ahead[i] = __ldcg(reinterpret_cast<const int4*>(next_at + (kDown ? row : x.t.token[row]) * row_bytes));
            }
        }
    };
    auto advance = [&] {
        next_first += kBatch * kGroup;
        if (next_first >= next_count) next.move(groups), enter();
        fetch();
    };
    if (kDown) asm volatile("griddepcontrol.wait;" ::: "memory");
    enter();
    fetch();
    int stage = group;
    uint32_t phase = 0;
    for (int64_t unit = w.first + group; unit < w.last; unit += groups) {
        const int count = next_count;  // at least one
        const uint32_t low_part = round_cols<true>(count) * kRow;
        if (!warp_wait(&ctl.empty[stage], phase ^ 1, x.waits)) break;
        uint8_t* b = x.stages + stage * p.stage_bytes + kABytes;
        float* scales = x.scales + static_cast<int>((unit - w.first) % kScaleRing) * kTokens;
        if (begin >= count) advance();  // none for this warp
        for (int first = begin; first < count; first += kBatch * kGroup) {
            int4 value[kBatchPairs];
#pragma unroll
            for (int i = 0; i < kBatchPairs; ++i) value[i] = ahead[i];
            advance();
#pragma unroll
            for (int i0 = 0; i0 < kBatchPairs; i0 += 2) {  // two at a time: there are registers for no more
                if (first + 2 * i0 >= count) break;
                float f[2][8], most[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    unpack8(value[i0 + i], f[i]);
                    most[i] = absmax8(f[i]);
                }
#pragma unroll
                for (int o = 8; o > 0; o >>= 1)
#pragma unroll
                    for (int i = 0; i < 2; ++i) most[i] = fmaxf(most[i], __shfl_xor_sync(kFullMask, most[i], o));
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    // 2^(7 - exponent), at most 2^126; an infinite value has no scale and makes the token's sums NaN, as NaN does
                    const int exponent = static_cast<int>(__float_as_uint(most[i]) >> 23);
                    const int up = min(134 - exponent, 126);
                    uint2 high, low;
                    split_e4m3(f[i], __uint_as_float(static_cast<uint32_t>(127 + up) << 23), &high, &low);
                    const int t = first + 2 * (i0 + i) + half;
                    if (t < count) {
                        const uint32_t at = t * kRow + (((piece >> 1) ^ (t & 7)) << 4) + (piece & 1) * 8;
                        *reinterpret_cast<uint2*>(b + at) = high;
                        *reinterpret_cast<uint2*>(b + low_part + at) = low;
                        if (piece == 0) scales[t] = exponent == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
                    }
                }
            }
        }
        fence_async_smem();
        __syncwarp();
        if (lane_id() == 0) bar_arrive<1>(smem_u32(&ctl.full[stage]));
        stage += groups;  // at most once around
        if (stage >= p.stages) stage -= p.stages, phase ^= 1;
    }
}

// 8 fp32 columns of this warp's 32 lanes of tensor memory: starts the load.
__device__ __forceinline__ void tc_ld8(uint32_t addr, uint32_t (&v)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(addr));
}

// Waits for this thread's loads; no use of `v` is scheduled before it.
__device__ __forceinline__ void tc_wait8(uint32_t (&v)[8]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7])
                 :: "memory");
}

__device__ __forceinline__ void sum_warps_barrier() { asm volatile("bar.sync 1, %0;" ::"n"(kSumWarps * kWarpSize) : "memory"); }

// After the sum warps wrote a part of what `parts` CTAs add up: whether this CTA is the last to arrive, and may read all.
template <bool kDown>
__device__ __forceinline__ bool last_to_arrive(const LayerRoles<kDown>& x, int ticket, int parts, int& turn) {
    sum_warps_barrier();
    if (threadIdx.x == 4 * kWarpSize) {
        const bool last = arrive_at(x.p.tickets + ticket) == parts - 1;
        if (last) x.p.tickets[ticket] = 0;  // for the next call
        x.ctl.last_arrival[turn & 1] = last;
    }
    sum_warps_barrier();
    return *const_cast<volatile int32_t*>(&x.ctl.last_arrival[turn++ & 1]) != 0;  // the other word is written next
}

// The sums of a run of one tile's units that this CTA has, for all columns of a thread's row of one product.
template <bool kFp8, int kTokens, bool kDown>
__device__ __forceinline__ void read_sums(const LayerRoles<kDown>& x, int steps, int quarter, int op, const Unit<kDown>& u, int& buf,
                                          uint32_t& acc_phase, bool& ok, float (&v)[kTokens]) {
    const LayerParams& p = x.p;
    LayerControl& ctl = x.ctl;
    const int count = unit_tokens<kFp8>(p, u), cols = unit_cols<kFp8>(p, u);
#pragma unroll
    for (int t = 0; t < kTokens; ++t) v[t] = 0.0f;
    const float* ws = nullptr;
    float w_next = 0.0f;
    if constexpr (kFp8) {
        const int rows = (kDown ? p.hidden : 2 * p.width) / kFp8Group;
        const int row = min(u.col / kFp8Group + op * (kDown ? 1 : p.width / kFp8Group), rows - 1);  // the last channels: no second half
        ws = p.w_scales + (static_cast<int64_t>(u.expert) * rows + row) * x.work.steps + u.step;
        w_next = __ldg(ws);
    }
    for (int s = 0; s < (kFp8 ? steps : 1); ++s) {
        const float w = w_next;
        if constexpr (kFp8) w_next = __ldg(ws + min(s + 1, steps - 1));
        if (ok) ok = warp_wait(&ctl.acc_full[buf], acc_phase, x.waits);
        if (!ok) return;
        tc_fence_after();
        const uint32_t from = ctl.tmem + (static_cast<uint32_t>(quarter * 32) << 16) + (buf * kOps + op) * p.op_cols;
        const float4* scales = reinterpret_cast<const float4*>(x.scales + static_cast<int>((u.at + s - x.work.first) % kScaleRing) * kTokens);
#pragma unroll
        for (int c = 0; c < kTokens; c += 8) {
            if (c >= count) break;
            uint32_t r[8], low[8];
            tc_ld8(from + c, r);
            if constexpr (kFp8) {
                tc_ld8(from + cols + c, low);
                tc_wait8(low);
            }
            tc_wait8(r);
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
                float4 f = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
                if constexpr (kFp8) f = scales[(c + i) / 4];
                const float ff[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float d = __uint_as_float(r[i + j]);
                    if constexpr (kFp8) v[c + i + j] = fmaf(d + __uint_as_float(low[i + j]), ff[j] * w, v[c + i + j]);
                    else v[c + i + j] = d;
                }
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane_id() == 0) bar_arrive<1>(smem_u32(&ctl.acc_empty[buf]));
        if (++buf == buffers(kTokens)) buf = 0, acc_phase ^= 1;
    }
}

// The same bits, which the compiler does not take apart early: 64 predicates have no registers.
__device__ __forceinline__ uint64_t unseen(uint64_t bits) {
    asm volatile("" : "+l"(bits));
    return bits;
}

// bf16, as the second product's operand is.
__device__ __forceinline__ void put_act(const LayerParams& p, int64_t act_row, int col, float gate, float up) {
    if (col < p.width)
        *reinterpret_cast<__nv_bfloat16*>(p.act + 2 * (act_row * p.width + col)) = __float2bfloat16_rn(activate(EP_ACT_SILU, both(gate)).x * up);
}

// Eight warps of the first kernel: accumulators to silu(gate) * up.  Four have the tile's gates, four its ups, each 32 rows and
// all tokens.
template <bool kFp8, int kTokens>
__device__ __forceinline__ void up_sums(const LayerRoles<false>& x, int warp) {
    const LayerParams& p = x.p;
    const Work<false>& w = x.work;
    const int quarter = warp & 3, op = (warp - 4) >> 2;
    const int row = quarter * 32 + lane_id();
    int buf = 0;
    uint32_t acc_phase = 0;
    int turn = 0;
    bool ok = true;
    for (Unit<false> u(w, w.first); u.more();) {
        const int steps = static_cast<int>(min(static_cast<int64_t>(w.steps - u.step), w.last - u.at));
        float v[kTokens];
        read_sums<kFp8, kTokens, false>(x, steps, quarter, op, u, buf, acc_phase, ok, v);
        const int count = count_bits(u.tokens);
        const uint64_t columns = kFp8 ? ~0ull >> (64 - count) : u.tokens;  // of the expert's tokens, in order
        const int64_t first = x.t.begin[u.expert];
        const int thread = threadIdx.x - 4 * kWarpSize;
        if (steps == w.steps) {
            // through shared memory, kSwap tokens at a time
            for (int base = 0; base < count; base += kSwap) {
                int q = -base;  // the token's number among the expert's, from base
                const uint64_t has = unseen(columns);
#pragma unroll
                for (int t = 0; t < kTokens; ++t)
                    if (has >> t & 1) {
                        if (q >= 0 && q < kSwap) x.sums[(q * kOps + op) * kTile + row] = v[t];
                        ++q;
                    }
                sum_warps_barrier();
                for (int i = thread; i < min(kSwap, count - base) * kTile; i += kSumWarps * kWarpSize) {
                    const float* from = x.sums + i / kTile * (kOps * kTile) + i % kTile;
                    put_act(p, first + base + i / kTile, u.col + i % kTile, from[0], from[kTile]);
                }
                sum_warps_barrier();
            }
        } else {
            const int64_t tile0 = u.at - u.step;
            const int a = w.shares.owner(tile0), b = w.shares.owner(tile0 + w.steps - 1);
            const int64_t each = static_cast<int64_t>(p.tokens) * kOps * kTile;
            float* own = p.partial + (2 * static_cast<int64_t>(blockIdx.x) + (u.step == 0)) * each + op * kTile + row;
            const uint64_t has = unseen(columns);
#pragma unroll
            for (int t = 0; t < kTokens; ++t)
                if (has >> t & 1) own[t * (kOps * kTile)] = v[t];
            if (last_to_arrive(x, a, b - a + 1, turn)) {
                // two tokens at a time, a thread one of a token's rows: the parts in the CTAs' order
                uint64_t left = columns;
                if (thread >= kTile) left &= left - 1;
                for (int q = thread / kTile; q < count; q += 2) {
                    const float* part = p.partial + (lowest_bit(left) * kOps) * kTile + thread % kTile;
                    float gate = __ldcg(part + (2 * static_cast<int64_t>(a) + 1) * each), up = __ldcg(part + (2 * static_cast<int64_t>(a) + 1) * each + kTile);
#pragma unroll 8
                    for (int c = a + 1; c <= b; ++c) {
                        gate += __ldcg(part + 2 * static_cast<int64_t>(c) * each);
                        up += __ldcg(part + 2 * static_cast<int64_t>(c) * each + kTile);
                    }
                    put_act(p, first + q, u.col + thread % kTile, gate, up);
                    left &= left - 1;
                    left &= left - 1;
                }
            }
        }
        u.move(steps);
    }
}

// The sum warps' 256 channels from `col` of all tokens, four channels a thread and four tokens at a time; sum(t, c): the sums of
// token t's four channels from c.
template <typename Sum>
__device__ __forceinline__ void put_outputs(const LayerParams& p, int col, Sum sum) {
    const int thread = threadIdx.x - 4 * kWarpSize, c = thread % 64 * 4;
    if (col + c >= p.hidden) return;
#pragma unroll 1
    for (int t = thread / 64; t < p.tokens; t += 4) {
        const int64_t at = 2 * (static_cast<int64_t>(t) * p.hidden + col + c);
        const uint2 b0 = p.bias_0 ? *reinterpret_cast<const uint2*>(p.bias_0 + at) : make_uint2(0, 0);
        const uint2 b1 = p.bias_1 ? *reinterpret_cast<const uint2*>(p.bias_1 + at) : make_uint2(0, 0);
        float4 s = sum(t, c);
        s.x += bf16_lo(b0.x) + bf16_lo(b1.x), s.y += bf16_hi(b0.x) + bf16_hi(b1.x);
        s.z += bf16_lo(b0.y) + bf16_lo(b1.y), s.w += bf16_hi(b0.y) + bf16_hi(b1.y);
        *reinterpret_cast<uint2*>(p.out + at) = make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
    }
}

// The tokens that a CTA's part of some channels can have something for: those of its experts there, all where these are many.
__device__ __forceinline__ uint64_t part_tokens(const Work<true>& w, int cta, int64_t tile0, int64_t each_tile) {
    const int64_t first = max(w.shares.begin(cta), tile0) - tile0, last = min(w.shares.begin(cta + 1), tile0 + each_tile) - 1 - tile0;
    const int from = static_cast<int>(first / w.steps), to = static_cast<int>(last / w.steps);
    if (to - from >= 32) return ~0ull;
    uint64_t m = 0;
    for (int i = from; i <= to; ++i) m |= w.t.tokens[w.t.hit[i]];
    return m;
}

// Eight warps of the second kernel: accumulators to the tokens' weighted sums.  A thread has one of the tile's channels, so
// that a sum belongs to one thread whatever the expert.
template <bool kFp8, int kTokens>
__device__ __forceinline__ void down_sums(const LayerRoles<true>& x, int warp) {
    constexpr int kChannels = kOps * kTile;
    const LayerParams& p = x.p;
    const Work<true>& w = x.work;
    const int quarter = warp & 3, op = (warp - 4) >> 2;
    const int mine = op * kTile + quarter * 32 + lane_id();
    if (w.hits == 0) {  // no token has an expert
        for (int j = blockIdx.x; j < w.across; j += gridDim.x)
            put_outputs(p, j * kChannels, [](int, int) { return make_float4(0.0f, 0.0f, 0.0f, 0.0f); });
        return;
    }
    float* const sums = x.sums + mine;
    for (int t = 0; t < p.tokens; ++t) sums[t * kChannels] = 0.0f;
    const int64_t each_tile = static_cast<int64_t>(w.hits) * w.steps;  // units of kChannels
    int buf = 0;
    uint32_t acc_phase = 0;
    int turn = 0;
    bool ok = true;
    int64_t tile0 = w.first / each_tile * each_tile;  // first unit of the channels that are being summed
    for (Unit<true> u(w, w.first); u.more();) {
        const int steps = static_cast<int>(min(static_cast<int64_t>(w.steps - u.step), w.last - u.at));
        float v[kTokens];
        read_sums<kFp8, kTokens, true>(x, steps, quarter, op, u, buf, acc_phase, ok, v);
        const float* weight = x.t.weight + x.t.begin[u.expert];
        uint64_t left = u.tokens;
#pragma unroll
        for (int q = 0; q < kTokens; ++q) {
            if (left == 0) break;
            sums[lowest_bit(left) * kChannels] += weight[q] * v[q];
            left &= left - 1;
        }
        const int col = u.col;
        u.move(steps);
        if (u.more() && u.at < tile0 + each_tile) continue;  // more of these channels
        const bool whole = tile0 >= w.first && u.at == tile0 + each_tile;
        if (whole) {
            sum_warps_barrier();
            put_outputs(p, col, [&](int t, int c) { return *reinterpret_cast<const float4*>(x.sums + t * kChannels + c); });
            sum_warps_barrier();
        } else {
            const int a = w.shares.owner(tile0), b = w.shares.owner(tile0 + each_tile - 1);
            const int64_t each = static_cast<int64_t>(p.tokens) * kChannels;
            float* own = p.partial + (2 * static_cast<int64_t>(blockIdx.x) + (tile0 >= w.first)) * each + mine;
            const uint64_t has = part_tokens(w, blockIdx.x, tile0, each_tile);
            for (int t = 0; t < p.tokens; ++t)
                if (has >> t & 1) own[t * kChannels] = sums[t * kChannels];
            if (last_to_arrive(x, a, b - a + 1, turn)) {  // the same for all
                // which parts a token is in, a warp 32 parts at a time
                const int words = part_words(p.ctas);
                for (int i = warp - 4; i <= (b - a) / kWarpSize; i += kSumWarps) {
                    const int c = a + i * kWarpSize + lane_id();
                    const uint64_t m = c <= b ? part_tokens(w, c, tile0, each_tile) : 0;
                    for (int t = 0; t < p.tokens; ++t) {
                        const uint32_t in = __ballot_sync(kFullMask, m >> t & 1);
                        if (lane_id() == 0) x.parts[t * words + i] = in;
                    }
                }
                sum_warps_barrier();
                put_outputs(p, col, [&](int t, int c) {
                    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    for (int word = 0; word <= (b - a) / kWarpSize; ++word) {
                        uint32_t in = x.parts[t * words + word];
                        const int c0 = a + word * kWarpSize;
                        while (in) {  // four parts on their way
                            float4 v[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const int cta = c0 + __ffs(in) - 1;
                                v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                                if (in) v[k] = __ldcg(reinterpret_cast<const float4*>(p.partial + (2 * static_cast<int64_t>(cta) + (cta == a)) * each + t * kChannels + c));
                                in &= in - 1;
                            }
#pragma unroll
                            for (int k = 0; k < 4; ++k) s.x += v[k].x, s.y += v[k].y, s.z += v[k].z, s.w += v[k].w;
                        }
                    }
                    return s;
                });
            }
        }
        for (int t = 0; t < p.tokens; ++t) sums[t * kChannels] = 0.0f;
        tile0 += each_tile;
    }
}

// The dynamic shared memory of a kernel, after alignment to 1024: stages, then the rest.
struct Layout {
    uint32_t tokens, parts, begin, hit, weight, token, scales, sums, bytes;
};

__host__ __device__ inline Layout layer_layout(const LayerParams& p, bool fp8, bool down) {
    Layout l;
    uint32_t at = p.stages * p.stage_bytes;
    l.scales = at, at += fp8 ? 4u * kScaleRing * (p.small ? kSmallTokens : kMaxTokens) : 0u;
    l.sums = at, at += 4u * kTile * kOps * (down ? p.tokens : kSwap);
    l.tokens = at, at += 8u * p.experts;
    l.parts = at, at += down ? 4u * part_words(p.ctas) * p.tokens : 0u;
    l.begin = at, at += 4u * p.experts;

    l.weight = at, at += down ? 4u * p.tokens * p.topk : 0u;
    const int most = p.tokens * p.topk < p.experts ? p.tokens * p.topk : p.experts;
    l.hit = at, at += 2u * most;
    l.token = at, at += fp8 && !down ? p.tokens * p.topk : 0u;
    l.bytes = at;
    return l;
}

template <bool kFp8, int kTokens, bool kDown>
__global__ void __launch_bounds__(layer_threads(kFp8, kTokens), kTokens <= kSmallTokens ? 2 : 1)
    layer_kernel(const __grid_constant__ LayerMaps maps, const LayerParams p) {
    constexpr int kThreads = layer_threads(kFp8, kTokens);
    extern __shared__ uint8_t raw[];
    __shared__ LayerControl ctl;
    uint8_t* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    const Layout l = layer_layout(p, kFp8, kDown);
    const Routing t = {reinterpret_cast<uint64_t*>(smem + l.tokens), reinterpret_cast<int32_t*>(smem + l.begin),
                       reinterpret_cast<uint16_t*>(smem + l.hit), reinterpret_cast<float*>(smem + l.weight), smem + l.token};
    const int warp = threadIdx.x / kWarpSize;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(&ctl.full[i], kFp8 ? 1 + split_group(kTokens) : 1);
            mbar_init(&ctl.empty[i], 1);
        }
        for (int i = 0; i < buffers(kTokens); ++i) {
            mbar_init(&ctl.acc_full[i], 2);
            mbar_init(&ctl.acc_empty[i], kSumWarps);
        }
        mbar_init(&ctl.drained, 1);
        ctl.abort_flag = 0;
        fence_barrier_init();
        prefetch_map(&maps.w);
        prefetch_map(&maps.x);
    }
    if (warp == 1) tmem_alloc<1>(&ctl.tmem, p.tmem_columns);
    // The second kernel starts when every CTA of the first is past its own wait: what lay in memory before the call is
    // there, the routing and the weights among it; only the first kernel's results are waited for, where they are read.
    if constexpr (kDown) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    else pdl_enter();
    build_routing<kThreads, kDown, kFp8 && !kDown>(t, p, ctl);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();

    const int steps = ((kDown ? p.width : p.hidden) * (kFp8 ? 1 : 2) + static_cast<int>(kRow) - 1) / static_cast<int>(kRow);
    const int across = kDown ? (p.hidden + kOps * kTile - 1) / (kOps * kTile) : (p.width + kTile - 1) / kTile;
    const int64_t units = static_cast<int64_t>(ctl.hits) * across * steps;
    // a CTA has kLeastUnits at least: a part costs its sum more than their loads
    const Shares shares = {units, static_cast<int>(min((units + kLeastUnits - 1) / kLeastUnits, static_cast<int64_t>(gridDim.x)))};
    const bool works = static_cast<int>(blockIdx.x) < shares.ctas;
    const Work<kDown> work = {t, shares, works ? shares.begin(blockIdx.x) : 0, works ? shares.begin(blockIdx.x + 1) : 0,
                              ctl.hits, across, steps};
    const LayerRoles<kDown> x = {maps, p, t, work, ctl, {&ctl.abort_flag, p.status, p.wait_limit_ns}, smem,
                                 reinterpret_cast<float*>(smem + l.scales), reinterpret_cast<float*>(smem + l.sums),
                                 reinterpret_cast<uint32_t*>(smem + l.parts)};
    // FP8: registers move from the loads' and products' warps to the others: of 640 threads of 96 (61440) 128 * 40 + 256 * 136 +
    // 256 * 80, of 512 of 64 (32768, so that two CTAs fit an SM) 128 * 40 + 256 * 72 + 128 * 72.
    constexpr bool kMany = kTokens > kSmallTokens;
    if (warp < 4) {
        if constexpr (kFp8) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == 0) {
            if (elect_one()) layer_loads<kFp8, kDown>(x);
        } else if (warp == 1) {
            if (elect_one()) layer_products<kFp8, kTokens, kDown>(x);
        }
    } else if (warp < 4 + kSumWarps) {
        if constexpr (kFp8 && kMany) asm volatile("setmaxnreg.inc.sync.aligned.u32 136;");
        else if constexpr (kFp8) asm volatile("setmaxnreg.inc.sync.aligned.u32 72;");
        if constexpr (kDown) down_sums<kFp8, kTokens>(x, warp);
        else up_sums<kFp8, kTokens>(x, warp);
    } else if constexpr (kFp8) {
        if constexpr (kMany) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        else asm volatile("setmaxnreg.inc.sync.aligned.u32 72;");
        layer_splits<kTokens, kDown>(x, warp - 4 - kSumWarps);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc<1>(ctl.tmem, p.tmem_columns);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

constexpr int kMostSmem = 226 * 1024;   // dynamic, of one kernel
constexpr int kBothSmem = 224 * 1024;   // of the two together, for an SM that holds a CTA of each
constexpr int kUpStages = 3;            // of the first kernel, then; the second takes what is left

int64_t align256(int64_t v) { return (v + 255) / 256 * 256; }

struct Workspace {
    int64_t up_partial, down_partial, bytes;  // the activations come first
};

Workspace workspace_of(const ep_handle* h, int64_t tokens, int32_t width) {
    const int64_t rows = tokens * (h->cfg.num_topk < h->cfg.num_experts ? h->cfg.num_topk : h->cfg.num_experts);
    const int64_t ctas = h->plan.num_sms;
    Workspace w;
    w.up_partial = align256(rows * width * 2);
    w.down_partial = w.up_partial + align256(ctas * 2 * tokens * kOps * kTile * 4);
    w.bytes = w.down_partial + align256(ctas * 2 * tokens * kOps * kTile * 4);
    return w;
}

template <bool kFp8, int kTokens>
cudaError_t plan_kernels(int smem) {
    cudaError_t err = cudaFuncSetAttribute(layer_kernel<kFp8, kTokens, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err == cudaSuccess)
        err = cudaFuncSetAttribute(layer_kernel<kFp8, kTokens, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    return err;
}

cudaError_t plan_layer() {
    constexpr int kSmem = kMostSmem;
    cudaError_t err = plan_kernels<false, kSmallTokens>(kSmem);
    if (err == cudaSuccess) err = plan_kernels<false, kMaxTokens>(kSmem);
    if (err == cudaSuccess) err = plan_kernels<true, kSmallTokens>(kSmem);
    if (err == cudaSuccess) err = plan_kernels<true, kMaxTokens>(kSmem);
    return err;
}

// Tensor memory and stages of a kernel that may have `room` bytes of shared memory and `most` stages; the bytes it takes.
int size_kernel(LayerParams* p, bool fp8, bool down, int room, int most) {
    p->cols = (p->tokens + col_step(fp8) - 1) / col_step(fp8) * col_step(fp8);
    p->op_cols = (fp8 ? 2 : 1) * p->cols;
    p->stage_bytes = kABytes + p->op_cols * kRow;
    p->tmem_columns = 32;
    while (p->tmem_columns < buffers(p->small ? kSmallTokens : kMaxTokens) * kOps * p->op_cols) p->tmem_columns *= 2;
    p->stages = 0;
    const int stages = (room - static_cast<int>(layer_layout(*p, fp8, down).bytes) - 1024) / static_cast<int>(p->stage_bytes);
    p->stages = stages < most ? stages : most;
    return static_cast<int>(layer_layout(*p, fp8, down).bytes) + 1024;
}

// Whether the two kernels shall fit an SM together.  Alone each has more stages, and the second starts when the first ends:
// one bf16 token through 8 of 32 experts of 7168 x 2048 121 us together and 119 alone, 8 tokens through 23 of them 315 and 308, but 8
// experts of 1024 x 512 18.3 and 20.9, 4 tokens of 2048 x 1024 51 and 59; FP8 81 and 85, 184 and 185, 20.8 and 21.6, 38 and 44.
bool both_on_an_sm(const LayerParams& p, bool fp8) {
    if (p.tokens > kSmallTokens) return false;
    const int64_t hits = p.tokens * p.topk < p.experts ? p.tokens * p.topk : p.experts;
    return fp8 || 6 * hits * p.hidden * p.width < (INT64_C(1) << 29);
}

// Both kernels' sizes: together on an SM if they fit with two stages each, else each for itself.
ep_status size_kernels(LayerParams* up, LayerParams* down, bool fp8, bool small, int* up_smem, int* down_smem) {
    up->small = down->small = small;
    if (small) {
        *up_smem = size_kernel(up, fp8, false, kMostSmem, kUpStages);
        *down_smem = size_kernel(down, fp8, true, kBothSmem - *up_smem, kMaxStages);
        if (up->stages >= 2 && down->stages >= 2) return EP_OK;
    }
    *up_smem = size_kernel(up, fp8, false, kMostSmem, kMaxStages);
    *down_smem = size_kernel(down, fp8, true, kMostSmem, kMaxStages);
    if (up->stages < 2 || down->stages < 2) return fail(EP_ERR_UNSUPPORTED, "the layer's tables need too much shared memory");
    return EP_OK;
}

template <bool kFp8, int kTokens, bool kDown>
cudaError_t start(const ep_handle* h, const LayerMaps& m, const LayerParams& p, int smem, cudaStream_t stream) {
    return launch_kernel(layer_kernel<kFp8, kTokens, kDown>, dim3(h->plan.num_sms), dim3(layer_threads(kFp8, kTokens)), smem, stream, 1, m, p);
}

template <bool kFp8>
ep_status run(ep_handle* h, LayerParams p, const void* x, const void* w_up, const float* up_scales, const void* w_down,
              const float* down_scales, uint8_t* workspace, cudaStream_t stream) {
    DeviceGuard guard(h->device);
    const ep_status planned = plan_once(&h->plan.layer_ready, [] { return plan_layer(); });
    if (planned != EP_OK) return planned;
    const Workspace ws = workspace_of(h, p.tokens, p.width);
    const uint64_t H = p.hidden, I = p.width, E = p.experts, esize = kFp8 ? 1 : 2;
    const Element element = kFp8 ? Element::kFp8 : Element::kBf16;
    const uint32_t inner = kFp8 ? 128 : 64;
    LayerParams up = p, down = p;
    up.tokens_x = static_cast<const uint8_t*>(x);
    down.tokens_x = up.act = workspace;
    up.w_scales = up_scales;
    down.w_scales = down_scales;
    up.partial = reinterpret_cast<float*>(workspace + ws.up_partial);
    down.partial = reinterpret_cast<float*>(workspace + ws.down_partial);
    up.tickets = h->layer_tickets;
    down.tickets = h->layer_tickets + h->plan.num_sms;
    int up_smem = 0, down_smem = 0;
    const bool small = both_on_an_sm(p, kFp8);
    ep_status st = size_kernels(&up, &down, kFp8, small, &up_smem, &down_smem);
    LayerMaps mu, md;
    if (st == EP_OK) st = encode(&mu.w, {w_up, element, 3, {H, 2 * I, E, 1}, {H * esize, H * esize * 2 * I, 0}, {inner, kTile, 1, 1}});
    if (st == EP_OK) st = encode(&md.w, {w_down, element, 3, {I, H, E, 1}, {I * esize, I * esize * H, 0}, {inner, kTile, 1, 1}});
    if (kFp8) {
        mu.x = mu.w, md.x = md.w;  // not used
    } else {
        const uint64_t act_rows = static_cast<uint64_t>(p.tokens) * (p.topk < p.experts ? p.topk : p.experts);
        if (st == EP_OK) st = encode(&mu.x, {x, Element::kBf16, 2, {H, static_cast<uint64_t>(p.tokens), 1, 1}, {2 * H, 0, 0}, {64, static_cast<uint32_t>(col_step(false)), 1, 1}});
        if (st == EP_OK) st = encode(&md.x, {workspace, Element::kBf16, 2, {I, act_rows, 1, 1}, {2 * I, 0, 0}, {64, static_cast<uint32_t>(col_step(false)), 1, 1}});
    }
    if (st != EP_OK) return st;
    cudaError_t err = small ? start<kFp8, kSmallTokens, false>(h, mu, up, up_smem, stream) : start<kFp8, kMaxTokens, false>(h, mu, up, up_smem, stream);
    if (err == cudaSuccess)
        err = small ? start<kFp8, kSmallTokens, true>(h, md, down, down_smem, stream) : start<kFp8, kMaxTokens, true>(h, md, down, down_smem, stream);
    if (err != cudaSuccess) return cuda_fail(err, "layer launch");
    return EP_OK;
}

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" {

int64_t ep_moe_layer_workspace(const ep_handle* h, int32_t num_tokens, int32_t width) {
    if (h == nullptr || num_tokens < 0 || width < 0 || static_cast<int64_t>(num_tokens) * h->cfg.num_ranks > kMaxTokens) return -1;
    return workspace_of(h, static_cast<int64_t>(num_tokens) * h->cfg.num_ranks, width).bytes;
}

ep_status ep_moe_layer(ep_handle* h, int32_t num_tokens, int32_t width, const void* x, const int64_t* topk_idx,
                       const float* topk_weights, const void* w_up, const float* w_up_scales, const void* w_down,
                       const float* w_down_scales, ep_dtype w_dtype, const void* bias_0, const void* bias_1, void* out,
                       void* workspace, int64_t workspace_bytes, ep_stream_t stream) {
    EP_TRACE();
    if (h == nullptr) return fail(EP_ERR_INVALID_ARG, "handle is NULL");
    const ep_config& c = h->cfg;
    EP_CHECK_ARG(num_tokens >= 0 && num_tokens <= c.num_max_tokens, "num_tokens %d outside [0, num_max_tokens=%d]", num_tokens, c.num_max_tokens);
    const int64_t tokens = static_cast<int64_t>(num_tokens) * c.num_ranks;
    if (tokens > kMaxTokens)
        return fail(EP_ERR_UNSUPPORTED, "%lld tokens: the layer takes at most %d in all", static_cast<long long>(tokens), kMaxTokens);
    EP_CHECK_ARG(w_dtype == EP_BF16 || w_dtype == EP_FP8_E4M3, "w_dtype must be EP_BF16 or EP_FP8_E4M3");
    EP_CHECK_ARG(width >= 8 && width % 8 == 0 && width <= (1 << 24), "width %d must be a positive multiple of 8", width);
    const bool fp8 = w_dtype == EP_FP8_E4M3;
    if (fp8 && (width % kFp8Group != 0 || c.hidden % kFp8Group != 0))
        return fail(EP_ERR_UNSUPPORTED, "FP8 weights need hidden %% 128 == 0 and width %% 128 == 0 (hidden %d, width %d)", c.hidden, width);
    EP_CHECK_ARG(fp8 ? w_up_scales && w_down_scales && aligned4(w_up_scales) && aligned4(w_down_scales) : !w_up_scales && !w_down_scales,
                 "w_up_scales and w_down_scales go with FP8 weights");
    if (tokens == 0) return EP_OK;
    EP_CHECK_ARG(x && w_up && w_down && out && aligned16(x) && aligned16(w_up) && aligned16(w_down) && aligned16(out),
                 "x, w_up, w_down and out must be 16-byte aligned device pointers");
    EP_CHECK_ARG(topk_idx && topk_weights && aligned8(topk_idx) && aligned4(topk_weights), "topk_idx or topk_weights is NULL or misaligned");
    EP_CHECK_ARG(aligned16(bias_0) && aligned16(bias_1), "bias_0 and bias_1 must be 16-byte aligned");
    const int64_t need = workspace_of(h, tokens, width).bytes;
    EP_CHECK_ARG(workspace && aligned16(workspace) && workspace_bytes >= need,
                 "the layer needs a 16-byte aligned workspace of %lld bytes (ep_moe_layer_workspace), got %lld",
                 static_cast<long long>(need), static_cast<long long>(workspace_bytes));
    LayerParams p = {};
    p.topk_idx = topk_idx;
    p.topk_weights = topk_weights;
    p.rank_mask = h->rank_mask;
    p.bias_0 = static_cast<const uint8_t*>(bias_0);
    p.bias_1 = static_cast<const uint8_t*>(bias_1);
    p.out = static_cast<uint8_t*>(out);
    p.status = h->status;
    p.wait_limit_ns = h->wait_limit_ns;
    p.tokens = static_cast<int32_t>(tokens);
    p.tokens_per_rank = num_tokens;
    p.topk = c.num_topk;
    p.experts = c.num_experts;
    p.local_experts = c.num_experts / c.num_ranks;
    p.hidden = c.hidden;
    p.width = width;
    p.ctas = h->plan.num_sms;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    return fp8 ? run<true>(h, p, x, w_up, w_up_scales, w_down, w_down_scales, ws, stream)
               : run<false>(h, p, x, w_up, nullptr, w_down, nullptr, ws, stream);
}

}  // extern "C"
