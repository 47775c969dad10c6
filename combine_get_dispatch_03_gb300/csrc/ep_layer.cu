// ep_layer.cu -- a whole mixture-of-experts layer for a few tokens, in two kernels (sm_103a).
//
//   y[t] = sum_k w[t][k] * W_down[e] * (silu(W_gate[e] x[t]) * (W_up[e] x[t])) + bias_0[t] + bias_1[t],   e = topk_idx[t][k]
//
// With up to 64 tokens the weights of the experts that they hit are all there is to read, so the weights are the rows of the
// tensor cores' products (128 at a time) and the tokens their columns (16 to 64): every byte of weights goes from memory to
// shared memory by tensor map and into tcgen05.mma once, and no product has empty rows of weights.
//   up     a tile is 128 gate rows and the 128 up rows beside them, times ALL tokens' x: no gather, the columns of tokens
//          that are not the expert's are not read back.  silu(gate) * up goes to a workspace row of (expert, token).
//   down   a tile is 128 output channels of one expert, times its rows of the workspace; a CTA adds up the weighted
//          results of the experts it works on in shared memory, [token][128 channels] in fp32.
//
// The work of a kernel is one row of units (a tile's step of 128 bytes of the contraction) that the CTAs share evenly, so
// that none waits for a last wave: 8 experts of 7168 x 2048 are 128 tiles of the first kernel on 152 SMs.  A tile that
// crosses CTAs leaves partial sums in the workspace; the last CTA to arrive (a ticket) adds them up in the CTAs' order.
//
// The second kernel is launched beside the first (programmatic dependent launch; for up to 16 tokens both fit an SM) and
// fills its shared memory with weights, which do not hang on the first kernel, before it waits for it.
//
// FP8 weights: e4m3 with one scale per 128 x 128.  The tokens stay bf16: a block of 128 channels is scaled by a power of two
// and split into two e4m3 values (split_e4m3()) whose products share an accumulator, so that nothing of bf16's eight bits is lost but
// what lies 2^-17 below the block's largest value.  A block's sums are scaled and added up in fp32 registers.
#include "ep_act.cuh"
#include "ep_groups.cuh"
#include "ep_handle.h"
#include "ep_maps.h"
#include "ep_tc.cuh"
#include "ep_trace.h"

namespace ep {
namespace {

constexpr int kMaxTokens = 64;
constexpr int kTile = 128;                  // rows of weights
constexpr uint32_t kRow = 128;              // bytes of the contraction in a stage
constexpr uint32_t kTileBytes = kTile * kRow;
constexpr int kColStep = 16;                // tokens (columns of products) come in steps of this
constexpr int kMaxStages = 8;
constexpr int kSumWarps = 8;                // warps 4 to 11: accumulators to sums and out
constexpr int kSplitWarps = 4;              // warps 12 to 15, FP8: x in two e4m3 parts
constexpr int kScaleRing = 16;              // blocks whose token scales are kept: more than stages and accumulators
constexpr int kBuffers = 2;                 // accumulators
constexpr int kSmallTokens = 16;            // up to which both kernels fit an SM
static_assert(kScaleRing > kMaxStages + kBuffers + 1, "a block's scales outlive it");
constexpr int layer_threads(bool fp8) { return (4 + kSumWarps + (fp8 ? kSplitWarps : 0)) * kWarpSize; }

struct LayerParams {
    const int64_t* topk_idx;
    const float* topk_weights;
    const int32_t* rank_mask;
    const uint8_t* tokens_x;   // up: x rows; down: the workspace's rows (bf16)
    const float* w_scales;     // FP8
    uint8_t* act;              // [rows][width] bf16
    float* partial;            // of this kernel: up [CTA][2][token][gate, up][128], down [CTA][2][token][128]
    int32_t* tickets;          // [CTAs], 0
    const uint8_t* bias_0;
    const uint8_t* bias_1;
    uint8_t* out;
    int32_t* status;
    uint64_t wait_limit_ns;
    int32_t tokens, tokens_per_rank, topk, experts, local_experts, hidden, width;
    int32_t cols;              // tokens, rounded up to kColStep
    int32_t stages;
    uint32_t stage_bytes, tmem_columns;
};

struct LayerMaps {
    CUtensorMap w, x;
};

struct LayerControl {
    uint64_t full[kMaxStages];
    uint64_t empty[kMaxStages];
    uint64_t acc_full[kBuffers];
    uint64_t acc_empty[kBuffers];
    uint64_t drained;
    uint32_t tmem;
    int32_t abort_flag;
    int32_t last_arrival;
    int32_t hits;
    int64_t sums[16];
};

// Which experts the tokens hit, in shared memory.
struct Routing {
    uint64_t* tokens;   // [experts] bit t: token t
    int32_t* begin;     // [experts] first workspace row of a hit expert
    uint16_t* hit;      // hit experts in ascending order
    float* weight;      // down: [rows] the weight of a row's (expert, token)
};

__device__ __forceinline__ int count_bits(uint64_t m) { return __popcll(static_cast<long long>(m)); }
__device__ __forceinline__ int lowest_bit(uint64_t m) { return __ffsll(static_cast<long long>(m)) - 1; }

// The expert of slot (token, k), -1 for none: as in the low-latency dispatch, a masked rank neither sends nor receives.
__device__ __forceinline__ int slot_expert(const LayerParams& p, int slot) {
    const int64_t e = p.topk_idx[slot];
    if (e < 0 || e >= p.experts) return -1;
    if (p.rank_mask[slot / p.topk / p.tokens_per_rank] || p.rank_mask[static_cast<int>(e) / p.local_experts]) return -1;
    return static_cast<int>(e);
}

template <int THREADS, bool kWeights>
__device__ __forceinline__ void build_routing(const Routing& t, const LayerParams& p, LayerControl& ctl) {
    for (int e = threadIdx.x; e < p.experts; e += THREADS) t.tokens[e] = 0;
    __syncthreads();
    const int slots = p.tokens * p.topk;
    for (int s = threadIdx.x; s < slots; s += THREADS) {
        const int64_t raw = p.topk_idx[s];
        if (raw < -1 || raw >= p.experts) report(p.status, EP_ERR_BAD_EXPERT);
        const int e = slot_expert(p, s);
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
    if constexpr (kWeights) {
        // an expert that a token names twice counts with both weights
        for (int s = threadIdx.x; s < slots; s += THREADS) {
            const int e = slot_expert(p, s);
            if (e < 0) continue;
            const int token = s / p.topk;
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

// A unit: a tile and a step of its contraction.
struct Unit {
    int expert, col, step;  // col: first gate row (up) or output channel (down) of the tile
    uint64_t tokens;
};

template <bool kDown>
struct Work {
    const Routing& t;
    Shares shares;
    int64_t first, last;
    int hits, across, steps;

    __device__ __forceinline__ Unit at(int64_t unit) const {
        const int tile = static_cast<int>(unit / steps);
        Unit u;
        u.step = static_cast<int>(unit - static_cast<int64_t>(tile) * steps);
        const int i = kDown ? tile % hits : tile / across;
        u.expert = t.hit[i];
        u.col = (kDown ? tile / hits : tile % across) * kTile;
        u.tokens = t.tokens[u.expert];
        return u;
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
    float* scales;   // FP8: [kScaleRing][kMaxTokens] of the tokens' blocks
    float* sums;     // down: [tokens][128]
};

constexpr uint32_t a_bytes(bool down) { return down ? kTileBytes : 2 * kTileBytes; }

__device__ __forceinline__ int round_cols(int n) { return (n + kColStep - 1) / kColStep * kColStep; }

// Weights of a unit into its stage.
template <bool kFp8, bool kDown>
__device__ __forceinline__ void load_weights(const LayerRoles<kDown>& x, const Unit& u, int stage) {
    const int k0 = u.step * (kFp8 ? 128 : 64);
    uint8_t* a = x.stages + stage * x.p.stage_bytes;
    const uint32_t bar = smem_u32(&x.ctl.full[stage]);
    tma_load_3d<1>(a, &x.maps.w, k0, u.col, u.expert, bar);
    if (!kDown) tma_load_3d<1>(a + kTileBytes, &x.maps.w, k0, x.p.width + u.col, u.expert, bar);
}

// Bytes and copies of a unit's tokens, bf16.
template <bool kDown>
__device__ __forceinline__ uint32_t token_bytes(const LayerParams& p, const Unit& u) {
    return (kDown ? round_cols(count_bits(u.tokens)) : p.cols) * kRow;
}

template <bool kDown>
__device__ __forceinline__ void load_tokens(const LayerRoles<kDown>& x, const Unit& u, int stage) {
    uint8_t* b = x.stages + stage * x.p.stage_bytes + a_bytes(kDown);
    const uint32_t bar = smem_u32(&x.ctl.full[stage]);
    const int first = kDown ? x.t.begin[u.expert] : 0;
    const int cols = kDown ? round_cols(count_bits(u.tokens)) : x.p.cols;
    for (int c = 0; c < cols; c += kColStep) tma_load_2d<1>(b + c * kRow, &x.maps.x, u.step * 64, first + c, bar);
}

// One thread: the loads.
template <bool kFp8, bool kDown>
__device__ __forceinline__ void layer_loads(const LayerRoles<kDown>& x) {
    const LayerParams& p = x.p;
    LayerControl& ctl = x.ctl;
    const Work<kDown>& w = x.work;
    int64_t unit = w.first;
    bool ok = true;
    int stage = 0, used = 0;
    uint32_t phase = 0;
    if constexpr (kDown) {
        // Weights for every stage, then the first kernel's results.
        const int ahead = static_cast<int>(min(static_cast<int64_t>(p.stages), w.last - w.first));
        for (int i = 0; i < ahead; ++i) {
            const Unit u = w.at(unit + i);
            bar_arrive_expect_tx<1>(smem_u32(&ctl.full[i]), a_bytes(kDown) + (kFp8 ? 0 : token_bytes<kDown>(p, u)));
            load_weights<kFp8, kDown>(x, u, i);
        }
        asm volatile("griddepcontrol.wait;" ::: "memory");
        if constexpr (!kFp8)
            for (int i = 0; i < ahead; ++i) load_tokens<kDown>(x, w.at(unit + i), i);
        unit += ahead;
        used = ahead;
        if (ahead == p.stages) phase = 1;
        else stage = ahead;
    }
    for (; unit < w.last; ++unit) {
        ok = wait_phase(&ctl.empty[stage], phase ^ 1, x.waits);
        if (!ok) break;
        const Unit u = w.at(unit);
        bar_arrive_expect_tx<1>(smem_u32(&ctl.full[stage]), a_bytes(kDown) + (kFp8 ? 0 : token_bytes<kDown>(p, u)));
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
template <bool kFp8, bool kDown>
__device__ __forceinline__ void layer_products(const LayerRoles<kDown>& x) {
    const LayerParams& p = x.p;
    LayerControl& ctl = x.ctl;
    const Work<kDown>& w = x.work;
    int stage = 0, buf = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool first = true;  // of an accumulator
    for (int64_t unit = w.first; unit < w.last; ++unit) {
        const Unit u = w.at(unit);
        if (!wait_phase(&ctl.full[stage], phase, x.waits)) break;
        if (first && !wait_phase(&ctl.acc_empty[buf], acc_phase ^ 1, x.waits)) break;
        tc_fence_after();
        const uint32_t cols = kDown ? round_cols(count_bits(u.tokens)) : p.cols;
        const uint32_t idesc = mma_desc(kFp8 ? 0 : 1, false, false, kTile, cols);
        const uint32_t a = smem_u32(x.stages) + stage * p.stage_bytes;
        const uint32_t d = ctl.tmem + buf * (kDown ? 1 : 2) * p.cols;
#pragma unroll
        for (int part = 0; part < (kFp8 ? 2 : 1); ++part) {
            const uint64_t db = smem_desc(a + a_bytes(kDown) + part * p.cols * kRow, 16);
#pragma unroll
            for (int op = 0; op < (kDown ? 1 : 2); ++op) {
                const uint64_t da = smem_desc(a + op * kTileBytes, 16);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    tc_mma<1, kFp8>(d + op * p.cols, da + i * 2, db + i * 2, idesc, !first || part || i);
            }
        }
        tc_commit<1>(&ctl.empty[stage]);
        first = false;
        if (kFp8 || u.step == w.steps - 1 || unit == w.last - 1) {
            // this thread's own arrival passes on what it acquired with the stage: the tokens' scales
            bar_arrive<1>(smem_u32(&ctl.acc_full[buf]));
            tc_commit<1>(&ctl.acc_full[buf]);
            if (++buf == kBuffers) buf = 0, acc_phase ^= 1;
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
        const float a = f[2 * i] * mult, b = f[2 * i + 1] * mult;
        const __nv_fp8x2_storage_t code = e4m3x2(a, b);
        const float2 back = __half22float2(static_cast<__half2>(__nv_cvt_fp8x2_to_halfraw2(code, __NV_E4M3)));
        h[i / 2] |= static_cast<uint32_t>(code) << (i % 2 * 16);
        l[i / 2] |= static_cast<uint32_t>(e4m3x2(a - back.x, b - back.y)) << (i % 2 * 16);
    }
    *high = make_uint2(h[0], h[1]);
    *low = make_uint2(l[0], l[1]);
}

// Four warps, FP8: the tokens' blocks of a unit, split, into the place and order in which a tensor-map load would put
// them.  Sixteen lanes have a token's 128 channels; the next unit's values are on their way meanwhile.
template <int kTokens, bool kDown>
__device__ __forceinline__ void layer_splits(const LayerRoles<kDown>& x, int warp) {
    constexpr int kPer = kTokens / (2 * kSplitWarps);  // tokens of half a warp
    const LayerParams& p = x.p;
    LayerControl& ctl = x.ctl;
    const Work<kDown>& w = x.work;
    const int64_t row_bytes = 2 * static_cast<int64_t>(kDown ? p.width : p.hidden);
    const int first_token = warp * 2 + (lane_id() >> 4), piece = lane_id() & 15;
    int4 next[kPer];
    auto fetch = [&](int64_t unit) {
        const Unit u = w.at(unit);
        const int count = kDown ? count_bits(u.tokens) : p.tokens;
        const int64_t row0 = kDown ? x.t.begin[u.expert] : 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int t = first_token + i * 2 * kSplitWarps;
            next[i] = make_int4(0, 0, 0, 0);
            if (t < count) next[i] = __ldcg(reinterpret_cast<const int4*>(p.tokens_x + (row0 + t) * row_bytes + u.step * 256) + piece);
        }
    };
    if (kDown) asm volatile("griddepcontrol.wait;" ::: "memory");
    int stage = 0;
    uint32_t phase = 0;
    if (w.first < w.last) fetch(w.first);
    for (int64_t unit = w.first; unit < w.last; ++unit) {
        const int count = kDown ? count_bits(w.at(unit).tokens) : p.tokens;
        if (!warp_wait(&ctl.empty[stage], phase ^ 1, x.waits)) break;
        uint8_t* b = x.stages + stage * p.stage_bytes + a_bytes(kDown);
        float* scales = x.scales + static_cast<int>((unit - w.first) % kScaleRing) * kMaxTokens;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int t = first_token + i * 2 * kSplitWarps;
            if (t - (lane_id() >> 4) >= count) break;  // the whole warp
            float f[8];
            unpack8(next[i], f);
            float most = absmax8(f);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(kFullMask, most, o));
            // 2^(7 - exponent), at most 2^126; an infinite value has no scale and makes the token's sums NaN, as NaN does
            const int exponent = static_cast<int>(__float_as_uint(most) >> 23);
            const int up = min(134 - exponent, 126);
            const float mult = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
            uint2 high, low;
            split_e4m3(f, mult, &high, &low);
            if (t < count) {
                const uint32_t at = t * kRow + (((piece >> 1) ^ (t & 7)) << 4) + (piece & 1) * 8;
                *reinterpret_cast<uint2*>(b + at) = high;
                *reinterpret_cast<uint2*>(b + p.cols * kRow + at) = low;
                if (piece == 0) scales[t] = exponent == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
            }
        }
        fence_async_smem();
        __syncwarp();
        if (lane_id() == 0) bar_arrive<1>(smem_u32(&ctl.full[stage]));
        if (unit + 1 < w.last) fetch(unit + 1);
        if (++stage == p.stages) stage = 0, phase ^= 1;
    }
}

// One fp32 column of this warp's 32 lanes of tensor memory: starts the load.
__device__ __forceinline__ void tc_ld1(uint32_t addr, uint32_t& v) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(v) : "r"(addr));
}

template <int N>
__device__ __forceinline__ void tc_wait_columns(uint32_t (&v)[N]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(v[i]));  // no use before the wait
}

__device__ __forceinline__ void sum_warps_barrier() { asm volatile("bar.sync 1, %0;" ::"n"(kSumWarps * kWarpSize) : "memory"); }

// After the sum warps wrote a part of what `parts` CTAs add up: whether this CTA is the last to arrive, and may read all.
template <bool kDown>
__device__ __forceinline__ bool last_to_arrive(const LayerRoles<kDown>& x, int ticket, int parts) {
    __threadfence();
    sum_warps_barrier();
    if (threadIdx.x == 4 * kWarpSize) {
        const bool last = atomicAdd(x.p.tickets + ticket, 1) == parts - 1;
        if (last) x.p.tickets[ticket] = 0;  // for the next call
        x.ctl.last_arrival = last;
        __threadfence();
    }
    sum_warps_barrier();
    const bool last = *const_cast<volatile int32_t*>(&x.ctl.last_arrival) != 0;
    sum_warps_barrier();  // read before the next one is written
    return last;
}

// The sums of a run of one tile's units that this CTA has, OPS values for each of a warp's tokens.  column(q): the
// accumulator's column of its q-th token.
template <bool kFp8, int OPS, int PER, bool kDown, typename Column>
__device__ __forceinline__ void read_sums(const LayerRoles<kDown>& x, int64_t unit, int steps, int mine, uint32_t lanes, const Unit& u,
                                          int& buf, uint32_t& acc_phase, bool& ok, Column column, float (&v)[OPS][PER]) {
    const LayerParams& p = x.p;
    LayerControl& ctl = x.ctl;
    constexpr int kBatch = 4;
#pragma unroll
    for (int o = 0; o < OPS; ++o)
#pragma unroll
        for (int q = 0; q < PER; ++q) v[o][q] = 0.0f;
    const float* ws[OPS];
    float w_next[OPS];
    if constexpr (kFp8) {
#pragma unroll
        for (int o = 0; o < OPS; ++o) {
            const int rows = (kDown ? p.hidden : 2 * p.width) / kFp8Group;
            const int row = u.col / kFp8Group + o * (p.width / kFp8Group);
            ws[o] = p.w_scales + (static_cast<int64_t>(u.expert) * rows + row) * x.work.steps + u.step;
            w_next[o] = __ldg(ws[o]);
        }
    }
    for (int s = 0; s < (kFp8 ? steps : 1); ++s) {
        float ww[OPS];
        if constexpr (kFp8) {
#pragma unroll
            for (int o = 0; o < OPS; ++o) {
                ww[o] = w_next[o];
                w_next[o] = __ldg(ws[o] + min(s + 1, steps - 1));
            }
        }
        if (ok) ok = warp_wait(&ctl.acc_full[buf], acc_phase, x.waits);
        if (!ok) return;
        tc_fence_after();
        const uint32_t from = ctl.tmem + lanes + buf * OPS * p.cols;
        const float* scales = x.scales + static_cast<int>((unit + s - x.work.first) % kScaleRing) * kMaxTokens;
#pragma unroll
        for (int q0 = 0; q0 < PER; q0 += kBatch) {
            if (q0 >= mine) break;
            uint32_t r[OPS * kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
#pragma unroll
                for (int o = 0; o < OPS; ++o) {
                    r[o * kBatch + i] = 0;
                    if (q0 + i < mine) tc_ld1(from + o * p.cols + column(q0 + i), r[o * kBatch + i]);
                }
            }
            tc_wait_columns(r);
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
#pragma unroll
                for (int o = 0; o < OPS; ++o) {
                    const float d = __uint_as_float(r[o * kBatch + i]);
                    if constexpr (!kFp8) v[o][q0 + i] = d;
                    else if (q0 + i < mine) v[o][q0 + i] = fmaf(d, ww[o] * scales[column(q0 + i)], v[o][q0 + i]);
                }
        }
        tc_fence_before();
        __syncwarp();
        if (lane_id() == 0) bar_arrive<1>(smem_u32(&ctl.acc_empty[buf]));
        if (++buf == kBuffers) buf = 0, acc_phase ^= 1;
    }
}

// Eight warps of the first kernel: accumulators to silu(gate) * up.  A warp has 32 rows of the tile and every second
// token of the expert.
template <bool kFp8, int kTokens>
__device__ __forceinline__ void up_sums(const LayerRoles<false>& x, int warp) {
    constexpr int kPer = kTokens / 2;
    const LayerParams& p = x.p;
    const Work<false>& w = x.work;
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const int row = quarter * 32 + lane_id();
    int buf = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (int64_t unit = w.first; unit < w.last;) {
        const Unit u = w.at(unit);
        const int steps = static_cast<int>(min(static_cast<int64_t>(w.steps - u.step), w.last - unit));
        const int count = count_bits(u.tokens);
        const int mine = (count + 1 - half) / 2;
        float v[2][kPer];
        // the columns of this warp's tokens, six bits each in order of q
        uint8_t tokens[kPer];
        {
            uint64_t m = half ? u.tokens & (u.tokens - 1) : u.tokens;
#pragma unroll
            for (int q = 0; q < kPer; ++q) {
                tokens[q] = static_cast<uint8_t>(m ? lowest_bit(m) : 0);
                m &= m - 1;
                m &= m - 1;
            }
        }
        read_sums<kFp8, 2, kPer, false>(x, unit, steps, mine, static_cast<uint32_t>(quarter * 32) << 16, u, buf, acc_phase, ok,
                                        [&](int q) { return static_cast<int>(tokens[q]); }, v);
        bool finish = true;
        if (steps < w.steps) {
            const int64_t tile0 = unit - u.step;
            const int a = w.shares.owner(tile0), b = w.shares.owner(tile0 + w.steps - 1);
            const int64_t each = static_cast<int64_t>(p.tokens) * 2 * kTile;
            float* own = p.partial + (2 * static_cast<int64_t>(blockIdx.x) + (u.step == 0)) * each + row;
#pragma unroll
            for (int q = 0; q < kPer; ++q) {
                if (q >= mine) break;
                own[(half + 2 * q) * 2 * kTile] = v[0][q];
                own[(half + 2 * q) * 2 * kTile + kTile] = v[1][q];
            }
            finish = last_to_arrive(x, a, b - a + 1);
            if (finish) {
#pragma unroll
                for (int q = 0; q < kPer; ++q) v[0][q] = v[1][q] = 0.0f;
                for (int c = a; c <= b; ++c) {
                    const float* part = p.partial + (2 * static_cast<int64_t>(c) + (c == a)) * each + row;
#pragma unroll
                    for (int q = 0; q < kPer; ++q) {
                        if (q >= mine) break;
                        v[0][q] += __ldcg(part + (half + 2 * q) * 2 * kTile);
                        v[1][q] += __ldcg(part + (half + 2 * q) * 2 * kTile + kTile);
                    }
                }
            }
        }
        if (finish && u.col + row < p.width) {
            const int64_t first = x.t.begin[u.expert];
#pragma unroll
            for (int q = 0; q < kPer; ++q) {
                if (q >= mine) break;
                const float a = activate(EP_ACT_SILU, v[0][q]) * v[1][q];
                // bf16, as the second product's operand is
                *reinterpret_cast<__nv_bfloat16*>(p.act + 2 * ((first + half + 2 * q) * p.width + u.col + row)) = __float2bfloat16_rn(a);
            }
        }
        unit += steps;
    }
}

// Output channel `row` of a tile for the tokens of one parity, from the sums.
__device__ __forceinline__ void put_output(const LayerParams& p, int token, int channel, float sum) {
    const int64_t at = 2 * (static_cast<int64_t>(token) * p.hidden + channel);
    if (p.bias_0) sum += __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(p.bias_0 + at));
    if (p.bias_1) sum += __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(p.bias_1 + at));
    *reinterpret_cast<__nv_bfloat16*>(p.out + at) = __float2bfloat16_rn(sum);
}

// Eight warps of the second kernel: accumulators to the tokens' weighted sums.  A warp has 32 channels of the tile and the
// tokens of one parity, so that a sum belongs to one thread whatever the expert.
template <bool kFp8, int kTokens>
__device__ __forceinline__ void down_sums(const LayerRoles<true>& x, int warp) {
    constexpr int kPer = kTokens / 2;
    const LayerParams& p = x.p;
    const Work<true>& w = x.work;
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const int row = quarter * 32 + lane_id();
    if (w.hits == 0) {  // no token has an expert
        for (int j = blockIdx.x; j < w.across; j += gridDim.x)
            for (int t = half; t < p.tokens; t += 2)
                if (j * kTile + row < p.hidden) put_output(p, t, j * kTile + row, 0.0f);
        return;
    }
    float* const sums = x.sums + row;
    for (int t = half; t < p.tokens; t += 2) sums[t * kTile] = 0.0f;
    const int64_t each_tile = static_cast<int64_t>(w.hits) * w.steps;  // units of 128 channels
    int buf = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (int64_t unit = w.first; unit < w.last;) {
        const Unit u = w.at(unit);
        const int steps = static_cast<int>(min(static_cast<int64_t>(w.steps - u.step), w.last - unit));
        const uint64_t parity = u.tokens & (half ? 0xaaaaaaaaaaaaaaaaull : 0x5555555555555555ull);
        const int mine = count_bits(parity);
        uint8_t tokens[kPer], cols[kPer];
        {
            uint64_t m = parity;
#pragma unroll
            for (int q = 0; q < kPer; ++q) {
                const int t = m ? lowest_bit(m) : 0;
                tokens[q] = static_cast<uint8_t>(t);
                cols[q] = static_cast<uint8_t>(count_bits(u.tokens & ((1ull << t) - 1)));
                m &= m - 1;
            }
        }
        float v[1][kPer];
        read_sums<kFp8, 1, kPer, true>(x, unit, steps, mine, static_cast<uint32_t>(quarter * 32) << 16, u, buf, acc_phase, ok,
                                       [&](int q) { return static_cast<int>(cols[q]); }, v);
        const float* weight = x.t.weight + x.t.begin[u.expert];
#pragma unroll
        for (int q = 0; q < kPer; ++q) {
            if (q >= mine) break;
            sums[tokens[q] * kTile] += weight[cols[q]] * v[0][q];
        }
        unit += steps;
        const int64_t tile0 = (unit - 1) / each_tile * each_tile;
        if (unit < w.last && unit < tile0 + each_tile) continue;  // more of these channels
        bool finish = true, summed = false;
        const bool whole = tile0 >= w.first && unit == tile0 + each_tile;
        int a = 0, b = 0;
        const int64_t each = static_cast<int64_t>(p.tokens) * kTile;
        if (!whole) {
            a = w.shares.owner(tile0), b = w.shares.owner(tile0 + each_tile - 1);
            float* own = p.partial + (2 * static_cast<int64_t>(blockIdx.x) + (tile0 >= w.first)) * each + row;
            for (int t = half; t < p.tokens; t += 2) own[t * kTile] = sums[t * kTile];
            finish = last_to_arrive(x, a, b - a + 1);
            summed = finish;
        }
        if (finish && u.col + row < p.hidden) {
            for (int t = half; t < p.tokens; t += 2) {
                float s = summed ? 0.0f : sums[t * kTile];
                if (summed) {
#pragma unroll 4
                    for (int c = a; c <= b; ++c) s += __ldcg(p.partial + (2 * static_cast<int64_t>(c) + (c == a)) * each + row + t * kTile);
                }
                put_output(p, t, u.col + row, s);
            }
        }
        for (int t = half; t < p.tokens; t += 2) sums[t * kTile] = 0.0f;
    }
}

// The dynamic shared memory of a kernel, after alignment to 1024: stages, then the rest.
struct Layout {
    uint32_t tokens, begin, hit, weight, scales, sums, bytes;
};

__host__ __device__ inline Layout layer_layout(const LayerParams& p, bool fp8, bool down) {
    Layout l;
    uint32_t at = p.stages * p.stage_bytes;
    l.tokens = at, at += 8u * p.experts;
    l.begin = at, at += 4u * p.experts;
    l.sums = at, at += down ? 4u * p.tokens * kTile : 0u;
    l.weight = at, at += down ? 4u * p.tokens * p.topk : 0u;
    l.scales = at, at += fp8 ? 4u * kScaleRing * kMaxTokens : 0u;
    const int most = p.tokens * p.topk < p.experts ? p.tokens * p.topk : p.experts;
    l.hit = at, at += 2u * most;
    l.bytes = at;
    return l;
}

template <bool kFp8, int kTokens, bool kDown>
__global__ void __launch_bounds__(layer_threads(kFp8), kTokens <= kSmallTokens ? 2 : 1)
    layer_kernel(const __grid_constant__ LayerMaps maps, const LayerParams p) {
    constexpr int kThreads = layer_threads(kFp8);
    extern __shared__ uint8_t raw[];
    __shared__ LayerControl ctl;
    uint8_t* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    const Layout l = layer_layout(p, kFp8, kDown);
    const Routing t = {reinterpret_cast<uint64_t*>(smem + l.tokens), reinterpret_cast<int32_t*>(smem + l.begin),
                       reinterpret_cast<uint16_t*>(smem + l.hit), reinterpret_cast<float*>(smem + l.weight)};
    const int warp = threadIdx.x / kWarpSize;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(&ctl.full[i], kFp8 ? 1 + kSplitWarps : 1);
            mbar_init(&ctl.empty[i], 1);
        }
        for (int i = 0; i < kBuffers; ++i) {
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
    build_routing<kThreads, kDown>(t, p, ctl);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();

    const int steps = ((kDown ? p.width : p.hidden) * (kFp8 ? 1 : 2) + static_cast<int>(kRow) - 1) / static_cast<int>(kRow);
    const int across = ((kDown ? p.hidden : p.width) + kTile - 1) / kTile;
    const int64_t units = static_cast<int64_t>(ctl.hits) * across * steps;
    const Shares shares = {units, static_cast<int>(min(units, static_cast<int64_t>(gridDim.x)))};
    const bool works = static_cast<int>(blockIdx.x) < shares.ctas;
    const Work<kDown> work = {t, shares, works ? shares.begin(blockIdx.x) : 0, works ? shares.begin(blockIdx.x + 1) : 0,
                              ctl.hits, across, steps};
    const LayerRoles<kDown> x = {maps, p, t, work, ctl, {&ctl.abort_flag, p.status, p.wait_limit_ns}, smem,
                                 reinterpret_cast<float*>(smem + l.scales), reinterpret_cast<float*>(smem + l.sums)};
    if (warp == 0) {
        if (elect_one()) layer_loads<kFp8, kDown>(x);
    } else if (warp == 1) {
        if (elect_one()) layer_products<kFp8, kDown>(x);
    } else if (warp >= 4 && warp < 4 + kSumWarps) {
        if constexpr (kDown) down_sums<kFp8, kTokens>(x, warp);
        else up_sums<kFp8, kTokens>(x, warp);
    } else if (kFp8 && warp >= 4 + kSumWarps) {
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

constexpr int64_t kSmallSmem[2] = {119 * 1024, 104 * 1024};  // up, down: together on an SM
constexpr int64_t kLargeSmem = 224 * 1024;

int64_t align256(int64_t v) { return (v + 255) / 256 * 256; }

struct Workspace {
    int64_t up_partial, down_partial, bytes;  // the activations come first
};

Workspace workspace_of(const ep_handle* h, int64_t tokens, int32_t width) {
    const int64_t rows = tokens * (h->cfg.num_topk < h->cfg.num_experts ? h->cfg.num_topk : h->cfg.num_experts);
    const int64_t ctas = h->plan.num_sms;
    Workspace w;
    w.up_partial = align256(rows * width * 2);
    w.down_partial = w.up_partial + align256(ctas * 2 * tokens * 2 * kTile * 4);
    w.bytes = w.down_partial + align256(ctas * 2 * tokens * kTile * 4);
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
    constexpr int kSmem = 226 * 1024;
    cudaError_t err = plan_kernels<false, kSmallTokens>(kSmem);
    if (err == cudaSuccess) err = plan_kernels<false, kMaxTokens>(kSmem);
    if (err == cudaSuccess) err = plan_kernels<true, kSmallTokens>(kSmem);
    if (err == cudaSuccess) err = plan_kernels<true, kMaxTokens>(kSmem);
    return err;
}

// Stages and tensor memory of a kernel.
ep_status size_kernel(LayerParams* p, bool fp8, bool down, uint32_t* smem) {
    p->cols = (p->tokens + kColStep - 1) / kColStep * kColStep;
    p->stage_bytes = (down ? kTileBytes : 2 * kTileBytes) + (fp8 ? 2 : 1) * p->cols * kRow;
    p->tmem_columns = 32;
    while (p->tmem_columns < static_cast<uint32_t>(kBuffers * (down ? 1 : 2) * p->cols)) p->tmem_columns *= 2;
    const int64_t room = p->tokens <= kSmallTokens ? kSmallSmem[down] : kLargeSmem;
    p->stages = 0;
    const int64_t rest = layer_layout(*p, fp8, down).bytes + 1024;
    // with very many experts the table takes more: then the kernels no longer fit an SM together
    int64_t stages = (room - rest) / p->stage_bytes;
    if (stages < 2) stages = 2;
    p->stages = static_cast<int32_t>(stages < kMaxStages ? stages : kMaxStages);
    *smem = layer_layout(*p, fp8, down).bytes + 1024;
    if (*smem > 226 * 1024) return fail(EP_ERR_UNSUPPORTED, "the layer's tables need too much shared memory");
    return EP_OK;
}

template <bool kFp8, int kTokens, bool kDown>
cudaError_t start(const ep_handle* h, const LayerMaps& m, const LayerParams& p, uint32_t smem, cudaStream_t stream) {
    return launch_kernel(layer_kernel<kFp8, kTokens, kDown>, dim3(h->plan.num_sms), dim3(layer_threads(kFp8)), smem, stream, 1, m, p);
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
    uint32_t up_smem = 0, down_smem = 0;
    ep_status st = size_kernel(&up, kFp8, false, &up_smem);
    if (st == EP_OK) st = size_kernel(&down, kFp8, true, &down_smem);
    LayerMaps mu, md;
    if (st == EP_OK) st = encode(&mu.w, {w_up, element, 3, {H, 2 * I, E, 1}, {H * esize, H * esize * 2 * I, 0}, {inner, kTile, 1, 1}});
    if (st == EP_OK) st = encode(&md.w, {w_down, element, 3, {I, H, E, 1}, {I * esize, I * esize * H, 0}, {inner, kTile, 1, 1}});
    if (kFp8) {
        mu.x = mu.w, md.x = md.w;  // not used
    } else {
        const uint64_t act_rows = static_cast<uint64_t>(p.tokens) * (p.topk < p.experts ? p.topk : p.experts);
        if (st == EP_OK) st = encode(&mu.x, {x, Element::kBf16, 2, {H, static_cast<uint64_t>(p.tokens), 1, 1}, {2 * H, 0, 0}, {64, kColStep, 1, 1}});
        if (st == EP_OK) st = encode(&md.x, {workspace, Element::kBf16, 2, {I, act_rows, 1, 1}, {2 * I, 0, 0}, {64, kColStep, 1, 1}});
    }
    if (st != EP_OK) return st;
    const bool small = p.tokens <= kSmallTokens;
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
    EP_CHECK_ARG((reinterpret_cast<uintptr_t>(bias_0) & 1u) == 0 && (reinterpret_cast<uintptr_t>(bias_1) & 1u) == 0, "misaligned bias");
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
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    return fp8 ? run<true>(h, p, x, w_up, w_up_scales, w_down, w_down_scales, ws, stream)
               : run<false>(h, p, x, w_up, nullptr, w_down, nullptr, ws, stream);
}

}  // extern "C"
