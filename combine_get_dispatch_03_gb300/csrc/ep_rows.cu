// ep_rows.cu -- a normal dispatch's rows in expert order, and the sum back (sm_103a).
//
// A normal dispatch delivers every token once per rank, [R][cap] rows in (source, token) order, with
// the local experts that want it in recv_topk_idx [R][cap][K].  A grouped product wants one row per (row, slot), all
// rows of an expert together.  The order is stable: rank, local expert, receive row, top-k slot.
//   layout   slot_row[r][row][k] = the expert-order row of that slot (or -1); counts and begins of the experts
//   gather   out[slot_row[r][row][k]] = x[r][row]            copies
//   reduce   out[r][row] = sum over k of y[slot_row[r][row][k]]    fp32, in slot order
// The gather's gradient is the reduce and the other way round.
//
// The layout is a stable counting sort of cap * K slots per rank in chunks of 2048: count, with the scan over a
// rank's chunks done by its last CTA, then place.  The data kernels move each row once: the gather reads a
// received row into shared memory with one bulk copy and writes it with one bulk copy per slot, so that it reads
// every row once however many experts want it; the reduce holds a row's columns in registers.
//
// Measured on a GB300 (6787 GB/s copied): 89 thousand received rows of 14336 bytes into 131072 expert rows, layout
// 13 us in a CUDA graph and 22 in calls, gather 454 to 459 us, 6.9 TB/s; of 7392 bytes (FP8 with scales) 521 us, 3.1 TB/s, the
// scales' small stores before each row's; the reduce of as many bf16 rows 541 us, 5.8 TB/s, and of 16288 rows of 4096
// bytes into 13.5 thousand 22 to 28 us, 4.4 to 5.6 TB/s (a row or two a warp: latency).
#include "ep_groups.cuh"
#include "ep_handle.h"
#include "ep_trace.h"

namespace ep {
namespace {

constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / kWarpSize;
constexpr int kWarpSlots = kLayoutChunk / kRowWarps;
constexpr int kGatherPiece = 16384;    // bytes of a row that one stage holds at most
constexpr int kGatherSmem = 65536;     // stages of one CTA: three CTAs per SM
constexpr int kGatherPerSm = 3;
// CTAs per resident CTA.  131072 rows of 14336 bytes: 530 us in one wave, 499 in 4, 473 in 16 (layout included); a CTA
// that starts when another ends keeps the copies spread over the GPU.  More than 16 only add empty CTAs.
constexpr int kGatherWaves = 16;
constexpr int kGatherMaxStages = 16;

// Slots of rank r that the dispatch filled.
__device__ __forceinline__ int filled_slots(const int32_t* num_recv, int r, int cap, int K) {
    return max(0, min(num_recv[r], cap)) * K;
}

// Local expert of a slot, -1 for none; one out of range sets EP_ERR_BAD_EXPERT and counts as none.
__device__ __forceinline__ int expert_of(const int64_t* idx, int64_t at, int EL, int32_t* status) {
    const int64_t e = idx[at];
    if (e < -1 || e >= EL) {
        report(status, EP_ERR_BAD_EXPERT);
        return -1;
    }
    return static_cast<int>(e);
}

// counts[r][chunk][j] = slots of the chunk that chose local expert j; the CTA of a rank that counts last turns the
// rank's counts into the rows before each chunk, a warp per expert, and writes group_count.  tickets [ranks] is zero
// before and after (a launch for the scan alone took 5 us of the layout's 27).
__global__ void __launch_bounds__(kRowThreads)
    layout_count_kernel(const int64_t* idx, const int32_t* num_recv, int cap, int K, int EL, int32_t* counts,
                        uint32_t* tickets, int32_t* group_count, int32_t* status) {
    extern __shared__ int32_t hist[];
    __shared__ bool last_of_rank;
    pdl_enter();
    const int r = blockIdx.y, chunk = blockIdx.x, chunks = gridDim.x;
    const int n = filled_slots(num_recv, r, cap, K);
    const int used = (n + kLayoutChunk - 1) / kLayoutChunk;
    if (chunk >= max(used, 1)) return;  // an empty rank's first CTA still writes its counts of 0
    for (int j = threadIdx.x; j < EL; j += kRowThreads) hist[j] = 0;
    __syncthreads();
    const int64_t base = static_cast<int64_t>(r) * cap * K;
    const int last = min(n, (chunk + 1) * kLayoutChunk);
    for (int i = chunk * kLayoutChunk + threadIdx.x; i < last; i += kRowThreads) {
        const int e = expert_of(idx, base + i, EL, status);
        if (e >= 0) atomicAdd(&hist[e], 1);
    }
    __syncthreads();
    int32_t* const mine = counts + static_cast<int64_t>(r) * chunks * EL;
    for (int j = threadIdx.x; j < EL; j += kRowThreads) mine[static_cast<int64_t>(chunk) * EL + j] = hist[j];
    // publish this CTA's counts, then take a ticket; the last one sees them all
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        last_of_rank = atomicAdd(&tickets[r], 1u) == static_cast<uint32_t>(max(used, 1)) - 1u;
        if (last_of_rank) tickets[r] = 0;
    }
    __syncthreads();
    if (!last_of_rank) return;
    __threadfence();
    for (int j = threadIdx.x / kWarpSize; j < EL; j += kRowWarps) {
        int total = 0;
        for (int c0 = 0; c0 < used; c0 += kWarpSize) {
            const int c = c0 + lane_id();
            int32_t* at = mine + static_cast<int64_t>(c) * EL + j;
            const int v = c < used ? __ldcg(at) : 0;
            int scan = v;
#pragma unroll
            for (int o = 1; o < kWarpSize; o <<= 1) {
                const int u = __shfl_up_sync(kFullMask, scan, o);
                if (lane_id() >= o) scan += u;
            }
            if (c < used) *at = total + scan - v;
            total += __shfl_sync(kFullMask, scan, kWarpSize - 1);
        }
        if (lane_id() == 0) group_count[r * EL + j] = total;
    }
}

// Begins of the experts (each rounded up to the alignment), and every slot's row.
__global__ void __launch_bounds__(kRowThreads)
    layout_place_kernel(const int64_t* idx, const int32_t* num_recv, int cap, int K, int EL, int experts, int alignment,
                        int64_t num_rows, const int32_t* before_chunk, const int32_t* group_count, int32_t* group_begin,
                        int32_t* slot_row, int32_t* status) {
    extern __shared__ int32_t place[];  // [1 + kRowWarps][EL]: the chunk's first row per expert, then per warp
    __shared__ int64_t sums[kRowWarps];
    pdl_enter();
    const int r = blockIdx.y, chunk = blockIdx.x, warp = threadIdx.x / kWarpSize;
    const int n = filled_slots(num_recv, r, cap, K);
    const int64_t base = static_cast<int64_t>(r) * cap * K;
    const int slots = cap * K;
    const bool first_cta = chunk == 0 && r == 0;
    if (chunk * kLayoutChunk < n || first_cta) {
        const int per = (experts + kRowThreads - 1) / kRowThreads;
        const int first = threadIdx.x * per, last = min(first + per, experts);
        int64_t sum = 0;
        for (int e = first; e < last; ++e) sum += (group_count[e] + static_cast<int64_t>(alignment) - 1) / alignment * alignment;
        // prefix over the block, in 64 bits: padding may pass 2^31 before the capacity check below
        int64_t scan = sum;
#pragma unroll
        for (int o = 1; o < kWarpSize; o <<= 1) {
            const int64_t u = __shfl_up_sync(kFullMask, scan, o);
            if (lane_id() >= o) scan += u;
        }
        if (lane_id() == kWarpSize - 1) sums[warp] = scan;
        __syncthreads();
        int64_t at = scan - sum;
        for (int w = 0; w < warp; ++w) at += sums[w];
        for (int e = first; e < last; ++e) {
            const int32_t begin = static_cast<int32_t>(min(at, static_cast<int64_t>(INT32_MAX)));
            if (first_cta) group_begin[e] = begin;
            if (e / EL == r) place[e % EL] = begin;
            at += (group_count[e] + static_cast<int64_t>(alignment) - 1) / alignment * alignment;
        }
        for (int j = threadIdx.x; j < kRowWarps * EL; j += kRowThreads) place[EL + j] = 0;
        __syncthreads();
    }
    int32_t* mine = place + (1 + warp) * EL;
    int expert[kWarpSlots / kWarpSize];
    const int from = chunk * kLayoutChunk + warp * kWarpSlots;
#pragma unroll
    for (int s = 0; s < kWarpSlots / kWarpSize; ++s) {
        const int i = from + s * kWarpSize + lane_id();
        expert[s] = i < n ? expert_of(idx, base + i, EL, status) : -1;
        if (expert[s] >= 0) atomicAdd(&mine[expert[s]], 1);
    }
    if (chunk * kLayoutChunk < n) {
        __syncthreads();
        const int32_t* before = before_chunk + (static_cast<int64_t>(r) * gridDim.x + chunk) * EL;
        for (int j = threadIdx.x; j < EL; j += kRowThreads) {
            uint32_t at = static_cast<uint32_t>(place[j]) + before[j];
            for (int w = 1; w <= kRowWarps; ++w) {
                const int c = place[w * EL + j];
                place[w * EL + j] = static_cast<int32_t>(at);
                at += c;
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int s = 0; s < kWarpSlots / kWarpSize; ++s) {
        const int i = from + s * kWarpSize + lane_id();
        const int e = expert[s];
        const unsigned same = __match_any_sync(kFullMask, e);
        int row = -1;
        if (e >= 0) {
            // unsigned: a begin past the rows there are, cut to 2^31 - 1, plus the rows before this one
            const uint32_t at = static_cast<uint32_t>(mine[e]) + __popc(same & lanemask_lt());
            if (at < num_rows) row = static_cast<int>(at);
            else report(status, EP_ERR_CAPACITY);
        }
        __syncwarp();
        if (e >= 0 && (same & lanemask_lt()) == 0) mine[e] += __popc(same);
        __syncwarp();
        if (i < slots) slot_row[base + i] = row;
    }
}

// The (rank, row) of the i-th received row; `upto`: lane r holds the rows of ranks 0..r.
struct Received {
    int upto, total;
};

__device__ __forceinline__ Received received_rows(const int32_t* num_recv, int R, int cap) {
    int v = lane_id() < R ? max(0, min(num_recv[lane_id()], cap)) : 0;
#pragma unroll
    for (int o = 1; o < kWarpSize; o <<= 1) {
        const int u = __shfl_up_sync(kFullMask, v, o);
        if (lane_id() >= o) v += u;
    }
    return {v, __shfl_sync(kFullMask, v, kWarpSize - 1)};
}

// Index in [R * cap] of the i-th received row.
__device__ __forceinline__ int64_t received_at(const Received& q, int i, int cap) {
    const int r = __popc(__ballot_sync(kFullMask, q.upto <= i));
    const int before = __shfl_sync(kFullMask, q.upto, r == 0 ? 0 : r - 1);
    return static_cast<int64_t>(r) * cap + (i - (r == 0 ? 0 : before));
}

struct GatherParams {
    const uint8_t* x;
    const float* x_scales;
    const float* topk_weights;
    const int32_t* slot_row;
    const int32_t* num_recv;
    uint8_t* out;
    float* out_scales;
    float* row_weights;
    int64_t row_bytes;
    int64_t num_rows;
    int32_t ranks, cap, topk, scale_words;
    int32_t pieces, piece_bytes, stages;
    int32_t* status;
};

__global__ void __launch_bounds__(kWarpSize) rows_gather_kernel(const GatherParams p) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ uint64_t full[kGatherMaxStages];
    if (lane_id() == 0) {
        for (int i = 0; i < p.stages; ++i) mbar_init(&full[i], 1);
        fence_barrier_init();
    }
    __syncwarp();
    pdl_enter();
    const Received q = received_rows(p.num_recv, p.ranks, p.cap);
    const int64_t units = static_cast<int64_t>(q.total) * p.pieces;
    // runs of `stages` units, dealt out in turn: a CTA's copies in flight are neighbours
    const int64_t runs = (units + p.stages - 1) / p.stages;
    const int64_t my_runs = blockIdx.x < runs ? (runs - blockIdx.x + gridDim.x - 1) / gridDim.x : 0;
    int64_t mine = my_runs * p.stages;
    if (my_runs > 0 && blockIdx.x + (my_runs - 1) * gridDim.x == runs - 1) mine -= runs * p.stages - units;

    // unit u of this CTA: a piece of a received row
    auto unit = [&](int64_t u, int64_t* row, int64_t* offset, uint32_t* bytes) {
        const int64_t at = (blockIdx.x + u / p.stages * gridDim.x) * p.stages + u % p.stages;
        *row = received_at(q, static_cast<int>(at / p.pieces), p.cap);
        *offset = at % p.pieces * p.piece_bytes;
        *bytes = static_cast<uint32_t>(min(static_cast<int64_t>(p.piece_bytes), p.row_bytes - *offset));
    };
    auto load = [&](int64_t u) {
        int64_t row, offset;
        uint32_t bytes;
        unit(u, &row, &offset, &bytes);
        if (lane_id() == 0) {
            const int s = static_cast<int>(u % p.stages);
            mbar_arrive_expect_tx(&full[s], bytes);
            bulk_load(ring + static_cast<int64_t>(s) * p.piece_bytes, p.x + row * p.row_bytes + offset, bytes, &full[s]);
        }
    };
    int64_t loaded = 0;
    for (; loaded < mine && loaded < p.stages - 1; ++loaded) load(loaded);
    bool ok = true;
    int64_t u = 0;
    for (; u < mine; ++u) {
        int64_t row, offset;
        uint32_t bytes;
        unit(u, &row, &offset, &bytes);
        int to = lane_id() < p.topk ? p.slot_row[row * p.topk + lane_id()] : -1;
        if (to >= p.num_rows) {
            report(p.status, EP_ERR_CAPACITY);
            to = -1;
        }
        if (offset == 0 && to >= 0 && p.row_weights) p.row_weights[to] = p.topk_weights[row * p.topk + lane_id()];
        if (offset == 0 && p.out_scales) {
            for (int w0 = 0; w0 < p.scale_words; w0 += kWarpSize) {
                const int w = w0 + lane_id();
                const float v = w < p.scale_words ? p.x_scales[row * p.scale_words + w] : 0.0f;
                for (unsigned m = __ballot_sync(kFullMask, to >= 0); m; m &= m - 1) {
                    const int dst = __shfl_sync(kFullMask, to, __ffs(m) - 1);
                    if (w < p.scale_words) p.out_scales[static_cast<int64_t>(dst) * p.scale_words + w] = v;
                }
            }
        }
        const int s = static_cast<int>(u % p.stages);
        ok = __all_sync(kFullMask, mbar_wait_bounded(&full[s], static_cast<uint32_t>(u / p.stages) & 1));
        if (!ok) break;
        if (to >= 0)
            bulk_store(p.out + static_cast<int64_t>(to) * p.row_bytes + offset, ring + static_cast<int64_t>(s) * p.piece_bytes,
                       bytes);
        bulk_commit();
        // the stage of the unit before this one is free once every lane's stores have read it
        bulk_wait_read<1>();
        __syncwarp();
        if (loaded < mine) load(loaded), ++loaded;
    }
    if (!ok) {
        report(p.status, EP_ERR_TIMEOUT);
        for (; u < loaded; ++u) mbar_wait_bounded(&full[u % p.stages], static_cast<uint32_t>(u / p.stages) & 1, 1u << 12);
    }
    bulk_wait_all();
}

struct ReduceParams {
    const uint8_t* y;
    int64_t y_row_bytes;
    const int32_t* slot_row;
    const int32_t* num_recv;
    const float* row_weights;
    uint8_t* out;
    float* out_topk_weights;
    int64_t num_rows;
    int32_t hidden, ranks, cap, topk;
    int32_t* status;
};

__global__ void __launch_bounds__(kRowThreads) rows_reduce_kernel(const ReduceParams p) {
    pdl_enter();
    // Loads in flight per lane: four column blocks of one row.  Two rows at once took registers from a third CTA per SM
    // and were slower (16288 rows of 4096 bytes: 23.9 against 22.0 us on one card).
    constexpr int kCols = 4;
    const Received q = received_rows(p.num_recv, p.ranks, p.cap);
    const int warps = gridDim.x * kRowWarps;
    for (int i = blockIdx.x * kRowWarps + threadIdx.x / kWarpSize; i < q.total; i += warps) {
        const int64_t row = received_at(q, i, p.cap);
        int from = lane_id() < p.topk ? p.slot_row[row * p.topk + lane_id()] : -1;
        if (from >= p.num_rows) {
            report(p.status, EP_ERR_CAPACITY);
            from = -1;
        }
        if (p.out_topk_weights && lane_id() < p.topk)
            p.out_topk_weights[row * p.topk + lane_id()] = from >= 0 ? p.row_weights[from] : 0.0f;
        const unsigned there = __ballot_sync(kFullMask, from >= 0);
        uint8_t* out = p.out + row * 2 * p.hidden;
        for (int c0 = lane_id() * 8; c0 - lane_id() * 8 < p.hidden; c0 += kCols * kWarpSize * 8) {
            float acc[kCols][8];
#pragma unroll
            for (int c = 0; c < kCols; ++c)
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[c][j] = 0.0f;
            for (unsigned m = there; m; m &= m - 1) {
                const uint8_t* y = p.y + __shfl_sync(kFullMask, from, __ffs(m) - 1) * p.y_row_bytes;
                int4 v[kCols];
#pragma unroll
                for (int c = 0; c < kCols; ++c) {
                    const int64_t col = c0 + c * kWarpSize * 8;
                    v[c] = col < p.hidden ? ld_stream_v4(reinterpret_cast<const int4*>(y + 2 * col)) : make_int4(0, 0, 0, 0);
                }
#pragma unroll
                for (int c = 0; c < kCols; ++c) {
                    float f[8];
                    unpack8(v[c], f);
#pragma unroll
                    for (int j = 0; j < 8; ++j) acc[c][j] += f[j];
                }
            }
#pragma unroll
            for (int c = 0; c < kCols; ++c) {
                const int col = c0 + c * kWarpSize * 8;
                if (col < p.hidden) st_stream_v4(reinterpret_cast<int4*>(out + 2 * static_cast<int64_t>(col)), pack8_bf16(acc[c]));
            }
        }
    }
}

// num_recv of a call: the caller's, or the record's of the last normal dispatch.
ep_status received(const ep_handle* h, const int32_t* num_recv, const int32_t** use) {
    if (h == nullptr) return fail(EP_ERR_INVALID_ARG, "handle is NULL");
    EP_CHECK_ARG(h->cfg.recv_capacity > 0, "handle was created with recv_capacity 0 (normal mode disabled)");
    if (h->cfg.recv_capacity * h->cfg.num_topk > INT32_MAX - kLayoutChunk || h->cfg.recv_capacity * h->cfg.num_ranks > INT32_MAX)
        return fail(EP_ERR_UNSUPPORTED, "recv_capacity %lld: recv_capacity * num_topk or * num_ranks exceeds 2^31",
                    static_cast<long long>(h->cfg.recv_capacity));
    EP_CHECK_ARG(aligned4(num_recv), "misaligned num_recv");
    if (num_recv == nullptr && h->normal_tokens < 0)
        return fail(EP_ERR_STATE, "no num_recv, and no normal dispatch on this handle yet");
    *use = num_recv ? num_recv : h->num_recv;
    return EP_OK;
}

ep_status check_rows(int64_t num_rows) {
    EP_CHECK_ARG(num_rows >= 0 && num_rows <= INT32_MAX, "num_rows %lld outside [0, 2^31)",
                 static_cast<long long>(num_rows));
    return EP_OK;
}

cudaError_t plan_rows(LaunchPlan* plan) {
    int per_sm = 0;
    cudaError_t err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, rows_reduce_kernel, kRowThreads, 0);
    plan->reduce_blocks = plan->num_sms * (per_sm > 0 ? per_sm : 1);
    if (err == cudaSuccess)
        err = cudaFuncSetAttribute(layout_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           (1 + kRowWarps) * kMaxExperts * static_cast<int>(sizeof(int32_t)));
    if (err == cudaSuccess)
        err = cudaFuncSetAttribute(rows_gather_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kGatherSmem);
    return err;
}

ep_status planned(ep_handle* h) {
    return plan_once(&h->plan.rows_ready, [h] { return plan_rows(&h->plan); });
}

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" {

ep_status ep_expert_layout(ep_handle* h, const int64_t* recv_topk_idx, const int32_t* num_recv, int64_t num_rows,
                           int32_t* group_count, int32_t* group_begin, int32_t* slot_row, ep_stream_t stream) {
    EP_TRACE();
    const int32_t* recv = nullptr;
    ep_status st = received(h, num_recv, &recv);
    if (st == EP_OK) st = check_rows(num_rows);
    if (st != EP_OK) return st;
    EP_CHECK_ARG(recv_topk_idx && aligned8(recv_topk_idx), "recv_topk_idx must be an 8-byte aligned device pointer");
    EP_CHECK_ARG(group_count && group_begin && slot_row && aligned4(group_count) && aligned4(group_begin) && aligned4(slot_row),
                 "group_count, group_begin and slot_row are required");
    const ep_config& c = h->cfg;
    const int R = c.num_ranks, E = c.num_experts, EL = E / R, cap = static_cast<int>(c.recv_capacity), K = c.num_topk;
    const int chunks = static_cast<int>(layout_chunks(c));
    DeviceGuard guard(h->device);
    st = planned(h);
    if (st != EP_OK) return st;
    cudaError_t err = launch_kernel(layout_count_kernel, dim3(chunks, R), dim3(kRowThreads), EL * sizeof(int32_t), stream, 1,
                                    recv_topk_idx, recv, cap, K, EL, h->expert_counts,
                                    reinterpret_cast<uint32_t*>(h->layout_tickets), group_count, h->status);
    if (err == cudaSuccess)
        err = launch_kernel(layout_place_kernel, dim3(chunks, R), dim3(kRowThreads), (1 + kRowWarps) * EL * sizeof(int32_t),
                            stream, 1, recv_topk_idx, recv, cap, K, EL, E, c.expert_alignment, num_rows, h->expert_counts,
                            group_count, group_begin, slot_row, h->status);
    if (err != cudaSuccess) return cuda_fail(err, "expert layout launch");
    return EP_OK;
}

ep_status ep_expert_gather(ep_handle* h, const void* x, ep_dtype x_dtype, const float* x_scales,
                           const float* topk_weights, const int32_t* slot_row, const int32_t* num_recv, int64_t num_rows,
                           void* out, float* out_scales, float* row_weights, ep_stream_t stream) {
    EP_TRACE();
    GatherParams p = {};
    ep_status st = received(h, num_recv, &p.num_recv);
    if (st == EP_OK) st = check_rows(num_rows);
    if (st != EP_OK) return st;
    const ep_config& c = h->cfg;
    EP_CHECK_ARG(x_dtype == EP_BF16 || x_dtype == EP_FP8_E4M3, "x_dtype must be EP_BF16 or EP_FP8_E4M3");
    const bool fp8 = x_dtype == EP_FP8_E4M3;
    if (fp8 && c.hidden % kFp8Group != 0)
        return fail(EP_ERR_UNSUPPORTED, "FP8 payloads need hidden %% 128 == 0 (hidden %d)", c.hidden);
    EP_CHECK_ARG(x && aligned16(x) && slot_row && aligned4(slot_row), "x (16-byte aligned) and slot_row are required");
    EP_CHECK_ARG(num_rows == 0 || (out && aligned16(out)), "out must be a 16-byte aligned device pointer");
    EP_CHECK_ARG((x_scales != nullptr) == fp8 && (out_scales != nullptr) == (fp8 && num_rows > 0) && aligned4(x_scales) &&
                     aligned4(out_scales),
                 "x_scales and out_scales go with an FP8 payload");
    EP_CHECK_ARG((topk_weights != nullptr) == (row_weights != nullptr) && aligned4(topk_weights) && aligned4(row_weights),
                 "topk_weights and row_weights go together");
    if (num_rows == 0) return EP_OK;
    p.x = static_cast<const uint8_t*>(x);
    p.x_scales = x_scales;
    p.topk_weights = topk_weights;
    p.slot_row = slot_row;
    p.out = static_cast<uint8_t*>(out);
    p.out_scales = out_scales;
    p.row_weights = row_weights;
    p.row_bytes = static_cast<int64_t>(c.hidden) * (fp8 ? 1 : 2);
    p.num_rows = num_rows;
    p.ranks = c.num_ranks;
    p.cap = static_cast<int32_t>(c.recv_capacity);
    p.topk = c.num_topk;
    p.scale_words = fp8 ? c.hidden / kFp8Group : 0;
    p.pieces = static_cast<int32_t>((p.row_bytes + kGatherPiece - 1) / kGatherPiece);
    p.piece_bytes = p.pieces == 1 ? static_cast<int32_t>(p.row_bytes) : kGatherPiece;
    p.stages = kGatherSmem / p.piece_bytes < kGatherMaxStages ? kGatherSmem / p.piece_bytes : kGatherMaxStages;
    p.status = h->status;
    const int64_t units = static_cast<int64_t>(p.cap) * p.ranks * p.pieces;
    const int64_t runs = (units + p.stages - 1) / p.stages;
    const int64_t most = static_cast<int64_t>(h->plan.num_sms) * kGatherPerSm * (h->plan.sm_limited ? 1 : kGatherWaves);
    DeviceGuard guard(h->device);
    st = planned(h);
    if (st != EP_OK) return st;
    const cudaError_t err = launch_kernel(rows_gather_kernel, dim3(static_cast<unsigned>(runs < most ? runs : most)),
                                          dim3(kWarpSize), static_cast<size_t>(p.stages) * p.piece_bytes, stream, 1, p);
    if (err != cudaSuccess) return cuda_fail(err, "expert gather launch");
    return EP_OK;
}

ep_status ep_expert_reduce(ep_handle* h, const void* y, int64_t y_row_bytes, const int32_t* slot_row,
                           const float* row_weights, const int32_t* num_recv, int64_t num_rows, void* out,
                           float* out_topk_weights, ep_stream_t stream) {
    EP_TRACE();
    ReduceParams p = {};
    ep_status st = received(h, num_recv, &p.num_recv);
    if (st == EP_OK) st = check_rows(num_rows);
    if (st != EP_OK) return st;
    const ep_config& c = h->cfg;
    EP_CHECK_ARG(num_rows == 0 || (y && aligned16(y)), "y must be a 16-byte aligned device pointer");
    EP_CHECK_ARG(y_row_bytes >= 2 * static_cast<int64_t>(c.hidden) && y_row_bytes % 16 == 0,
                 "y_row_bytes %lld must be a multiple of 16 that holds a row", static_cast<long long>(y_row_bytes));
    EP_CHECK_ARG(slot_row && aligned4(slot_row) && out && aligned16(out), "slot_row and out (16-byte aligned) are required");
    EP_CHECK_ARG((row_weights != nullptr) == (out_topk_weights != nullptr) && aligned4(row_weights) && aligned4(out_topk_weights),
                 "row_weights and out_topk_weights go together");
    p.y = static_cast<const uint8_t*>(y);
    p.y_row_bytes = y_row_bytes;
    p.slot_row = slot_row;
    p.row_weights = row_weights;
    p.out = static_cast<uint8_t*>(out);
    p.out_topk_weights = out_topk_weights;
    p.num_rows = num_rows;
    p.hidden = c.hidden;
    p.ranks = c.num_ranks;
    p.cap = static_cast<int32_t>(c.recv_capacity);
    p.topk = c.num_topk;
    p.status = h->status;
    const int64_t wanted = (static_cast<int64_t>(p.cap) * p.ranks + kRowWarps - 1) / kRowWarps;
    DeviceGuard guard(h->device);
    st = planned(h);
    if (st != EP_OK) return st;
    const int64_t most = h->plan.reduce_blocks;  // resident at once: warps stride over the rows
    const cudaError_t err = launch_kernel(rows_reduce_kernel, dim3(static_cast<unsigned>(wanted < most ? wanted : most)),
                                          dim3(kRowThreads), 0, stream, 1, p);
    if (err != cudaSuccess) return cuda_fail(err, "expert reduce launch");
    return EP_OK;
}

}  // extern "C"
