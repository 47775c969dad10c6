// ep_act.cu -- the gradient of the products' epilogue (sm_103a).
//
// From dy (of the output, without what a residual adds to it) and v (the product with its bias, as kept in bf16):
//   not gated   d v = dy * w * act'(v)                                   d w = sum over the row of dy * act(v)
//   gated       d gate = dy * w * up * act'(gate),  d up = dy * w * act(gate)     d w = sum of dy * act(gate) * up
// with the row's weight w (1 without), and d bias[e] = the sum of the unrounded d v over the rows of expert e.
//
// A CTA takes kChunkRows rows of one group, a warp kWarpRows of them, 256 columns at a time: a lane's sums over its rows
// stay in registers, its rows' sums over columns in a word of shared memory each.  The warps' column sums are added up
// through shared memory and go out as one row of partial sums a chunk; a second kernel adds up the chunks of each
// group in their order.  No atomics: the same input gives the same sums.
#include "ep_act.cuh"
#include "ep_groups.cuh"
#include "ep_handle.h"
#include "ep_trace.h"

namespace ep {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / kWarpSize;
constexpr int kWarpRows = 4;
constexpr int kChunkRows = kWarps * kWarpRows;
constexpr int kLaneCols = 8;
constexpr int kWarpCols = kWarpSize * kLaneCols;

struct ActGradParams {
    Groups groups;
    int32_t width;
    const uint8_t* dy;
    int64_t dy_row_bytes;
    const uint8_t* pre;       // NULL: not needed
    int64_t pre_row_bytes;
    const float* row_weights;
    uint8_t* d_pre;           // NULL: not wanted
    int64_t d_pre_row_bytes;
    float* d_row_weights;
    float* partial;           // [chunks][n] column sums, or NULL
    float* d_bias;            // [groups][n]
    int32_t* status;
};

// The table of chunks before each group, in shared memory; returns how many there are, -1 where groups overlap.
__device__ __forceinline__ int build_chunks(const Groups& groups, int32_t* before, int32_t* begin, int32_t* count,
                                            int64_t* sums, int32_t* status) {
    const int per = (groups.groups + kThreads - 1) / kThreads;
    const int first = threadIdx.x * per, last = min(first + per, groups.groups);
    int64_t chunks = 0, rows = 0, all_chunks = 0, all_rows = 0;
    for (int g = first; g < last; ++g) {
        const Group q = load_group(groups, g, status);
        before[g] = static_cast<int32_t>(chunks);
        begin[g] = q.begin;
        count[g] = q.count;
        chunks += (q.count + kChunkRows - 1) / kChunkRows;
        rows += q.count;
    }
    block_prefix<kThreads>(rows, sums, &all_rows);
    __syncthreads();
    const int64_t base = block_prefix<kThreads>(chunks, sums, &all_chunks);
    for (int g = first; g < last; ++g) before[g] += static_cast<int32_t>(base);
    __syncthreads();
    if (all_rows > groups.num_rows) {
        report(status, EP_ERR_CAPACITY);
        return -1;
    }
    return static_cast<int>(all_chunks);
}

template <int ACT, bool kGated>
__global__ void __launch_bounds__(kThreads) act_grad_kernel(const ActGradParams p) {
    constexpr int kParts = kGated ? 2 : 1;
    extern __shared__ int32_t table[];
    __shared__ int64_t sums[kWarps];
    __shared__ float row_sums[kChunkRows][kWarpSize];
    __shared__ float4 col_sums[kWarps][kParts * kWarpSize * 2];
    const int groups = p.groups.groups;
    int32_t* before = table;
    int32_t* begin = before + groups;
    int32_t* count = begin + groups;
    pdl_enter();
    const int chunks = build_chunks(p.groups, before, begin, count, sums, p.status);
    const int warp = threadIdx.x / kWarpSize;
    const int n = kParts * p.width;
    const int64_t half = 2 * static_cast<int64_t>(p.width);  // bytes from gate to up
    for (int chunk = blockIdx.x; chunk < chunks; chunk += gridDim.x) {
        const int g = find_group(before, groups, chunk);
        const int in_group = (chunk - before[g]) * kChunkRows + warp * kWarpRows;
        const int rows = min(kWarpRows, count[g] - in_group);
        const int64_t row0 = static_cast<int64_t>(begin[g]) + in_group;
#pragma unroll
        for (int r = 0; r < kWarpRows; ++r) row_sums[warp * kWarpRows + r][lane_id()] = 0.0f;
        for (int c0 = 0; c0 < p.width; c0 += kWarpCols) {
            const int col = c0 + lane_id() * kLaneCols;
            const bool in = col < p.width;
            float acc[kParts][kLaneCols];
#pragma unroll
            for (int i = 0; i < kParts; ++i)
#pragma unroll
                for (int j = 0; j < kLaneCols; ++j) acc[i][j] = 0.0f;
#pragma unroll 2
            for (int r = 0; r < rows; ++r) {
                if (!in) break;
                const int64_t row = row0 + r;
                const int4 d4 = ld_stream_v4(reinterpret_cast<const int4*>(p.dy + row * p.dy_row_bytes + 2 * col));
                int4 v4 = make_int4(0, 0, 0, 0), u4 = v4;
                if (p.pre) {
                    const uint8_t* pre = p.pre + row * p.pre_row_bytes + 2 * col;
                    v4 = ld_stream_v4(reinterpret_cast<const int4*>(pre));
                    if (kGated) u4 = ld_stream_v4(reinterpret_cast<const int4*>(pre + half));
                }
                const float w = p.row_weights ? __ldg(p.row_weights + row) : 1.0f;
                float d[8], v[8], u[8], dv[8], du[8];
                unpack8(d4, d);
                unpack8(v4, v);
                if (kGated) unpack8(u4, u);
                float dot = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 a = activate_with_slope(ACT, v[j]);
                    const float dw = d[j] * w;
                    dv[j] = kGated ? dw * u[j] * a.y : dw * a.y;
                    dot += kGated ? d[j] * a.x * u[j] : d[j] * a.x;
                    acc[0][j] += dv[j];
                    if (kGated) du[j] = dw * a.x, acc[kParts - 1][j] += du[j];
                }
                if (p.d_pre) {
                    uint8_t* out = p.d_pre + row * p.d_pre_row_bytes + 2 * col;
                    st_stream_v4(reinterpret_cast<int4*>(out), pack8_bf16(dv));
                    if (kGated) st_stream_v4(reinterpret_cast<int4*>(out + half), pack8_bf16(du));
                }
                row_sums[warp * kWarpRows + r][lane_id()] += dot;
            }
            if (p.partial) {
#pragma unroll
                for (int i = 0; i < kParts; ++i) {
                    col_sums[warp][(i * 2 + 0) * kWarpSize + lane_id()] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
                    col_sums[warp][(i * 2 + 1) * kWarpSize + lane_id()] = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
                }
                __syncthreads();
                // thread: four columns of a part
                for (int i = threadIdx.x; i < kParts * 2 * kWarpSize; i += kThreads) {
                    float4 s = col_sums[0][i];
#pragma unroll
                    for (int w = 1; w < kWarps; ++w) {
                        const float4 t = col_sums[w][i];
                        s.x += t.x, s.y += t.y, s.z += t.z, s.w += t.w;
                    }
                    const int part = i / (2 * kWarpSize), quad = i / kWarpSize % 2, c = c0 + (i % kWarpSize) * kLaneCols + 4 * quad;
                    if (c < p.width)
                        *reinterpret_cast<float4*>(p.partial + static_cast<int64_t>(chunk) * n + static_cast<int64_t>(part) * p.width + c) = s;
                }
                __syncthreads();
            }
        }
        if (p.d_row_weights) {
            __syncwarp();
#pragma unroll
            for (int r = 0; r < kWarpRows; ++r) {
                float s = row_sums[warp * kWarpRows + r][lane_id()];
#pragma unroll
                for (int o = kWarpSize / 2; o > 0; o >>= 1) s += __shfl_xor_sync(kFullMask, s, o);
                if (lane_id() == 0 && r < rows) p.d_row_weights[row0 + r] = s;
            }
        }
    }
}

// d bias: the chunks' rows of partial sums, added up for each group.  A CTA has 128 columns of one group, a warp every
// kWarps-th chunk of it.
__global__ void __launch_bounds__(kThreads) bias_sum_kernel(const ActGradParams p, int n) {
    extern __shared__ int32_t table[];
    __shared__ int64_t sums[kWarps];
    __shared__ float4 col_sums[kWarps][kWarpSize];
    const int groups = p.groups.groups;
    int32_t* before = table;
    int32_t* begin = before + groups;
    int32_t* count = begin + groups;
    pdl_enter();
    if (build_chunks(p.groups, before, begin, count, sums, p.status) < 0) return;
    const int warp = threadIdx.x / kWarpSize;
    const int blocks = (n + 4 * kWarpSize - 1) / (4 * kWarpSize);
    for (int64_t item = blockIdx.x; item < static_cast<int64_t>(groups) * blocks; item += gridDim.x) {
        const int g = static_cast<int>(item / blocks);
        const int col = static_cast<int>(item % blocks) * 4 * kWarpSize + 4 * lane_id();
        const int chunks = (count[g] + kChunkRows - 1) / kChunkRows;
        const float* from = p.partial + static_cast<int64_t>(before[g]) * n + col;
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (col < n) {
#pragma unroll 4
            for (int c = warp; c < chunks; c += kWarps) {
                const float4 t = *reinterpret_cast<const float4*>(from + static_cast<int64_t>(c) * n);
                s.x += t.x, s.y += t.y, s.z += t.z, s.w += t.w;
            }
        }
        col_sums[warp][lane_id()] = s;
        __syncthreads();
        if (warp == 0 && col < n) {
#pragma unroll
            for (int w = 1; w < kWarps; ++w) {
                const float4 t = col_sums[w][lane_id()];
                s.x += t.x, s.y += t.y, s.z += t.z, s.w += t.w;
            }
            *reinterpret_cast<float4*>(p.d_bias + static_cast<int64_t>(g) * n + col) = s;
        }
        __syncthreads();
    }
}

size_t table_bytes(int groups) { return 3 * sizeof(int32_t) * static_cast<size_t>(groups); }

int64_t most_chunks(int64_t num_rows, int groups) { return num_rows / kChunkRows + groups; }

template <int ACT, bool kGated>
cudaError_t start(const ep_handle* h, const ActGradParams& p, cudaStream_t stream) {
    const int64_t wanted = most_chunks(p.groups.num_rows, p.groups.groups);
    const int64_t most = static_cast<int64_t>(h->plan.num_sms) * (h->plan.sm_limited ? 4 : 16);
    return launch_kernel(act_grad_kernel<ACT, kGated>, dim3(static_cast<unsigned>(wanted < most ? wanted : most)), dim3(kThreads),
                         table_bytes(p.groups.groups), stream, 1, p);
}

template <bool kGated>
cudaError_t start_act(const ep_handle* h, const ActGradParams& p, int act, cudaStream_t stream) {
    switch (act) {
        case EP_ACT_RELU: return start<EP_ACT_RELU, kGated>(h, p, stream);
        case EP_ACT_SILU: return start<EP_ACT_SILU, kGated>(h, p, stream);
        case EP_ACT_GELU: return start<EP_ACT_GELU, kGated>(h, p, stream);
        default: return start<EP_ACT_NONE, kGated>(h, p, stream);
    }
}

bool rows_ok(const void* p, int64_t bytes, int64_t least) { return aligned16(p) && bytes >= least && bytes % 16 == 0 && bytes < (INT64_C(1) << 40); }

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" {

int64_t ep_act_grad_workspace(const ep_handle* h, int64_t num_rows, int32_t n) {
    if (h == nullptr || num_rows < 0 || num_rows > INT32_MAX || n < 0) return -1;
    return most_chunks(num_rows, h->cfg.num_experts) * n * static_cast<int64_t>(sizeof(float));
}

ep_status ep_act_grad(ep_handle* h, int64_t num_rows, int32_t n, const int32_t* group_count, const int32_t* group_begin,
                      const void* dy, int64_t dy_row_bytes, const void* pre, int64_t pre_row_bytes, int32_t act,
                      int32_t gated, const float* row_weights, void* d_pre, int64_t d_pre_row_bytes, float* d_row_weights,
                      float* d_bias, void* workspace, int64_t workspace_bytes, ep_stream_t stream) {
    EP_TRACE();
    if (h == nullptr) return fail(EP_ERR_INVALID_ARG, "handle is NULL");
    const ep_status st = check_group_args(h, num_rows, group_count, group_begin);
    if (st != EP_OK) return st;
    EP_CHECK_ARG(n >= 8 && n % 8 == 0 && n <= (1 << 28) && (!gated || n % 16 == 0),
                 "n %d must be a positive multiple of 8, gated: two widths of one", n);
    EP_CHECK_ARG(act >= EP_ACT_NONE && act <= EP_ACT_GELU, "act %d is no activation", act);
    const int32_t width = gated ? n / 2 : n;
    EP_CHECK_ARG(d_bias == nullptr || aligned16(d_bias), "d_bias must be 16-byte aligned");
    DeviceGuard guard(h->device);
    if (num_rows == 0) {
        if (d_bias == nullptr) return EP_OK;
        const cudaError_t err = cudaMemsetAsync(d_bias, 0, static_cast<size_t>(h->cfg.num_experts) * n * sizeof(float), stream);
        return err == cudaSuccess ? EP_OK : cuda_fail(err, "clearing d_bias");
    }
    EP_CHECK_ARG(dy && rows_ok(dy, dy_row_bytes, 2 * static_cast<int64_t>(width)),
                 "dy must be 16-byte aligned with a row stride in multiples of 16 that holds a row (%lld bytes)", static_cast<long long>(dy_row_bytes));
    EP_CHECK_ARG(pre || (act == EP_ACT_NONE && !gated && !d_row_weights), "pre may be NULL only without activation, gate and d_row_weights");
    EP_CHECK_ARG(!pre || rows_ok(pre, pre_row_bytes, 2 * static_cast<int64_t>(n)),
                 "pre must be 16-byte aligned with a row stride in multiples of 16 that holds a row (%lld bytes)", static_cast<long long>(pre_row_bytes));
    EP_CHECK_ARG(!d_pre || rows_ok(d_pre, d_pre_row_bytes, 2 * static_cast<int64_t>(n)),
                 "d_pre must be 16-byte aligned with a row stride in multiples of 16 that holds a row (%lld bytes)", static_cast<long long>(d_pre_row_bytes));
    EP_CHECK_ARG(aligned4(row_weights) && aligned4(d_row_weights), "misaligned row_weights or d_row_weights");
    const int64_t need = ep_act_grad_workspace(h, num_rows, n);
    EP_CHECK_ARG(!d_bias || (workspace && aligned16(workspace) && workspace_bytes >= need),
                 "d_bias needs a 16-byte aligned workspace of %lld bytes (ep_act_grad_workspace), got %lld",
                 static_cast<long long>(need), static_cast<long long>(workspace_bytes));
    ActGradParams p = {};
    p.groups = {group_count, group_begin, num_rows, static_cast<int32_t>(num_rows / h->cfg.num_experts), h->cfg.num_experts};
    p.width = width;
    p.dy = static_cast<const uint8_t*>(dy);
    p.dy_row_bytes = dy_row_bytes;
    p.pre = static_cast<const uint8_t*>(pre);
    p.pre_row_bytes = pre_row_bytes;
    p.row_weights = row_weights;
    p.d_pre = static_cast<uint8_t*>(d_pre);
    p.d_pre_row_bytes = d_pre_row_bytes;
    p.d_row_weights = d_row_weights;
    p.partial = d_bias ? static_cast<float*>(workspace) : nullptr;
    p.d_bias = d_bias;
    p.status = h->status;
    cudaError_t err = gated ? start_act<true>(h, p, act, stream) : start_act<false>(h, p, act, stream);
    if (err == cudaSuccess && d_bias) {
        const int64_t wanted = static_cast<int64_t>(h->cfg.num_experts) * ((n + 4 * kWarpSize - 1) / (4 * kWarpSize));
        const int64_t most = static_cast<int64_t>(h->plan.num_sms) * (h->plan.sm_limited ? 4 : 16);
        err = launch_kernel(bias_sum_kernel, dim3(static_cast<unsigned>(wanted < most ? wanted : most)), dim3(kThreads),
                            table_bytes(h->cfg.num_experts), stream, 1, p, n);
    }
    if (err != cudaSuccess) return cuda_fail(err, "activation gradient launch");
    return EP_OK;
}

}  // extern "C"
