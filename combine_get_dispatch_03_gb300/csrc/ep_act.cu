// ep_act.cu -- the gradient of the products' epilogue (sm_103a).
//
// From dy (of the output, without what a residual adds to it) and v (the product with its bias, as kept in bf16):
//   not gated   d v = dy * w * act'(v)                                   d w = sum over the row of dy * act(v)
//   gated       d gate = dy * w * up * act'(gate),  d up = dy * w * act(gate)     d w = sum of dy * act(gate) * up
// with the row's weight w (1 without), and d bias[e] = the sum of the unrounded d v over the rows of expert e.
//
// A CTA takes chunk_rows() rows of one group.  A warp has 256 columns of them, all of its rows, or where there are fewer than
// 2048 columns every second, third... row: a lane's column sums stay in registers, and what the warps have of the same
// columns is added up through shared memory once a chunk, as are the rows' sums.  (With rows for each warp and the columns in
// turn, two barriers for every 256 columns: 69 us for 32672 rows of 1024 gates and ups.)  The column sums go out as one row
// of partial sums a chunk; a second kernel adds up the chunks of each group in their order.  No atomics: the same
// input gives the same sums.
#include "ep_act.cuh"
#include "ep_groups.cuh"
#include "ep_handle.h"
#include "ep_trace.h"

namespace ep {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / kWarpSize;
constexpr int kMostChunkRows = 64;
constexpr int kLaneCols = 8;
constexpr int kWarpCols = kWarpSize * kLaneCols;

// Rows of a chunk: fewer where there are few rows, so that every SM has some; more of many, whose partial sums cost less then.  By the rows
// alone: the sums' order is the same whatever the handle may use of the GPU.  us at 8, 16, 32, 64 rows a chunk, 32 groups, gated
// 2 x 1024 columns, all sums: 4096 rows 15.9, 16.6, 18.8, 25.2; 8192 24.6, 24.2, 26.3, 33.7; 16384 43.6, 40.3, 42.0, 46.0; 24576 59, 56, 53,
// 51; 31968 74, 68, 69, 80; 48000 107, 96, 95, 95; 65536 145, 126, 122, 129; 98304 223, 187, 175, 178; 131072 293, 253, 229, 227.  Not gated, 264
// columns: 4096 rows 11.7, 11.3, 14.2, 17.1; 11968 20, 16, 15, 21; 16384 25, 19, 19, 21; 48000 56, 43, 37, 35; 98304 104, 76, 68, 65.
__host__ __device__ inline int chunk_rows(int64_t num_rows) { return num_rows >= 100000 ? kMostChunkRows : num_rows >= 32000 ? 32 : num_rows >= 12000 ? 16 : 8; }

struct ActGradParams {
    Groups groups;
    int32_t width;
    const uint8_t* dy;
    int64_t dy_row_bytes;
    const uint8_t* pre;       // NULL: not needed; it may be d_pre
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
template <int THREADS>
__device__ __forceinline__ int build_chunks(const Groups& groups, int32_t* before, int32_t* begin, int32_t* count,
                                            int64_t* sums, int32_t* status) {
    const int each = chunk_rows(groups.num_rows);
    const int per = (groups.groups + THREADS - 1) / THREADS;
    const int first = threadIdx.x * per, last = min(first + per, groups.groups);
    int64_t chunks = 0, rows = 0, all_chunks = 0, all_rows = 0;
    for (int g = first; g < last; ++g) {
        const Group q = load_group(groups, g, status);
        before[g] = static_cast<int32_t>(chunks);
        begin[g] = q.begin;
        count[g] = q.count;
        chunks += (q.count + each - 1) / each;
        rows += q.count;
    }
    block_prefix<THREADS>(rows, sums, &all_rows);
    __syncthreads();
    const int64_t base = block_prefix<THREADS>(chunks, sums, &all_chunks);
    for (int g = first; g < last; ++g) before[g] += static_cast<int32_t>(base);
    __syncthreads();
    if (all_rows > groups.num_rows) {
        report(status, EP_ERR_CAPACITY);
        return -1;
    }
    return static_cast<int>(all_chunks);
}

template <int ACT, bool kGated>
__global__ void __launch_bounds__(kThreads, 3) act_grad_kernel(const ActGradParams p) {
    constexpr int kParts = kGated ? 2 : 1;
    constexpr int kRows = kGated ? 2 : 4;  // in flight
    extern __shared__ int32_t table[];
    __shared__ int64_t sums[kWarps];
    __shared__ float row_sums[kMostChunkRows][kWarps];
    __shared__ float4 col_sums[kWarps][kParts * kWarpSize * 2];
    const int groups = p.groups.groups;
    int32_t* before = table;
    int32_t* begin = before + groups;
    int32_t* count = begin + groups;
    pdl_enter();
    const int chunks = build_chunks<kThreads>(p.groups, before, begin, count, sums, p.status);
    const int warp = threadIdx.x / kWarpSize;
    const int n = kParts * p.width, each = chunk_rows(p.groups.num_rows);
    const int64_t half = 2 * static_cast<int64_t>(p.width);  // bytes from gate to up
    const int blocks = (p.width + kWarpCols - 1) / kWarpCols;  // of columns
    const int across = min(blocks, kWarps), turns = kWarps / across;  // warps side by side, and sharing rows
    const int mine = warp / across, block0 = warp % across;
    for (int chunk = blockIdx.x; chunk < chunks; chunk += gridDim.x) {
        const int g = find_group(before, groups, chunk);
        const int in_group = (chunk - before[g]) * each;
        const int rows = min(each, count[g] - in_group);
        const int64_t row0 = static_cast<int64_t>(begin[g]) + in_group;
        for (int block = block0; mine < turns && block < blocks; block += across) {
            const int col = block * kWarpCols + lane_id() * kLaneCols;
            const bool in = col < p.width;
            float2 acc[kParts][kLaneCols / 2];
#pragma unroll
            for (int i = 0; i < kParts; ++i)
#pragma unroll
                for (int j = 0; j < kLaneCols / 2; ++j) acc[i][j] = both(0.0f);
            for (int r0 = mine; r0 < rows; r0 += kRows * turns) {
                int4 d4[kRows], v4[kRows], u4[kRows];
                float w[kRows];
#pragma unroll
                for (int i = 0; i < kRows; ++i) {
                    const int64_t row = row0 + r0 + i * turns;
                    d4[i] = v4[i] = u4[i] = make_int4(0, 0, 0, 0);
                    w[i] = 1.0f;
                    if (r0 + i * turns < rows && in) {
                        d4[i] = ld_stream_v4(reinterpret_cast<const int4*>(p.dy + row * p.dy_row_bytes + 2 * col));
                        if (p.pre) {
                            const uint8_t* pre = p.pre + row * p.pre_row_bytes + 2 * col;
                            v4[i] = ld_stream_written_v4(reinterpret_cast<const int4*>(pre));
                            if (kGated) u4[i] = ld_stream_written_v4(reinterpret_cast<const int4*>(pre + half));
                        }
                        if (p.row_weights) w[i] = __ldg(p.row_weights + row);
                    }
                }
#pragma unroll
                for (int i = 0; i < kRows; ++i) {
                    const int r = r0 + i * turns;
                    if (r >= rows) break;
                    float d[8], v[8], u[8], dv[8], du[8];
                    unpack8(d4[i], d);
                    unpack8(v4[i], v);
                    if (kGated) unpack8(u4[i], u);
                    float2 dot = both(0.0f);
#pragma unroll
                    for (int j = 0; j < 8; j += 2) {
                        float2 slope;
                        const float2 a = activate_with_slope(ACT, make_float2(v[j], v[j + 1]), &slope);
                        const float2 dd = make_float2(d[j], d[j + 1]), dw = __fmul2_rn(dd, both(w[i]));
                        float2 one = __fmul2_rn(dw, slope), value = a;
                        if (kGated) {
                            const float2 uu = make_float2(u[j], u[j + 1]), two = __fmul2_rn(dw, a);
                            one = __fmul2_rn(one, uu);
                            value = __fmul2_rn(a, uu);
                            du[j] = two.x, du[j + 1] = two.y;
                            acc[kParts - 1][j / 2] = __fadd2_rn(acc[kParts - 1][j / 2], two);
                        }
                        dot = __ffma2_rn(dd, value, dot);
                        dv[j] = one.x, dv[j + 1] = one.y;
                        acc[0][j / 2] = __fadd2_rn(acc[0][j / 2], one);
                    }
                    if (p.d_pre && in) {
                        uint8_t* out = p.d_pre + (row0 + r) * p.d_pre_row_bytes + 2 * col;
                        st_stream_v4(reinterpret_cast<int4*>(out), pack8_bf16(dv));
                        if (kGated) st_stream_v4(reinterpret_cast<int4*>(out + half), pack8_bf16(du));
                    }
                    if (p.d_row_weights) {
                        float s = dot.x + dot.y;
#pragma unroll
                        for (int o = kWarpSize / 2; o > 0; o >>= 1) s += __shfl_xor_sync(kFullMask, s, o);
                        if (lane_id() == 0) row_sums[r][block0] = block == block0 ? s : row_sums[r][block0] + s;
                    }
                }
            }
            if (p.partial) {
#pragma unroll
                for (int i = 0; i < kParts; ++i) {
                    const float4 low = make_float4(acc[i][0].x, acc[i][0].y, acc[i][1].x, acc[i][1].y);
                    const float4 high = make_float4(acc[i][2].x, acc[i][2].y, acc[i][3].x, acc[i][3].y);
                    if (turns > 1) {
                        col_sums[warp][i * 2 * kWarpSize + 2 * lane_id()] = low;
                        col_sums[warp][i * 2 * kWarpSize + 2 * lane_id() + 1] = high;
                    } else if (in) {
                        float4* to = reinterpret_cast<float4*>(p.partial + static_cast<int64_t>(chunk) * n + static_cast<int64_t>(i) * p.width + col);
                        to[0] = low, to[1] = high;
                    }
                }
            }
        }
        if ((p.partial && turns > 1) || p.d_row_weights) {
            __syncthreads();
            if (p.partial && turns > 1)
                for (int i = threadIdx.x; i < kParts * across * 2 * kWarpSize; i += kThreads) {  // four columns of a part
                    const int part = i / (across * 2 * kWarpSize), quad = i % (across * 2 * kWarpSize), w = quad / (2 * kWarpSize);
                    float4 s = col_sums[w][part * 2 * kWarpSize + quad % (2 * kWarpSize)];
                    for (int k = 1; k < turns; ++k) {
                        const float4 t = col_sums[k * across + w][part * 2 * kWarpSize + quad % (2 * kWarpSize)];
                        s.x += t.x, s.y += t.y, s.z += t.z, s.w += t.w;
                    }
                    if (4 * quad < p.width)
                        *reinterpret_cast<float4*>(p.partial + static_cast<int64_t>(chunk) * n + static_cast<int64_t>(part) * p.width + 4 * quad) = s;
                }
            if (p.d_row_weights && static_cast<int>(threadIdx.x) < rows) {
                float s = row_sums[threadIdx.x][0];
                for (int k = 1; k < across; ++k) s += row_sums[threadIdx.x][k];
                p.d_row_weights[row0 + threadIdx.x] = s;
            }
            __syncthreads();
        }
    }
}

// d bias: the chunks' rows of partial sums, added up for each group.  A CTA has 128 columns of one group, a warp
// every kSumWarps-th chunk of it: many warps where few CTAs have something to do (1 group of 32672 rows, 512 columns: 24 us for
// eight warps, 11 for 32; 32 groups of 1021 rows, 2048 columns: 7 and 19).
template <int kSumThreads>
__global__ void __launch_bounds__(kSumThreads) bias_sum_kernel(const ActGradParams p, int n) {
    constexpr int kSumWarps = kSumThreads / kWarpSize;
    extern __shared__ int32_t table[];
    __shared__ int64_t sums[kSumWarps];
    __shared__ float4 col_sums[kSumWarps][kWarpSize];
    const int groups = p.groups.groups;
    int32_t* before = table;
    int32_t* begin = before + groups;
    int32_t* count = begin + groups;
    pdl_enter();
    if (build_chunks<kSumThreads>(p.groups, before, begin, count, sums, p.status) < 0) return;
    const int warp = threadIdx.x / kWarpSize, each = chunk_rows(p.groups.num_rows);
    const int blocks = (n + 4 * kWarpSize - 1) / (4 * kWarpSize);
    for (int64_t item = blockIdx.x; item < static_cast<int64_t>(groups) * blocks; item += gridDim.x) {
        const int g = static_cast<int>(item / blocks);
        const int col = static_cast<int>(item % blocks) * 4 * kWarpSize + 4 * lane_id();
        const int chunks = (count[g] + each - 1) / each;
        const float* from = p.partial + static_cast<int64_t>(before[g]) * n + col;
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (col < n) {
#pragma unroll 4
            for (int c = warp; c < chunks; c += kSumWarps) {
                const float4 t = *reinterpret_cast<const float4*>(from + static_cast<int64_t>(c) * n);
                s.x += t.x, s.y += t.y, s.z += t.z, s.w += t.w;
            }
        }
        col_sums[warp][lane_id()] = s;
        __syncthreads();
        const int used = min(chunks, kSumWarps);
        if (warp == 0 && col < n) {
            for (int w = 1; w < used; ++w) {
                const float4 t = col_sums[w][lane_id()];
                s.x += t.x, s.y += t.y, s.z += t.z, s.w += t.w;
            }
            *reinterpret_cast<float4*>(p.d_bias + static_cast<int64_t>(g) * n + col) = s;
        }
        __syncthreads();
    }
}

size_t table_bytes(int groups) { return 3 * sizeof(int32_t) * static_cast<size_t>(groups); }

int64_t most_chunks(int64_t num_rows, int groups) { return num_rows / chunk_rows(num_rows) + groups; }

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
        const dim3 grid(static_cast<unsigned>(wanted < most ? wanted : most));
        const size_t table = table_bytes(h->cfg.num_experts);
        err = wanted >= 256 ? launch_kernel(bias_sum_kernel<256>, grid, dim3(256), table, stream, 1, p, n)
                            : launch_kernel(bias_sum_kernel<1024>, grid, dim3(1024), table, stream, 1, p, n);
    }
    if (err != cudaSuccess) return cuda_fail(err, "activation gradient launch");
    return EP_OK;
}

}  // extern "C"
