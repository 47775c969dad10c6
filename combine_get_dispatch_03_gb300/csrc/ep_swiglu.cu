// ep_swiglu.cu -- the gated activation between an expert's two products, and its gradient (sm_103a).
//
// A row of the first product holds gate and up values, [gate: width][up: width] bf16.  With
// sig = 1 / (1 + exp(-gate)) and the row's weight p (1 without weights):
//   forward    v = gate * sig * up * p, to bf16, or to e4m3 codes and one scale per 128 columns
//   gradient   dgate = dv * p * up * sig * (1 + gate * (1 - sig));  dup = dv * p * gate * sig;
//              dp = sum over the row of dv * gate * sig * up
// All in fp32, rounded once.  2^x and the reciprocal are the hardware's approximations, and a value is good to 2^-20 at
// every gate above -87 (sigmoid2).  Below -88.7 exp(-gate) passes fp32 and the sigmoid is 0, as in the formula in 32 bits; in
// 64 bits a gate of -90 would leave 7e-38 * up.  The kernels are near the bound of their instructions, not only of memory.
//
// A warp owns a row: 32 lanes of 8 columns, so that a scale's 128 columns are 16 lanes and their maximum four
// shuffles.  Only rows of a group are touched; warps stride over them through the group table.
//
// Measured on a GB300 (6787 GB/s copied): the cast of 131072 rows of 2048 217 us, 6.2 TB/s, 72 % of the issue
// slots before the correction; the gradient of 32672 rows of 1024 50.3 us, 6.6 TB/s; 128 rows of 1024 3.0 us, a launch.
#include "ep_groups.cuh"
#include "ep_handle.h"
#include "ep_trace.h"

namespace ep {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = 4;  // CTAs per resident CTA: the GPU's own balancing, 54.9 -> 50.3 us for the gradient of 32672 rows
constexpr int kLaneCols = 8;
constexpr int kWarpCols = kWarpSize * kLaneCols;

struct SwigluParams {
    Groups groups;
    int32_t width;
    int32_t round_scale;
    const uint8_t* x;
    int64_t x_row_bytes;
    const uint8_t* dy;
    int64_t dy_row_bytes;
    const float* row_weights;
    uint8_t* out;
    int64_t out_row_bytes;
    float* out_scales;      // [num_rows][width / 128]
    float* d_row_weights;   // [num_rows]
    int32_t* status;
};

enum SwigluForm { kToBf16 = 0, kToFp8 = 1, kGradient = 2 };

// 1 / (1 + exp(-g)) of a bf16 gate.  exp(-g) = 2^(-g * hi) * exp(-g * lo) with log2(e) = hi + lo / ln(2): hi has 15
// significant bits and g 8, so that the product which goes into the exponent is exact, and lo is small enough for
// 1 - g * lo (second order: 1e-7 at g = -90; past 128 the first factor is 0).  One product with log2(e) rounded to 24 bits
// was off by 5e-7 at |gate| = 16 and 4e-6 at 80.  The reciprocal is taken of a quarter of the sum, which the flushing
// instruction leaves a normal result of up to exp(-g) = 2^128: gates down to -88.7 keep a (subnormal) sigmoid, below
// that it is 0, as exp(-g) is infinite in 32 bits.
// Two gates at a time: the cast of 131072 rows of 2048 takes 214.6 us without the correction, 222.6 with it one by one, 216.6 packed
// (with the products that follow).
__device__ __forceinline__ float2 sigmoid2(float2 g) {
    constexpr float kHi = 1.44268798828125f, kLo = 4.8884951521e-6f;
    const float2 quarter = make_float2(0.25f, 0.25f);
    const float2 t = __fmul2_rn(g, make_float2(-kHi, -kHi));
    float2 e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
    e = __ffma2_rn(e, __fmul2_rn(make_float2(fminf(g.x, 128.0f), fminf(g.y, 128.0f)), make_float2(-kLo, -kLo)), e);
    e = __ffma2_rn(e, quarter, quarter);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(e.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(e.y));
    return __fmul2_rn(r, quarter);
}

template <int FORM>
__device__ __forceinline__ void swiglu_row(const SwigluParams& p, int64_t row) {
    const uint8_t* gate = p.x + row * p.x_row_bytes;
    const uint8_t* up = gate + 2 * static_cast<int64_t>(p.width);
    const uint8_t* dy = FORM == kGradient ? p.dy + row * p.dy_row_bytes : nullptr;
    uint8_t* out = p.out + row * p.out_row_bytes;
    const float weight = p.row_weights ? p.row_weights[row] : 1.0f;
    float dp = 0.0f;
    // two passes of 256 columns at a time: up to six 16-byte loads of a lane in flight
    for (int c0 = 0; c0 < p.width; c0 += 2 * kWarpCols) {
        int4 g4[2], u4[2], d4[2];
        int col[2];
        bool in[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            col[i] = c0 + i * kWarpCols + lane_id() * kLaneCols;
            in[i] = col[i] < p.width;
            if (in[i]) {
                g4[i] = ld_stream_v4(reinterpret_cast<const int4*>(gate + 2 * col[i]));
                u4[i] = ld_stream_v4(reinterpret_cast<const int4*>(up + 2 * col[i]));
                if (FORM == kGradient) d4[i] = ld_stream_v4(reinterpret_cast<const int4*>(dy + 2 * col[i]));
            } else {
                g4[i] = u4[i] = d4[i] = make_int4(0, 0, 0, 0);
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (c0 + i * kWarpCols >= p.width) break;
            float g[8], u[8];
            unpack8(g4[i], g);
            unpack8(u4[i], u);
            float sig[8], act[8];  // act = g * sig
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const float2 two = make_float2(g[j], g[j + 1]);
                const float2 s = sigmoid2(two), a = __fmul2_rn(two, s);
                sig[j] = s.x, sig[j + 1] = s.y;
                act[j] = a.x, act[j + 1] = a.y;
            }
            if constexpr (FORM == kGradient) {
                float d[8], dg[8], du[8];
                unpack8(d4[i], d);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float dv = d[j] * weight;
                    dg[j] = dv * u[j] * (sig[j] * (1.0f + g[j] * (1.0f - sig[j])));
                    du[j] = dv * act[j];
                    dp += d[j] * act[j] * u[j];
                }
                if (in[i]) {
                    st_stream_v4(reinterpret_cast<int4*>(out + 2 * col[i]), pack8_bf16(dg));
                    st_stream_v4(reinterpret_cast<int4*>(out + 2 * (static_cast<int64_t>(p.width) + col[i])), pack8_bf16(du));
                }
            } else {
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    const float2 a = __fmul2_rn(make_float2(act[j], act[j + 1]), make_float2(u[j], u[j + 1]));
                    const float2 two = __fmul2_rn(a, make_float2(weight, weight));
                    v[j] = two.x, v[j + 1] = two.y;
                }
                if constexpr (FORM == kToBf16) {
                    if (in[i]) st_stream_v4(reinterpret_cast<int4*>(out + 2 * col[i]), pack8_bf16(v));
                } else {
                    float amax = absmax8(v);
#pragma unroll
                    for (int o = 1; o < kFp8Group / kLaneCols; o <<= 1)
                        amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, o));
                    const Fp8Scale s = fp8_scale(amax, p.round_scale != 0);
                    // of an infinite scale 0 (as 448 / amax is), where the power of two has none
                    const float mult = isinf(s.scale) ? 0.0f : s.mult;
                    if (in[i]) {
                        st_stream_v2(reinterpret_cast<int2*>(out + col[i]), cast8_e4m3(v, mult));
                        if (lane_id() % (kFp8Group / kLaneCols) == 0)
                            p.out_scales[row * (p.width / kFp8Group) + col[i] / kFp8Group] = s.scale;
                    }
                }
            }
        }
    }
    if (FORM == kGradient && p.d_row_weights) {
#pragma unroll
        for (int o = kWarpSize / 2; o > 0; o >>= 1) dp += __shfl_xor_sync(kFullMask, dp, o);
        if (lane_id() == 0) p.d_row_weights[row] = dp;
    }
}

template <int FORM>
__global__ void __launch_bounds__(kThreads) swiglu_kernel(const SwigluParams p) {
    extern __shared__ int32_t table[];
    __shared__ int64_t sums[kThreads / kWarpSize];
    const int groups = p.groups.groups;
    int32_t* before = table;              // [groups] rows before each group
    int32_t* begin = table + groups;      // [groups]
    pdl_enter();
    const int per = (groups + kThreads - 1) / kThreads;
    const int first = threadIdx.x * per, last = min(first + per, groups);
    int64_t sum = 0, rows = 0;
    for (int g = first; g < last; ++g) {
        const Group q = load_group(p.groups, g, p.status);
        before[g] = static_cast<int32_t>(sum);
        begin[g] = q.begin;
        sum += q.count;
    }
    const int64_t base = block_prefix<kThreads>(sum, sums, &rows);
    if (rows > p.groups.num_rows) {  // overlapping groups
        report(p.status, EP_ERR_CAPACITY);
        return;
    }
    for (int g = first; g < last; ++g) before[g] += static_cast<int32_t>(base);
    __syncthreads();
    const int total = static_cast<int>(rows);
    const int warps = gridDim.x * (kThreads / kWarpSize);
    for (int i = blockIdx.x * (kThreads / kWarpSize) + threadIdx.x / kWarpSize; i < total; i += warps) {
        const int g = find_group(before, groups, i);
        swiglu_row<FORM>(p, static_cast<int64_t>(begin[g]) + (i - before[g]));
    }
}

size_t table_bytes(int groups) { return 2 * sizeof(int32_t) * static_cast<size_t>(groups); }

template <int FORM>
cudaError_t plan_form(LaunchPlan* plan, int groups) {
    int per_sm = 0;
    const cudaError_t err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, swiglu_kernel<FORM>, kThreads, table_bytes(groups));
    plan->swiglu_blocks[FORM] = plan->num_sms * (plan->sm_limited ? 1 : kWaves) * (per_sm > 0 ? per_sm : 1);
    return err;
}

cudaError_t plan_swiglu(LaunchPlan* plan, int groups) {
    cudaError_t err = plan_form<kToBf16>(plan, groups);
    if (err == cudaSuccess) err = plan_form<kToFp8>(plan, groups);
    if (err == cudaSuccess) err = plan_form<kGradient>(plan, groups);
    return err;
}

template <int FORM>
ep_status launch(ep_handle* h, const SwigluParams& p, cudaStream_t stream) {
    DeviceGuard guard(h->device);
    const ep_status planned = plan_once(&h->plan.swiglu_ready, [h] { return plan_swiglu(&h->plan, h->cfg.num_experts); });
    if (planned != EP_OK) return planned;
    // no more warps than rows; past kWaves waves, warps stride over the rows
    const int64_t wanted = (p.groups.num_rows + kThreads / kWarpSize - 1) / (kThreads / kWarpSize);
    const int64_t most = h->plan.swiglu_blocks[FORM];
    const cudaError_t err = launch_kernel(swiglu_kernel<FORM>, dim3(static_cast<unsigned>(wanted < most ? wanted : most)),
                                          dim3(kThreads), table_bytes(p.groups.groups), stream, 1, p);
    if (err != cudaSuccess) return cuda_fail(err, "swiglu launch");
    return EP_OK;
}

ep_status check(const ep_handle* h, int64_t num_rows, int32_t width, const int32_t* group_count,
                const int32_t* group_begin, const void* x, int64_t x_row_bytes, const float* row_weights,
                SwigluParams* p) {
    if (h == nullptr) return fail(EP_ERR_INVALID_ARG, "handle is NULL");
    const ep_status st = check_group_args(h, num_rows, group_count, group_begin);
    if (st != EP_OK) return st;
    EP_CHECK_ARG(width >= 8 && width % 8 == 0 && width <= (1 << 28), "width %d must be a positive multiple of 8", width);
    EP_CHECK_ARG(num_rows == 0 || (x && aligned16(x)), "x must be a 16-byte aligned device pointer");
    EP_CHECK_ARG(x_row_bytes >= 4 * static_cast<int64_t>(width) && x_row_bytes % 16 == 0,
                 "x_row_bytes %lld must be a multiple of 16 and hold 2 * width = %d values",
                 static_cast<long long>(x_row_bytes), 2 * width);
    EP_CHECK_ARG(aligned4(row_weights), "misaligned row_weights");
    p->groups = {group_count, group_begin, num_rows, static_cast<int32_t>(num_rows / h->cfg.num_experts),
                 h->cfg.num_experts};
    p->width = width;
    p->x = static_cast<const uint8_t*>(x);
    p->x_row_bytes = x_row_bytes;
    p->row_weights = row_weights;
    p->status = h->status;
    return EP_OK;
}

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" {

ep_status ep_swiglu(ep_handle* h, int64_t num_rows, int32_t width, const int32_t* group_count,
                    const int32_t* group_begin, const void* x, int64_t x_row_bytes, const float* row_weights,
                    int32_t cast_to_fp8, int32_t round_scale, void* out, int64_t out_row_bytes, float* out_scales,
                    ep_stream_t stream) {
    EP_TRACE();
    SwigluParams p = {};
    const ep_status st = check(h, num_rows, width, group_count, group_begin, x, x_row_bytes, row_weights, &p);
    if (st != EP_OK) return st;
    if (cast_to_fp8 && width % kFp8Group != 0)
        return fail(EP_ERR_UNSUPPORTED, "the FP8 cast needs width %% 128 == 0 (width %d)", width);
    EP_CHECK_ARG(cast_to_fp8 || (!round_scale && out_scales == nullptr), "scales go with cast_to_fp8");
    EP_CHECK_ARG(!cast_to_fp8 || num_rows == 0 || (out_scales && aligned4(out_scales)), "cast_to_fp8 needs out_scales");
    EP_CHECK_ARG(num_rows == 0 || (out && aligned16(out)), "out must be a 16-byte aligned device pointer");
    EP_CHECK_ARG(out_row_bytes >= static_cast<int64_t>(width) * (cast_to_fp8 ? 1 : 2) && out_row_bytes % 16 == 0,
                 "out_row_bytes %lld must be a multiple of 16 that holds a row", static_cast<long long>(out_row_bytes));
    if (num_rows == 0) return EP_OK;
    p.round_scale = round_scale != 0;
    p.out = static_cast<uint8_t*>(out);
    p.out_row_bytes = out_row_bytes;
    p.out_scales = out_scales;
    return cast_to_fp8 ? launch<kToFp8>(h, p, stream) : launch<kToBf16>(h, p, stream);
}

ep_status ep_swiglu_grad(ep_handle* h, int64_t num_rows, int32_t width, const int32_t* group_count,
                         const int32_t* group_begin, const void* dy, int64_t dy_row_bytes, const void* x,
                         int64_t x_row_bytes, const float* row_weights, void* dx, int64_t dx_row_bytes,
                         float* d_row_weights, ep_stream_t stream) {
    EP_TRACE();
    SwigluParams p = {};
    const ep_status st = check(h, num_rows, width, group_count, group_begin, x, x_row_bytes, row_weights, &p);
    if (st != EP_OK) return st;
    EP_CHECK_ARG(num_rows == 0 || (dy && dx && aligned16(dy) && aligned16(dx)),
                 "dy and dx must be 16-byte aligned device pointers");
    EP_CHECK_ARG(dy_row_bytes >= 2 * static_cast<int64_t>(width) && dy_row_bytes % 16 == 0 &&
                     dx_row_bytes >= 4 * static_cast<int64_t>(width) && dx_row_bytes % 16 == 0,
                 "row strides must be multiples of 16 that hold a row (dy %lld, dx %lld bytes)",
                 static_cast<long long>(dy_row_bytes), static_cast<long long>(dx_row_bytes));
    EP_CHECK_ARG(aligned4(d_row_weights), "misaligned d_row_weights");
    if (num_rows == 0) return EP_OK;
    p.dy = static_cast<const uint8_t*>(dy);
    p.dy_row_bytes = dy_row_bytes;
    p.out = static_cast<uint8_t*>(dx);
    p.out_row_bytes = dx_row_bytes;
    p.d_row_weights = d_row_weights;
    return launch<kGradient>(h, p, stream);
}

}  // extern "C"
