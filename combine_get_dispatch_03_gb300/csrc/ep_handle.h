// ep_handle.h -- the handle behind include/ep.h and the host-side helpers every entry point uses
// (internal to the library).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "ep_kernels.h"

namespace ep {
constexpr uint64_t kWaitLimitNs = 4000000000ull;
}

struct ep_handle {
    ep_config cfg;
    int device = -1;
    ep::LaunchPlan plan;
    void* dmem = nullptr;
    size_t dmem_bytes = 0;
    int32_t* status = nullptr;
    int32_t* rank_prefix = nullptr;          // [R][R]
    int32_t* channel_prefix = nullptr;       // [R][R][C]
    int32_t* recv_channel_prefix = nullptr;  // [R][R][C]
    int32_t* num_recv = nullptr;             // [R]
    int32_t* recv_src_idx = nullptr;         // [R][cap]
    int32_t* send_head = nullptr;            // [R][maxT][R]
    int32_t* ll_slot = nullptr;              // [R][maxT][K]
    int32_t* ll_cnt = nullptr;               // [R][E]
    int32_t* rank_mask = nullptr;            // [R], nonzero = masked
    int32_t* rdma_channel_prefix = nullptr;    // [R][NN][C], NN = R / 8 whole nodes (see has_nodes)
    int32_t* recv_rdma_rank_prefix = nullptr;  // [R][NN]
    int32_t* claims = nullptr;                 // [2]: the combine's next token and finished warps
    int32_t* layout_scratch = nullptr;         // tile states of the one-pass layout + record scan
    int32_t* expert_counts = nullptr;          // [R][layout_chunks][EL]: the expert layout's counts per chunk of slots
    int32_t* layout_tickets = nullptr;         // [R]: CTAs of a rank that the expert layout has counted
    int normal_tokens = -1;                  // T of the current dispatch record, -1 = none
    bool prepared = false;                   // record built by ep_notify_dispatch, not yet used
    int ll_tokens = -1;                      // T of the last LL dispatch, -1 = none
    uint64_t wait_limit_ns = ep::kWaitLimitNs;  // of a wait inside the grouped products
};

namespace ep {

// Sets the calling thread's ep_last_error() text and returns `code`.
ep_status fail(ep_status code, const char* fmt, ...);
ep_status cuda_fail(cudaError_t err, const char* what);

#define EP_CHECK_ARG(cond, ...)                                           \
    do {                                                                  \
        if (!(cond)) return ::ep::fail(EP_ERR_INVALID_ARG, __VA_ARGS__);  \
    } while (0)

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

// The checks of rows grouped by expert that every expert call shares.
ep_status check_group_args(const ep_handle* h, int64_t num_rows, const int32_t* group_count, const int32_t* group_begin);

// Makes the handle's device current for the duration of a call.
class DeviceGuard {
public:
    explicit DeviceGuard(int device) {
        cudaGetDevice(&prev_);
        if (prev_ != device) cudaSetDevice(device);
        restore_ = prev_ != device;
    }
    ~DeviceGuard() {
        if (restore_) cudaSetDevice(prev_);
    }

private:
    int prev_ = 0;
    bool restore_ = false;
};

// Makes a part of the handle's launch plan when the first call needs it: a handle that only dispatches loads none of the
// experts' kernels (eleven products, 0.7 ms and 2 MB of device memory in a process's first handle).  That call may be
// under stream capture; nothing here belongs to the stream.
template <typename Plan>
ep_status plan_once(bool* ready, Plan plan) {
    if (*ready) return EP_OK;
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    cudaError_t err = cudaThreadExchangeStreamCaptureMode(&mode);
    if (err == cudaSuccess) {
        err = plan();
        const cudaError_t back = cudaThreadExchangeStreamCaptureMode(&mode);
        if (err == cudaSuccess) err = back;
    }
    if (err != cudaSuccess) return cuda_fail(err, "planning launches");
    *ready = true;
    return EP_OK;
}

}  // namespace ep
