// What the plans beside the matrix products share: the device a plan is
// bound to, and the device memory its calls write (workspaces).  Host only.
#pragma once

#include <cstring>
#include <new>

#include <cuda_runtime.h>

#include "olc_matmul.h"
#include "stream_order.h"

namespace olc {

constexpr int kPlanDefaultSms = 152;   // GB300; used while no device is visible
constexpr int64_t kPlanMaxBytes = int64_t(1) << 62;   // as for the matrix plans: offsets fit int64

inline olc_status plan_status(cudaError_t e) {
    if (e == cudaSuccess) return OLC_OK;
    cudaGetLastError();
    return e == cudaErrorMemoryAllocation ? OLC_ERR_OOM : OLC_ERR_CUDA;
}

// a * b * bytes within the largest tensor the plans accept (a, b >= 0)
inline bool plan_fits(int64_t a, int64_t b, int64_t bytes) {
    int64_t n;
    if (a == 0 || b == 0) return true;
    return !__builtin_mul_overflow(a, b, &n) && !__builtin_mul_overflow(n, bytes, &n) && n <= kPlanMaxBytes;
}

#ifdef __CUDACC__
// A launch in full stream order.  The kernels of these plans neither start
// before their predecessor has ended nor let a successor start early
// (programmatic dependent launch).  An earlier form of them did, and under a
// stress of the gated product's gradient its stream once stood still.  Which
// part did it was not shown: roles that met .aligned barriers with their warps
// apart were mended in the same days, and a dependent grid's blocks are only
// placed when all of its predecessor's are.  Full order needs no such answer.
template <typename... KArgs, typename... Args>
inline cudaError_t plan_launch(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                               Args&&... args) {
    kernel<<<grid, block, smem, s>>>(static_cast<KArgs>(args)...);
    return cudaGetLastError();
}
#endif

inline int64_t plan_elem_bytes(olc_dtype dt) { return dt == OLC_FLOAT ? 4 : 2; }
inline bool plan_dtype_ok(int dt) { return dt == OLC_FLOAT || dt == OLC_FLOAT16 || dt == OLC_BFLOAT16; }
inline bool plan_misaligned(const void* p, int64_t bytes) {
    return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) != 0;
}
inline bool plan_aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Device binding and the plan's own device memory, with the order of the calls
// that use it.
struct PlanState : StreamOrder {
    struct Earlier {
        void* memory;
        Earlier* next;
    };
    int device;              // -1: made while no device was visible
    int sm_count;
    void* memory;
    size_t bytes;
    Earlier* earlier;        // smaller blocks that `memory` has replaced

    void init() {
        std::memset(this, 0, sizeof *this);
        device = -1;
        sm_count = kPlanDefaultSms;
        int n = 0, dev = 0, sms = 0;
        if (cudaGetDeviceCount(&n) == cudaSuccess && n > 0 && cudaGetDevice(&dev) == cudaSuccess &&
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && sms > 0) {
            device = dev;
            sm_count = sms;
        }
        cudaGetLastError();
    }

    // the current device has to be the plan's
    olc_status bind() {
        int cur = -1;
        if (cudaGetDevice(&cur) != cudaSuccess) return plan_status(cudaErrorNoDevice);
        if (device < 0) device = cur;
        return cur == device ? OLC_OK : OLC_ERR_WRONG_DEVICE;
    }

    // Grow the plan's memory.  A graph captured earlier may name the smaller
    // block: it is kept until the plan is destroyed.
    olc_status ensure(size_t want) {
        if (want <= bytes) return OLC_OK;
        Earlier* const keep = memory ? new (std::nothrow) Earlier{memory, earlier} : nullptr;
        void* larger = nullptr;
        const cudaError_t e = memory && !keep ? cudaErrorMemoryAllocation : cudaMalloc(&larger, want);
        if (e != cudaSuccess) {
            delete keep;
            return plan_status(e);
        }
        if (keep) earlier = keep;
        memory = larger;
        bytes = want;
        return OLC_OK;
    }

    // free another piece of device memory of the plan (null: nothing)
    void release(void* p) {
        if (p) on_device([&] { cudaFree(p); });
    }

    void destroy() {
        release(memory);
        memory = nullptr;
        bytes = 0;
        while (earlier) {
            Earlier* const e = earlier;
            earlier = e->next;
            release(e->memory);
            delete e;
        }
        if (event) on_device([&] { cudaEventDestroy(event); });
        event = nullptr;
    }

  private:
    template <typename F>
    void on_device(F&& f) {
        int cur = -1;
        cudaGetDevice(&cur);
        if (device >= 0 && cur != device) cudaSetDevice(device);
        f();
        if (device >= 0 && cur >= 0 && cur != device) cudaSetDevice(cur);
        cudaGetLastError();
    }
};

}  // namespace olc
