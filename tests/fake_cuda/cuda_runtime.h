// A stand-in for the CUDA runtime's header: just what plan_state.h calls, each
// call counted or written down, so that its rules run on a host without a GPU.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <string>

enum cudaError_t { cudaSuccess = 0, cudaErrorMemoryAllocation = 2, cudaErrorNoDevice = 100, cudaErrorLaunchFailure = 719 };
enum cudaStreamCaptureStatus { cudaStreamCaptureStatusNone, cudaStreamCaptureStatusActive };
enum cudaDeviceAttr { cudaDevAttrMultiProcessorCount };
constexpr unsigned cudaEventDisableTiming = 2;

struct FakeStream {
    unsigned long long id;
    bool capturing;
};
using cudaStream_t = FakeStream*;
using cudaEvent_t = int*;

namespace fake {
inline std::string log;
inline FakeStream* const per_thread = reinterpret_cast<FakeStream*>(2);      // one handle, a stream a thread
inline unsigned long long thread_stream_id = 1000;
inline cudaError_t malloc_result = cudaSuccess;
inline const FakeStream* of(cudaStream_t s) {
    static FakeStream own{0, false};
    if (s != per_thread) return s;
    own.id = thread_stream_id;
    return &own;
}
inline void note(const char* what, cudaStream_t s) { log += what + std::to_string(of(s)->id) + " "; }
}  // namespace fake

inline cudaError_t cudaGetLastError() { return cudaSuccess; }
inline cudaError_t cudaGetDeviceCount(int* n) { *n = 1; return cudaSuccess; }
inline cudaError_t cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
inline cudaError_t cudaSetDevice(int) { return cudaSuccess; }
inline cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) { *v = 152; return cudaSuccess; }
inline cudaError_t cudaMalloc(void** p, size_t n) {
    if (fake::malloc_result == cudaSuccess) *p = std::malloc(n);
    return fake::malloc_result;
}
inline cudaError_t cudaFree(void* p) { std::free(p); return cudaSuccess; }
inline cudaError_t cudaStreamIsCapturing(cudaStream_t s, cudaStreamCaptureStatus* c) {
    *c = fake::of(s)->capturing ? cudaStreamCaptureStatusActive : cudaStreamCaptureStatusNone;
    return cudaSuccess;
}
// (as the real one: not while the stream is capturing)
inline cudaError_t cudaStreamGetId(cudaStream_t s, unsigned long long* id) {
    *id = fake::of(s)->id;
    return fake::of(s)->capturing ? cudaErrorLaunchFailure : cudaSuccess;
}
inline cudaError_t cudaStreamWaitEvent(cudaStream_t s, cudaEvent_t, unsigned) { fake::note("wait", s); return cudaSuccess; }
inline cudaError_t cudaEventCreateWithFlags(cudaEvent_t* e, unsigned) { *e = new int(0); return cudaSuccess; }
inline cudaError_t cudaEventRecord(cudaEvent_t, cudaStream_t s) { fake::note("record", s); return cudaSuccess; }
inline cudaError_t cudaEventDestroy(cudaEvent_t e) { delete e; return cudaSuccess; }
