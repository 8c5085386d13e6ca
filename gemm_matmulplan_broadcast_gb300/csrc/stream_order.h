// The order of a plan's calls that use device memory of its own, across
// streams.  Host only.
#pragma once

#include <cuda_runtime.h>

namespace olc {

// A call on another stream than the last such one waits for it on the GPU (an
// event, created at the first use), so calls from several streams follow one
// another on that memory; on one stream, stream order does it.  Streams are told
// apart by their identity: a handle may name another stream later (the default
// stream of each host thread, a stream made after one was destroyed).  While a
// stream is capturing a graph nothing is recorded or waited for: ordering
// captured work is the graph's.  All zeros: no call yet.
struct StreamOrder {
    cudaEvent_t event;
    unsigned long long stream;      // identity of the last call's
    int event_live;

    cudaError_t before_use(cudaStream_t s) {
        if (!event_live) return cudaSuccess;
        cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
        cudaError_t e = cudaStreamIsCapturing(s, &cs);
        if (e != cudaSuccess) return e;
        if (cs != cudaStreamCaptureStatusNone) return cudaSuccess;
        unsigned long long id = 0;      // (asking would break a capture)
        e = cudaStreamGetId(s, &id);
        if (e != cudaSuccess || id == stream) return e;
        return cudaStreamWaitEvent(s, event, 0);
    }

    cudaError_t after_use(cudaStream_t s) {
        cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
        cudaError_t e = cudaStreamIsCapturing(s, &cs);
        if (e != cudaSuccess) return e;
        if (cs != cudaStreamCaptureStatusNone) return cudaSuccess;
        if (!event) {
            e = cudaEventCreateWithFlags(&event, cudaEventDisableTiming);
            if (e != cudaSuccess) {
                event = nullptr;
                return e;
            }
        }
        unsigned long long id = 0;
        e = cudaStreamGetId(s, &id);
        if (e == cudaSuccess) e = cudaEventRecord(event, s);
        if (e != cudaSuccess) return e;
        stream = id;
        event_live = 1;
        return cudaSuccess;
    }

    // f enqueues the call's work, and all that it did enqueue is recorded: work
    // that went ahead of a failure uses the memory like any other.  The first
    // error.
    template <typename F>
    cudaError_t use(cudaStream_t s, F&& f) {
        const cudaError_t before = before_use(s);
        if (before != cudaSuccess) return before;
        const cudaError_t e = f();
        const cudaError_t after = after_use(s);
        return e != cudaSuccess ? e : after;
    }
};

}  // namespace olc
