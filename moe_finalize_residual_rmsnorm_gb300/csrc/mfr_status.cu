// A plan's status word: kernels raise bits in it with atomicOr, from any
// stream, and the host takes them.
//
// Taking is one atomic exchange on the device, so that a bit raised by a kernel
// of another stream is either in this reading or left for the next one.  (A copy
// to the host followed by a clear loses what is raised between the two, and a
// clear that is still pending when the reading returns loses the bits of
// calls made after it.)  The exchanged bits go to a second word, from where the
// host copies them; readers of one plan take turns, so that it is theirs alone.
#include <cuda_runtime.h>

#include "mfr_status.h"

namespace mfr {
namespace {

__global__ void take_status_kernel(int* words) { words[1] = atomicExch(&words[0], 0); }

// Makes a device current and puts the one before back.
struct OnDevice {
    int before = -1;
    cudaError_t error;
    explicit OnDevice(int device) {
        error = cudaGetDevice(&before);
        if (error != cudaSuccess || before == device) before = -1;
        else if ((error = cudaSetDevice(device)) != cudaSuccess) before = -1;
    }
    ~OnDevice() {
        if (before >= 0) cudaSetDevice(before);
    }
};

// Lets this thread free and wait while a graph is being captured elsewhere:
// outside the relaxed mode such calls fail and end that capture.
struct Relaxed {
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;    // then the one before
    const bool changed = cudaThreadExchangeStreamCaptureMode(&mode) == cudaSuccess;
    ~Relaxed() {
        if (changed) cudaThreadExchangeStreamCaptureMode(&mode);
    }
};

}  // namespace

bool being_captured(cudaStream_t s) {
    cudaStreamCaptureStatus st = cudaStreamCaptureStatusNone;
    const cudaError_t e = cudaStreamIsCapturing(s, &st);
    if (e == cudaSuccess) return st != cudaStreamCaptureStatusNone;
    cudaGetLastError();
    // the default stream, while a stream that it is in step with is being
    // captured; any other error is for the calls that follow to report
    return e == cudaErrorStreamCaptureImplicit;
}

cudaError_t status_make(StatusWord& w) {
    cudaFuncAttributes a;     // loads the kernel, which a later capture could not
    cudaError_t e = cudaGetDevice(&w.device);
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, take_status_kernel);
    if (e == cudaSuccess) e = cudaMalloc(&w.words, 2 * sizeof(int));
    if (e == cudaSuccess) e = cudaMemset(w.words, 0, 2 * sizeof(int));
    if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);   // cleared before a run on any stream
    if (e != cudaSuccess) {
        status_free(w);
        cudaGetLastError();   // the caller reports it; nothing later does
    }
    return e;
}

// A plan may go at any time (Python's collector chooses its own), also while a
// graph is being captured, by this thread or another.
void status_free(StatusWord& w) {
    if (!w.words) return;
    const Relaxed relaxed;
    cudaFree(w.words);
    w.words = nullptr;
    cudaGetLastError();
}

cudaError_t status_take(StatusWord& w, cudaStream_t s, int* bits) {
    const OnDevice on(w.device);
    if (on.error != cudaSuccess) return on.error;
    const Relaxed relaxed;
    void* args[] = {&w.words};
    int h = 0;
    cudaError_t e = cudaLaunchKernel(reinterpret_cast<const void*>(take_status_kernel), dim3(1), dim3(1), args, 0, s);
    if (e == cudaSuccess) e = cudaMemcpyAsync(&h, w.words + 1, sizeof(int), cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e == cudaSuccess) *bits = h;
    return e;
}

}  // namespace mfr
