// A plan's status word (mfr_status.cu).
#pragma once

#include <mutex>

#include <cuda_runtime.h>

namespace mfr {

struct StatusWord {
    int* words = nullptr;   // device: [0] the bits that kernels raise, [1] the bits on their way to the host
    int device = -1;
    std::mutex turn;        // held around status_take; with debug_checks around the launch before it as well
};

// Allocates the words on the current device, cleared when it returns.
cudaError_t status_make(StatusWord& w);
void status_free(StatusWord& w);
// Waits for the stream, reads the bits and clears them in one step, nothing
// pending on return.  The caller holds w.turn.
cudaError_t status_take(StatusWord& w, cudaStream_t s, int* bits);

// Whether the stream is being captured, so that nothing may wait for it.
bool being_captured(cudaStream_t s);

// A call's turn with a plan that checks each call (debug_checks): from its launch to
// its reading, so that the bits it finds are its own.  No lock otherwise.
class DebugTurn {
public:
    DebugTurn(StatusWord& w, bool checks) : turn_(w.turn, std::defer_lock) {
        if (checks) turn_.lock();
    }

private:
    std::unique_lock<std::mutex> turn_;
};

}  // namespace mfr
