// blocks.h -- device memory that the library owns and that grows on demand
// (host code only).
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>

namespace rc {

// A block and the smaller ones it replaced.  Those stay allocated until
// release(): a captured graph, or a launch that another thread is about to
// make, may hold their address.  Sizes at least double, so together they are
// no larger than the block in use.
struct Block {
    static constexpr int kMost = 40;     // doubling from 1 MiB reaches any GPU's memory long before
    void *ptr = nullptr;
    size_t bytes = 0;
    void *old[kMost] = {};
    int olds = 0;
};

// Makes the block at least `need` bytes long; its contents are arbitrary
// whenever b.ptr changes.  Allocating is no stream operation, so it is done in
// the capture mode that lets it pass while this or another thread captures.
inline cudaError_t grow(Block &b, size_t need)
{
    if (b.bytes >= need) return cudaSuccess;
    if (b.ptr && b.olds == Block::kMost) return cudaErrorMemoryAllocation;
    const size_t unit = (size_t)1 << 20;
    const size_t least = (need + unit - 1) / unit * unit;
    size_t want = least > 2 * b.bytes ? least : 2 * b.bytes;
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    cudaError_t e = cudaThreadExchangeStreamCaptureMode(&mode);
    if (e != cudaSuccess) return e;
    void *p = nullptr;
    e = cudaMalloc(&p, want);
    if (e != cudaSuccess && want > least) {
        (void)cudaGetLastError();
        want = least;
        e = cudaMalloc(&p, want);
    }
    const cudaError_t back = cudaThreadExchangeStreamCaptureMode(&mode);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return e;
    }
    if (b.ptr) b.old[b.olds++] = b.ptr;
    b.ptr = p;
    b.bytes = want;
    return back;
}

// Frees the block and those it replaced; no call may be using them.
inline void release(Block &b)
{
    for (int i = 0; i < b.olds; ++i) cudaFree(b.old[i]);
    if (b.ptr) cudaFree(b.ptr);
    b = Block{};
}

} // namespace rc
