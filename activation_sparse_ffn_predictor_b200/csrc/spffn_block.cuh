// What the kernels of the dense half of a batched block (include/spffn_block.h) share on the host side:
// error bits, statuses of CUDA calls, alignment and device checks.
#pragma once
#include <atomic>
#include "spffn_internal.cuh"
#include "../../include/spffn_block.h"

namespace spffn {

// Device error word bits beside those of spffn_internal.cuh.
enum : uint32_t {
    ERR_BATCH_ROWS = 1u << 5,      // paged cache: a sequence's rows do not lie in the call's rows (skipped)
    ERR_BATCH_LEN = 1u << 6,       // paged cache: a length below its new tokens or above the table's reach
    ERR_PAGE_RANGE = 1u << 7,      // paged cache: a page outside the pool (its tokens are left out)
};

// the status of a CUDA call (kept for spffn_last_cuda_error_string), and the SM count of the current device
spffn_status record_cuda(cudaError_t e);
int current_sms();
inline bool aligned_to(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool on_device(int device) {
    int now = -1;
    return cudaGetDevice(&now) == cudaSuccess && now == device;
}
// allow a kernel its dynamic shared memory, once for each device (`ready` is the kernel's own)
template <typename K>
inline cudaError_t allow_smem(K kern, size_t bytes, int device, std::atomic<uint64_t>& ready) {
    const uint64_t bit = 1ull << (device & 63);
    if (device < 64 && (ready.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) ready.fetch_or(bit, std::memory_order_relaxed);
    return e;
}
// read and clear a latched error word at the head of a workspace (synchronises the stream)
inline spffn_status take_device_error(uint32_t* err, uint32_t* code, void* stream) {
    cudaStream_t st = (cudaStream_t)stream;
    uint32_t v = 0;
    cudaError_t e = cudaMemcpyAsync(&v, err, sizeof(v), cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaMemsetAsync(err, 0, sizeof(v), st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e != cudaSuccess) return record_cuda(e);
    if (code) *code = v;
    if (v & (ERR_BARRIER_TIMEOUT | ERR_PIPE_TIMEOUT)) return SPFFN_ERR_TIMEOUT;
    return v ? SPFFN_ERR_DEVICE_CHECK : SPFFN_OK;
}

}  // namespace spffn
