// status.cu -- reading a device status word and taking off what was read.
#include <cuda_runtime.h>

#include <cstdint>

#include "dkv_internal.h"

namespace dkv {
namespace {

// Kernels of other streams may set bits meanwhile: those stay.
__global__ void clear_bits_kernel(int32_t *word, int32_t bits) { atomicAnd(word, ~bits); }

}  // namespace

cudaError_t take_status(int32_t *word, int32_t *bits, cudaStream_t st) {
    int32_t h = 0;
    cudaError_t e = cudaMemcpyAsync(&h, word, sizeof(h), cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e == cudaSuccess && h) {
        clear_bits_kernel<<<1, 1, 0, st>>>(word, h);
        e = cudaGetLastError();
        if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    }
    if (e == cudaSuccess) *bits = h;
    return e;
}

}  // namespace dkv
