// Host helpers shared by the library's translation units (defined in gka_api.cu).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace gka {

// Brackets a launch with a pair of events while the launch profiler is on.
struct ProfScope {
    int kernel;
    cudaStream_t s;
    cudaEvent_t start = nullptr;
    ProfScope(int k, cudaStream_t st);
    ~ProfScope();
};

// Keeps the CUDA error for gka_last_cuda_error() and returns GKA_ERR_CUDA.
int cuda_fail(cudaError_t e);
// GKA_OK, or GKA_ERR_CUDA with the error of the launch just made.
int check_launch();

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
inline size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }
inline bool supported_d(int D) { return D == 32 || D == 64 || D == 128; }

// Opts a kernel into `bytes` of dynamic shared memory (beyond the 48 KiB
// default, which also counts the kernel's static shared memory).  Remembered
// per (kernel, device) so the attribute call happens once.
cudaError_t set_smem_bytes(const void *kernel, size_t bytes);
template <typename K>
cudaError_t set_smem(K kernel, size_t bytes) {
    return set_smem_bytes(reinterpret_cast<const void *>(kernel), bytes);
}

// cuTensorMapEncodeTiled through the runtime's driver entry point (no -lcuda).
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

// Device address of the flag a kernel raises when a bounded wait gives up.
int timeout_flag_ptr(int **ptr);

}  // namespace gka
