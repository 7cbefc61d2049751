// Host-side services of mla_api.cu for the library's other translation units: the per-device
// context, launch bookkeeping and TMA descriptor encoding.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <utility>

#include "mla.h"

namespace mla {

struct HostDevice {
  int sms;
  unsigned int* status;  // the device's status word
};

// The current device's context (created on first use), or an MLA_ERR_* code.
int host_device(HostDevice* out);
// Records the failing call for mla_error_detail; returns MLA_ERR_CUDA.
int host_cuda_error(cudaError_t e, const char* where);
// Counts `kernels` launches and returns the launch error, if any, as MLA_ERR_CUDA.
int host_launched(int kernels = 1);
bool host_pdl();
uint64_t host_wait_ns();
// MLA_TEST_STALL of the environment, read at each call: 0 unless it is a number from 1 to 299.
int host_stall();
// The checks of mla_dims that neither limit the batch nor look at d_model.
int host_check_dims(const mla_dims* d);
int host_encode(CUtensorMap* m, CUtensorMapDataType dt, const void* base, int rank,
                const uint64_t* dims, const uint64_t* strides_bytes, const uint32_t* box,
                CUtensorMapSwizzle sw);

// A launch with programmatic stream serialisation (see host_pdl); errors by host_launched().
template <typename... KArgs, typename... Args>
void host_launch(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                 Args&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = host_pdl() ? 1 : 0;
  (void)cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

}  // namespace mla
