// hqq_adapters.h -- launch interface of the low-rank adapters of many requests
// (hqq_adapters.hip).  Not part of the public ABI.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace hqq {

constexpr int kMaxAdapterRank = 256;
constexpr int kMaxAdapters = 1024;  // sorted as experts

struct AdapterParams {
  int dtype;                // 0 binary16, 1 bfloat16
  const uint16_t* X;        // M x K
  const uint16_t* A;        // adapters x rank x K
  const uint16_t* B;        // adapters x N x rank
  const int32_t* ids;       // M
  const float* scales;      // adapters
  const void* base;         // M x N (backward: M x K), or null: zeros
  int base_f32;
  int base_slabs;           // above 0: base is that many fp32 slabs, to be added in order
  int64_t base_stride;      // floats of a slab
  void* out;                // Y: M x N (backward dX: M x K)
  int out_f32;
  const uint16_t* dY;       // backward: M x N
  float* dA;                // backward: adapters x rank x K
  float* dB;                // backward: adapters x N x rank
  int64_t M, N, K;
  int rank, adapters;
  void* workspace;
};

// A projection by a quantized weight with adapters, and its gradients: binary16 (dtype 0), base
// null; `q` holds the weight (its X, Y and M are not read).
struct MatmulParams;
int64_t matmul_adapters_workspace_bytes(const MatmulParams& q, const AdapterParams& p);
int64_t matmul_adapters_backward_workspace_bytes(const MatmulParams& q, const AdapterParams& p);
hipError_t launch_matmul_adapters(MatmulParams q, AdapterParams p, int cus, hipStream_t stream);
hipError_t launch_matmul_adapters_backward(const MatmulParams& q, const AdapterParams& p, hipStream_t stream);

int64_t adapters_workspace_bytes(int64_t M, int64_t N, int64_t K, int rank, int adapters);
int64_t adapters_backward_workspace_bytes(int64_t M, int64_t N, int64_t K, int rank, int adapters);
hipError_t launch_adapters(const AdapterParams& p, hipStream_t stream);
hipError_t launch_adapters_backward(const AdapterParams& p, hipStream_t stream);

}  // namespace hqq
