// hqq_matmul_t.h -- launch interface of the gradient of the product with a quantized weight
// (hqq_matmul_t.hip).  Not part of the public ABI.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "hqq_low_tile.h"

namespace hqq {

struct MatmulTParams {
  const uint16_t* dY;       // M x N binary16
  const uint8_t* packed;    // experts x N x K codes
  const uint16_t* scale16;
  const uint16_t* zero16;
  void* dX;                 // M x K, binary16 or fp32
  int64_t M, N, K;
  int nbits, group_size, group_shift;
  int out_f32;
  const int32_t* offsets;   // rows sorted by expert: first row of each; null: one weight
  int experts;
  LowRank low;              // adapters (low.low set, offsets null): rows order[i] of dY and dX
  float* slabs;             // matmul_t_workspace_bytes(...) bytes
  int xcd_slabs;            // slabs of an XCD (set by the launcher)
};

int64_t matmul_t_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t experts);
hipError_t launch_matmul_t(MatmulTParams prm, hipStream_t stream);

}  // namespace hqq
