// hqq_group_gemm.h -- launch interface of the tiled products of sorted rows with quantized
// weights (hqq_group_gemm.hip).  Not part of the public ABI.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "hqq_low_tile.h"

namespace hqq {

struct GroupGemmParams {
  const uint16_t* X;        // binary16 rows of K, 16-byte aligned
  const uint8_t* packed;
  const uint16_t* scale16;
  const uint16_t* zero16;
  void* Y;                  // rows of N, binary16 or fp32
  int64_t M, N, K;          // M sorted rows
  int nbits, group_shift;
  int out_f32;
  const int32_t* order;     // experts: null, or row i is X[order[i] / topk]; adapters: row of X and Y
  const int32_t* offsets;   // first sorted row of every group, groups + 1 values
  int groups, topk;
  LowRank low;              // adapters (low.low set): all rows multiply with the one weight
  float* slabs;             // group_gemm_workspace_bytes(...) bytes
  int xcd_slabs;            // slabs of an XCD (set by the launcher)
};

int64_t group_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t groups, bool adapters);

// experts x N x K weights (p.low.low null), or one weight and adapters.
hipError_t launch_group_gemm(GroupGemmParams p, hipStream_t stream);

}  // namespace hqq
