// hqq_route.h -- launch interface of the token order of experts (hqq_route.hip).  Not part
// of the public ABI.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace hqq {

constexpr int kMaxExperts = 1024;  // one LDS counter per wavefront and expert (64 KB)

// Bytes of the sort's workspace (the blocks' counts; 0 where one block sorts everything).
int64_t route_sort_workspace_bytes(int64_t slots, int experts);

hipError_t launch_route_sort(const int32_t* ids, int64_t slots, int experts, int32_t* order,
                             int32_t* position, int32_t* offsets, int32_t* workspace,
                             hipStream_t stream);

struct RouteRows {
  const void* in;         // rows read: tokens x width (gather), slots x width (combine)
  const void* grad;       // combine backward: tokens x width
  void* out;
  const int32_t* position;
  const float* weights;   // tokens x topk, or null (weights of 1)
  float* dweights;        // combine backward: tokens x topk, or null
  int64_t tokens, width;
  int topk;
};

hipError_t launch_route_gather(const RouteRows& p, int dtype, hipStream_t stream);
hipError_t launch_route_combine(const RouteRows& p, int dtype, hipStream_t stream);
hipError_t launch_route_combine_backward(const RouteRows& p, int dtype, hipStream_t stream);

}  // namespace hqq
