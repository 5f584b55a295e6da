// hqq_matmul.h -- launch interface of the product with a quantized weight
// (hqq_matmul.hip).  Not part of the public ABI.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace hqq {

struct MatmulParams {
  const uint16_t* X;        // M x K binary16 activations, row-major
  const uint8_t* packed;    // N x K codes, LSB-first bitstream over row-major elements
  const uint16_t* scale16;  // N x K/g binary16 s
  const uint16_t* zero16;   // N x K/g binary16 z
  void* Y;                  // M x N, binary16 or fp32
  int64_t M, N, K;
  int nbits, group_size;
  int group_shift;          // log2(group_size)
  int out_f32;
  float* part;              // split-K partial slabs (caller's workspace), or null
  int64_t slab;             // floats per partial slab: M*N rounded up to a multiple of 4
  int ksplit;               // splits of K (1: no partials)
  // products of many experts (GROUPED kernels): M rows sorted by expert, experts x N x K codes
  const int32_t* offsets = nullptr;  // first row of every expert, experts + 1 values
  const int32_t* order = nullptr;    // null: X holds the sorted rows; else row i is X[order[i] / topk]
  int experts = 0, topk = 1;
  // adapters added by the per-row kernel (LOW): part[split][m][r] sums to A x of row m
  const float* low = nullptr;        // splits x M x rank, or null
  int low_splits = 0, rank = 0, adapters = 0;
  const uint16_t* factor = nullptr;  // adapters x N x rank binary16
  const int32_t* ids = nullptr;
  const float* scales = nullptr;
};

// Rows of X up to which the wavefront-per-row kernel is used (kGemvAlignedMaxRows where
// the aligned skinny kernel applies: 2-, 4-, 8-bit codes, groups of 32-128, K a multiple
// of 256, 16-byte aligned s and z), and up to which a skinny matrix-core kernel is used
// above that (then the tiled matrix-core kernel).
constexpr int kGemvMaxRows = 8;
constexpr int kGemvAlignedMaxRows = 2;
constexpr int kSkinnyMaxRows = 64;
constexpr int kSplitMinRows = 16;  // above this (and up to kSkinnyMaxRows) K is split
// Sorted rows of many experts up to which every row is a product of its own.
constexpr int kExpertGemvMaxRows = 8;
// Mean rows of an expert up to which blocks split K over their wavefronts (above: tiles).
constexpr int kExpertSkinnyMaxMean = 48;

// Bytes of workspace the product needs for these shapes (the split-K partial slabs of
// the skinny path; 0 when the path writes Y directly).  Depends on the shapes only.
int64_t matmul_workspace_bytes(int64_t M, int64_t N, int64_t K, int nbits, int group_size);

// `prm.part` must hold matmul_workspace_bytes(...) bytes where that is not 0.
hipError_t launch_matmul(MatmulParams prm, int cus, hipStream_t stream);

// The product as the base of something added to it, in fp32: either `slabs` partial slabs of
// `stride` floats in prm.part, to be added in order, or prm.Y (fp32) and slabs = 0.
struct MatmulBase {
  int slabs;
  int64_t stride;
};
hipError_t launch_matmul_base(MatmulParams prm, int cus, MatmulBase* base, hipStream_t stream);

// Whether the per-row kernel takes the product and may add adapters itself (prm.low set).
bool matmul_adds_low(const MatmulParams& prm);

// The products of sorted rows with their experts' weights: prm.offsets set.
int64_t matmul_experts_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t experts);
// `prm.part` must hold matmul_experts_workspace_bytes(...) bytes where that is not 0.
hipError_t launch_matmul_experts(MatmulParams prm, hipStream_t stream);

}  // namespace hqq
