// hqq_experts.hip -- launches of the products of rows sorted by expert with the quantized
// weights of their experts (kernels: hqq_matmul_kernels.h, GROUPED).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "hqq_group_gemm.h"
#include "hqq_internal.h"
#include "hqq_matmul.h"
#include "hqq_matmul_kernels.h"
#include "hqq_tiles.h"

namespace hqq {
namespace {

bool skinny_aligned(const MatmulParams& P) {
  const bool aligned16 = ((reinterpret_cast<uintptr_t>(P.scale16) | reinterpret_cast<uintptr_t>(P.zero16)) & 15) == 0;
  return P.nbits != 3 && P.K % 256 == 0 && aligned16 && P.group_shift >= 5 && P.group_shift <= 7 &&
         P.N * (P.K >> P.group_shift) % 8 == 0;  // every expert's s and z too
}

template <int NB, int R>
void launch_gemv(const MatmulParams& P, hipStream_t st) {
  constexpr int kRowsPerBlock = R * (kBlock / kWave);
  const dim3 grid((unsigned)((P.N + kRowsPerBlock - 1) / kRowsPerBlock), (unsigned)P.M), block(kBlock);
  if (P.group_size == 16) hipLaunchKernelGGL((hqq_gemv_packed_kernel<NB, 1, R, true, true>), grid, block, 0, st, P);
  else hipLaunchKernelGGL((hqq_gemv_packed_kernel<NB, 1, R, false, true>), grid, block, 0, st, P);
}

template <int NB, int MT, int NW>
void launch_skinny_nw(const MatmulParams& P, hipStream_t st) {
  const dim3 grid((unsigned)((P.N + 16 * NW - 1) / (16 * NW)), (unsigned)max_row_tiles(P.M, P.experts, 16 * MT));
  if constexpr (NB != 3) {
    if (skinny_aligned(P)) {
      const dim3 block(kSkinnyWaves2 * kWave);
      switch (P.group_shift) {
        case 5: hipLaunchKernelGGL((hqq_skinny_kernel<NB, MT, NW, 5, true>), grid, block, 0, st, P); return;
        case 6: hipLaunchKernelGGL((hqq_skinny_kernel<NB, MT, NW, 6, true>), grid, block, 0, st, P); return;
        default: hipLaunchKernelGGL((hqq_skinny_kernel<NB, MT, NW, 7, true>), grid, block, 0, st, P); return;
      }
    }
  }
  const dim3 block(kSkinnyWaves * kWave);
  hipLaunchKernelGGL((hqq_skinny_general_kernel<NB, MT, NW, true>), grid, block, 0, st, P);
}

template <int NB, int MT>
void launch_skinny(const MatmulParams& P, hipStream_t st) {
  if (P.N >= 4096) launch_skinny_nw<NB, MT, 2>(P, st);  // 32 weight rows a block, as for one weight
  else launch_skinny_nw<NB, MT, 1>(P, st);
}

hipError_t launch_tiles(const MatmulParams& P, hipStream_t st) {
  GroupGemmParams g = {};
  g.X = P.X;
  g.packed = P.packed;
  g.scale16 = P.scale16;
  g.zero16 = P.zero16;
  g.Y = P.Y;
  g.M = P.M;
  g.N = P.N;
  g.K = P.K;
  g.nbits = P.nbits;
  g.group_shift = P.group_shift;
  g.out_f32 = P.out_f32;
  g.offsets = P.offsets;
  g.order = P.order;
  g.groups = P.experts;
  g.topk = P.topk;
  g.slabs = P.part;
  return launch_group_gemm(g, st);
}

template <int NB>
hipError_t launch_nb(const MatmulParams& P, hipStream_t st) {
  if constexpr (NB != 3) {
    // few rows: a row mostly has its expert to itself, and a wavefront takes one row and 1, 2
    // or 4 weight rows (enough wavefronts to fill the chip first)
    if (P.M <= kExpertGemvMaxRows) {
      if (P.N * P.M >= 8192) launch_gemv<NB, 4>(P, st);
      else if (P.N * P.M >= 4096) launch_gemv<NB, 2>(P, st);
      else launch_gemv<NB, 1>(P, st);
      return hipGetLastError();
    }
  }
  const int64_t mean = P.M / P.experts;  // rows an expert
  if (mean > kExpertSkinnyMaxMean) return launch_tiles(P, st);
  // One 16-row tile a block while a second walk over an expert's codes costs less than the registers
  // and LDS of two tiles: 8 experts of 4096 x 11008, mean 12 / 16 / 24 rows, one tile against two:
  // 75 / 97 / 111 and 79 / 80 / 94 us (2 bits), 69 / 89 / 102 and 95 / 100 / 122 us (4 bits).
  constexpr int64_t kOneTile = NB == 2 ? 12 : NB == 3 ? 8 : 24;
  if (mean <= kOneTile) launch_skinny<NB, 1>(P, st);
  else if (mean <= 24) launch_skinny<NB, 2>(P, st);
  else launch_skinny<NB, 4>(P, st);
  return hipGetLastError();
}

}  // namespace

int64_t matmul_experts_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t experts) {
  if (M <= kExpertGemvMaxRows || M / experts <= kExpertSkinnyMaxMean) return 0;
  return group_gemm_workspace_bytes(M, N, K, experts, false);
}

hipError_t launch_matmul_experts(MatmulParams prm, hipStream_t stream) {
  prm.ksplit = 1;
  prm.slab = 0;
  switch (prm.nbits) {
    case 2: return launch_nb<2>(prm, stream);
    case 3: return launch_nb<3>(prm, stream);
    case 4: return launch_nb<4>(prm, stream);
    case 8: return launch_nb<8>(prm, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace hqq
