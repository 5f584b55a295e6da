// hqq_matmul.hip -- launches of the product with one quantized weight, Y = X Q^-1(W_q)^T
// (kernels: hqq_matmul_kernels.h).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "hqq_internal.h"
#include "hqq_matmul.h"
#include "hqq_matmul_kernels.h"

namespace hqq {
namespace {

// The aligned skinny kernel applies: byte-aligned codes, groups of 32-128, K a multiple
// of 256, 16-byte aligned s and z.
bool skinny_aligned(const MatmulParams& P) {
  const bool aligned16 = ((reinterpret_cast<uintptr_t>(P.scale16) | reinterpret_cast<uintptr_t>(P.zero16)) & 15) == 0;
  return P.nbits != 3 && P.K % 256 == 0 && aligned16 && P.group_shift >= 5 && P.group_shift <= 7;
}

// Split-K geometry of the aligned skinny path, from the shapes and the code width alone
// (results do not depend on the device): 16 NW weight rows per wavefront (NW = 2 only for
// 8-bit codes from 4096 rows), and K split so that a launch has about kSplitTargetWaves
// wavefronts where K allows (two per SIMD; with 8-wavefront blocks, 4096 split the
// 28672-row matrices in two and were 1-4% slower at M = 32-64 than no split there).
constexpr int kSplitTargetWaves = 2048;
struct SplitGeom {
  int waves, nw, ksplit;
  int64_t row_blocks;
};
SplitGeom split_geometry(int64_t N, int64_t K, int nbits) {
  SplitGeom g;
  g.waves = nbits == 8 ? split_waves<8>() : split_waves<2>();
  g.nw = nbits == 8 && N >= 4096 ? 2 : 1;
  const int64_t rows = (int64_t)g.waves * 16 * g.nw;
  g.row_blocks = (N + rows - 1) / rows;
  const int64_t target = kSplitTargetWaves / g.waves;  // blocks
  int64_t ks = (target + g.row_blocks / 2) / g.row_blocks;
  const int64_t nkb = K >> 8;
  if (ks > nkb) ks = nkb;
  g.ksplit = ks < 1 ? 1 : (int)ks;
  return g;
}

// The split-K path applies (s and z alignment aside, checked at the call): 17 to 64 rows
// of X (up to 16 the aligned skinny kernel, which needs no workspace, is as fast).
bool splitk_shapes(int64_t M, int64_t K, int nbits, int group_size) {
  return nbits != 3 && K % 256 == 0 && group_size >= 32 && group_size <= 128 &&
         M > kSplitMinRows && M <= kSkinnyMaxRows;
}

template <int NB, int MT, int NW>
void launch_splitk_nw(const MatmulParams& P, dim3 grid, hipStream_t st) {
  const dim3 block(split_waves<NB>() * kWave);
  constexpr int PD = split_prefetch<NB>();
  switch (P.group_shift) {
    case 5: hipLaunchKernelGGL((hqq_splitk_kernel<NB, MT, NW, 5, PD>), grid, block, 0, st, P); return;
    case 6: hipLaunchKernelGGL((hqq_splitk_kernel<NB, MT, NW, 6, PD>), grid, block, 0, st, P); return;
    default: hipLaunchKernelGGL((hqq_splitk_kernel<NB, MT, NW, 7, PD>), grid, block, 0, st, P); return;
  }
}

template <int NB, int MT>
void launch_splitk(MatmulParams P, hipStream_t st) {
  const SplitGeom g = split_geometry(P.N, P.K, NB);
  P.ksplit = g.ksplit;
  P.slab = (P.M * P.N + 3) & ~(int64_t)3;
  const dim3 grid((unsigned)g.row_blocks, (unsigned)g.ksplit);
  if constexpr (NB == 8) {
    if (g.nw == 2) {
      launch_splitk_nw<NB, MT, 2>(P, grid, st);
    } else {
      launch_splitk_nw<NB, MT, 1>(P, grid, st);
    }
  } else {
    launch_splitk_nw<NB, MT, 1>(P, grid, st);
  }
  if (g.ksplit > 1 && P.Y) {  // (without Y the slabs are what is wanted)
    int64_t blocks = (P.M * P.N + 4 * kBlock - 1) / (4 * kBlock);
    if (blocks > 4096) blocks = 4096;
    hipLaunchKernelGGL(hqq_splitk_reduce_kernel, dim3((unsigned)blocks), dim3(kBlock), 0, st, P);
  }
}

template <int NB, int MT, int NW>
void launch_skinny_nw(const MatmulParams& P, dim3 grid, hipStream_t st) {
  const dim3 block(kSkinnyWaves * kWave), block2(kSkinnyWaves2 * kWave);
  if constexpr (NB != 3) {
    if (skinny_aligned(P)) {
      switch (P.group_shift) {
        case 5: hipLaunchKernelGGL((hqq_skinny_kernel<NB, MT, NW, 5>), grid, block2, 0, st, P); return;
        case 6: hipLaunchKernelGGL((hqq_skinny_kernel<NB, MT, NW, 6>), grid, block2, 0, st, P); return;
        default: hipLaunchKernelGGL((hqq_skinny_kernel<NB, MT, NW, 7>), grid, block2, 0, st, P); return;
      }
    }
  }
  hipLaunchKernelGGL((hqq_skinny_general_kernel<NB, MT, NW>), grid, block, 0, st, P);
}

template <int NB, int MT>
void launch_skinny(const MatmulParams& P, hipStream_t st) {
  if (P.N >= 4096)  // 32 weight rows per block where there are enough rows
    launch_skinny_nw<NB, MT, 2>(P, dim3((unsigned)((P.N + 31) / 32)), st);
  else
    launch_skinny_nw<NB, MT, 1>(P, dim3((unsigned)((P.N + 15) / 16)), st);
}

template <int NB>
hipError_t launch_nb(const MatmulParams& P, int cus, hipStream_t st) {
  // the aligned skinny kernel costs about the same for 3-16 rows as the per-row one for 3
  const int64_t gemv_max = skinny_aligned(P) ? kGemvAlignedMaxRows : kGemvMaxRows;
  if constexpr (NB != 3) {  // packed binary16 codes (3-bit codes straddle bytes)
    if (P.M <= gemv_max) {
      // rows per wavefront: enough wavefronts to fill the chip (>= 2048) with as many
      // rows sharing each chunk of X as that allows
      if (P.N >= 8192) return launch_gemv_packed<NB, 4>(P, st);
      if (P.N >= 4096) return launch_gemv_packed<NB, 2>(P, st);
      return launch_gemv_packed<NB, 1>(P, st);
    }
  }
  if constexpr (NB != 3) {
    if (skinny_aligned(P) && splitk_shapes(P.M, P.K, NB, P.group_size)) {
      if (P.M <= 32) launch_splitk<NB, 2>(P, st);
      else launch_splitk<NB, 4>(P, st);
      return hipGetLastError();
    }
  }
  if (P.M > gemv_max && P.M <= kSkinnyMaxRows) {
    if (P.M <= 16) launch_skinny<NB, 1>(P, st);
    else if (P.M <= 32) launch_skinny<NB, 2>(P, st);
    else launch_skinny<NB, 4>(P, st);
    return hipGetLastError();
  }
  if (P.M <= kGemvMaxRows) {
    int64_t blocks = (P.N + kBlock / kWave - 1) / (kBlock / kWave);  // a wavefront per row
    const int64_t cap = (int64_t)cus * 32;
    if (blocks > cap) blocks = cap;
    const dim3 grid((unsigned)blocks), block(kBlock);
    if (P.M <= 1) hipLaunchKernelGGL((hqq_gemv_kernel<NB, 1>), grid, block, 0, st, P);
    else if (P.M <= 2) hipLaunchKernelGGL((hqq_gemv_kernel<NB, 2>), grid, block, 0, st, P);
    else if (P.M <= 4) hipLaunchKernelGGL((hqq_gemv_kernel<NB, 4>), grid, block, 0, st, P);
    else hipLaunchKernelGGL((hqq_gemv_kernel<NB, 8>), grid, block, 0, st, P);
  } else {
    // 256 x 128 tiles of 8 wavefronts from 512 rows (each weight tile is dequantized once
    // per 256 rows of X: half the decode per MFMA of 128 x 128 tiles), else 128 x 128 (4
    // wavefronts: twice the blocks for a few hundred rows); both 64 x 64 per wavefront, 2
    // wavefronts per SIMD
    if (P.M >= 512) {
      const dim3 grid((unsigned)((P.N + 127) / 128), (unsigned)((P.M + 255) / 256));
      hipLaunchKernelGGL((hqq_gemm_kernel<NB, 4, 2, 2>), grid, dim3(8 * kWave), 0, st, P);
    } else {
      const dim3 grid((unsigned)((P.N + 127) / 128), (unsigned)((P.M + 127) / 128));
      hipLaunchKernelGGL((hqq_gemm_kernel<NB, 2, 2, 2>), grid, dim3(4 * kWave), 0, st, P);
    }
  }
  return hipGetLastError();
}

}  // namespace

int64_t matmul_workspace_bytes(int64_t M, int64_t N, int64_t K, int nbits, int group_size) {
  if (!splitk_shapes(M, K, nbits, group_size) || N <= 0) return 0;
  const SplitGeom g = split_geometry(N, K, nbits);
  if (g.ksplit <= 1) return 0;
  return (int64_t)g.ksplit * ((M * N + 3) & ~(int64_t)3) * (int64_t)sizeof(float);
}

bool matmul_adds_low(const MatmulParams& prm) {
  return prm.nbits != 3 && prm.M <= kGemvAlignedMaxRows && prm.K > 0;
}

hipError_t launch_matmul_base(MatmulParams prm, int cus, MatmulBase* base, hipStream_t stream) {
  *base = {0, 0};
  if (prm.nbits != 3 && skinny_aligned(prm) && splitk_shapes(prm.M, prm.K, prm.nbits, prm.group_size)) {
    const SplitGeom g = split_geometry(prm.N, prm.K, prm.nbits);
    if (g.ksplit > 1) {
      *base = {g.ksplit, (prm.M * prm.N + 3) & ~(int64_t)3};
      prm.Y = nullptr;
    }
  }
  prm.out_f32 = 1;
  return launch_matmul(prm, cus, stream);
}

hipError_t launch_matmul(MatmulParams prm, int cus, hipStream_t stream) {
  prm.ksplit = 1;
  prm.slab = 0;
  switch (prm.nbits) {
    case 2: return launch_nb<2>(prm, cus, stream);
    case 3: return launch_nb<3>(prm, cus, stream);
    case 4: return launch_nb<4>(prm, cus, stream);
    case 8: return launch_nb<8>(prm, cus, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace hqq
