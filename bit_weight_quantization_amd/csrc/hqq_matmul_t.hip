// hqq_matmul_t.hip -- gfx950 kernels of the gradient of the product with a quantized weight,
// dX = dY Q^-1(W_q), for one weight or for rows sorted by expert with a weight each.
//
// dX[m][k] = sum over n of dY[m][n] s[n][k/g] (q[n][k] - z[n][k/g]): the contraction runs over
// the weight's rows, while codes are packed along k.  The weight tile is dequantized once per
// block into LDS as it is stored (rows n, binary16, as in the forward kernels), and the matrix
// operand, which needs 8 consecutive n of one k in a lane, is read with gfx950's transposing LDS
// read (ds_read_b64_tr_b16: of each 16 lanes' 4 x 16 block of halves lane i gets column i).
// Bound by the matrix cores for many rows; for few, by the latency of one block's walk over n,
// which is then split over blocks and joined in a fixed order.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "hqq_codes.h"
#include "hqq_internal.h"
#include "hqq_matmul_t.h"
#include "hqq_tiles.h"

namespace hqq {
namespace {

constexpr int kTN = 64;              // n per step
constexpr int kTK = 128;             // columns (k) of a tile
constexpr int kTRowA = kTN + 8;      // halves per LDS row of dY: rows 4 banks apart
// halves per LDS row of the weight: 320 bytes, so that the four rows of a transposing read
// start 16 banks apart (of 64) and its 64-byte pieces cover the banks once
constexpr int kTRowB = kTK + 32;

typedef short short4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) short4_t lds_short4;

// 8 binary16 from p (2-byte aligned), of which the first `valid` exist; the others are zero.
__device__ __forceinline__ uint4 load8_part(const uint16_t* p, int64_t valid) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = 2 * i < valid ? p[2 * i] : 0u;
    const uint32_t hi = 2 * i + 1 < valid ? p[2 * i + 1] : 0u;
    w[i] = lo | (hi << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 load8(const uint16_t* p) {  // 2-byte aligned, one 16-byte load
  uint4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}

// (64 WM) x 128 output tile per block of 2 WM wavefronts (64 x 64 each: 2 x 2 tiles of
// v_mfma_f32_32x32x16_f16), n in steps of 64.  Thread t stages row t / 2 of dY (32 values) and
// CB codes of one weight row per step.  Pipelined as the forward kernel: loads two steps
// ahead in registers, LDS double-buffered, one LDS-only barrier per step.
template <int NB, int WM, bool GROUPED>
__global__ __launch_bounds__(2 * WM * kWave) __attribute__((amdgpu_waves_per_eu(2)))
void hqq_matmul_t_kernel(const MatmulTParams P) {
  constexpr int T = 2 * WM * kWave, BM = 64 * WM;
  constexpr int CB = kTN * kTK / T;  // codes per thread and step
  static_assert(CB == 16 || CB == 32, "16 or 32 codes of a weight row per thread");
  constexpr int BP = kTK / CB;       // threads per weight row
  constexpr int CW = CB == 32 ? NB : Codes16<NB>::kWords;
  __shared__ __align__(16) _Float16 As[2][BM][kTRowA];
  __shared__ __align__(16) _Float16 Bs[2][kTN][kTRowB];
  const int tid = threadIdx.x, wid = tid / kWave, lane = tid & (kWave - 1);
  const int wm = wid >> 1, wn = wid & 1;

  int64_t row0 = (int64_t)blockIdx.y * BM;
  int64_t rows = P.M - row0 < BM ? P.M - row0 : BM;
  int64_t w0 = 0;                    // first weight row of the expert
  int64_t N = P.N;
  if constexpr (GROUPED) {
    const RowTile t = find_row_tile(P.offsets, P.experts, P.M, BM, blockIdx.y);
    if (t.rows <= 0) return;
    row0 = t.row0;
    rows = t.rows;
    w0 = (int64_t)t.group * P.N;
    if (t.group == P.experts) N = 0, w0 = 0;  // rows of no expert: zeros
  }
  const int64_t k0 = (int64_t)blockIdx.x * kTK;
  const int64_t steps = (N + kTN - 1) / kTN;
  const int64_t st0 = steps * blockIdx.z / P.nsplit, st1 = steps * (blockIdx.z + 1) / P.nsplit;

  const int xr = tid >> 1, xh = tid & 1;
  const uint16_t* yrow = P.dY + (row0 + (xr < rows ? xr : rows - 1)) * P.N;
  const int br = tid / BP, bp = tid % BP;
  const int64_t kc = k0 + CB * bp < P.K ? k0 + CB * bp : 0;  // (columns past K are not stored)
  const int64_t row_bytes = (P.K >> 3) * NB, gpr = P.K >> P.group_shift;
  const int g2 = P.group_size == 16 ? 1 : 0;

  uint4 ar[2][4];
  uint32_t cw[2][CW];
  uint32_t s16[2][2], z16[2][2];
  auto load_global = [&](auto st_const, int64_t step) {
    constexpr int S = decltype(st_const)::value;
    const int64_t nb = step * kTN;
    const int64_t ea = nb + 32 * xh;
    if (nb + kTN <= N) {
#pragma unroll
      for (int i = 0; i < 4; ++i) ar[S][i] = load8(yrow + ea + 8 * i);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) ar[S][i] = load8_part(yrow + ea + 8 * i, N - ea - 8 * i);
    }
    const int64_t n = nb + br < N ? nb + br : N - 1;
    const uint8_t* cp = P.packed + (w0 + n) * row_bytes;
    if constexpr (CB == 32) load_codes32<NB>(cp + (kc >> 5) * (4 * NB), cw[S]);
    else load_codes16<NB>(cp + (kc >> 4) * (2 * NB), cw[S]);
    const int64_t g0 = (w0 + n) * gpr + (kc >> P.group_shift);
    s16[S][0] = P.scale16[g0];
    z16[S][0] = P.zero16[g0];
    if constexpr (CB == 32) {
      s16[S][1] = P.scale16[g0 + g2];
      z16[S][1] = P.zero16[g0 + g2];
    }
  };
  auto dequant_b = [&](auto st_const, int64_t step, uint4 (&bv)[CB / 8]) {
    constexpr int S = decltype(st_const)::value;
    const bool ok = step * kTN + br < N;  // rows past N enter as zeros
    const float s0 = ok ? h2f(s16[S][0]) : 0.f;
    const float sz0 = ok ? s0 * h2f(z16[S][0]) : 0.f;
    if constexpr (CB == 32) {
      const float s1 = ok ? h2f(s16[S][1]) : 0.f;
      const float sz1 = ok ? s1 * h2f(z16[S][1]) : 0.f;
      dequant32<NB>(cw[S], s0, sz0, s1, sz1, bv);
    } else {
      dequant16<NB>(cw[S], s0, sz0, bv);
    }
  };
  auto write_lds = [&](auto st_const, int buf, const uint4 (&bv)[CB / 8]) {
    constexpr int S = decltype(st_const)::value;
    uint4* ad = reinterpret_cast<uint4*>(&As[buf][xr][32 * xh]);
#pragma unroll
    for (int i = 0; i < 4; ++i) ad[i] = ar[S][i];
    uint4* bd = reinterpret_cast<uint4*>(&Bs[buf][br][CB * bp]);
#pragma unroll
    for (int i = 0; i < CB / 8; ++i) bd[i] = bv[i];
  };

  float16_t acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;

  // the lane's place in a transposing read: group lane / 16 covers columns 16 (group & 1) .. + 16
  // of rows 8 (group / 2) .. + 4 (a second read: + 4 .. + 8); lane i of it supplies row i / 4,
  // columns 4 (i % 4) .. + 4
  const int tr_row = 8 * (lane >> 5) + ((lane & 15) >> 2);
  const int tr_col = 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
  auto mfma_step = [&](int buf) {
#pragma unroll
    for (int ks = 0; ks < kTN / 16; ++ks) {
      half8_t af[2], bf[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        af[i] = *reinterpret_cast<const half8_t*>(&As[buf][wm * 64 + i * 32 + (lane & 31)][ks * 16 + (lane >> 5) * 8]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const _Float16* src = &Bs[buf][ks * 16 + tr_row][wn * 64 + j * 32 + tr_col];
        const short4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4*)src);
        const short4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4*)(src + 4 * kTRowB));
        bf[j] = __builtin_bit_cast(half8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(af[i], bf[j], acc[i][j], 0, 0, 0);
    }
  };
  auto step = [&](auto st_const, int64_t c) {
    constexpr int S = decltype(st_const)::value;
    constexpr std::integral_constant<int, S ^ 1> other{};
    load_global(st_const, c + 2 < st1 ? c + 2 : st0);
    uint4 bv[CB / 8];
    dequant_b(other, c + 1 < st1 ? c + 1 : st0, bv);
    mfma_step(S);
    write_lds(other, S ^ 1, bv);  // (after the last step: unused)
    lds_barrier();
  };

  if (st0 < st1) {
    constexpr std::integral_constant<int, 0> s0{};
    constexpr std::integral_constant<int, 1> s1{};
    load_global(s0, st0);
    load_global(s1, st0 + 1 < st1 ? st0 + 1 : st0);
    uint4 bv[CB / 8];
    dequant_b(s0, st0, bv);
    write_lds(s0, 0, bv);
    lds_barrier();
    for (int64_t c = st0; c < st1; c += 2) {
      step(s0, c);
      if (c + 1 >= st1) break;
      step(s1, c + 1);
    }
  }

  float* part = P.nsplit > 1 ? P.part + blockIdx.z * (P.M * P.K) : nullptr;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int64_t k = k0 + wn * 64 + j * 32 + (lane & 31);
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int64_t m = wm * 64 + i * 32 + 8 * (v >> 2) + 4 * (lane >> 5) + (v & 3);
        if (m < rows && k < P.K) {
          const int64_t at = (row0 + m) * P.K + k;
          if (part) part[at] = acc[i][j][v];
          else if (P.out_f32) static_cast<float*>(P.dX)[at] = acc[i][j][v];
          else static_cast<_Float16*>(P.dX)[at] = (_Float16)acc[i][j][v];
        }
      }
    }
  }
}

// dX = the sum of the nsplit slabs in split order, 4 elements per thread (M K is a multiple of 32).
__global__ __launch_bounds__(kBlock) void hqq_matmul_t_reduce_kernel(const MatmulTParams P) {
  typedef float float4_t __attribute__((ext_vector_type(4)));
  const int64_t mk = P.M * P.K;
  for (int64_t i = ((int64_t)blockIdx.x * kBlock + threadIdx.x) * 4; i < mk; i += (int64_t)gridDim.x * kBlock * 4) {
    float4_t y = *reinterpret_cast<const float4_t*>(P.part + i);
    for (int s = 1; s < P.nsplit; ++s) y += *reinterpret_cast<const float4_t*>(P.part + s * mk + i);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      if (P.out_f32) static_cast<float*>(P.dX)[i + v] = y[v];
      else static_cast<_Float16*>(P.dX)[i + v] = (_Float16)y[v];
    }
  }
}

// Tiles of 256 rows from 256 rows an expert on (each weight tile is dequantized once per 256
// rows), else of 128; the walk over n is split where the tiles alone are fewer than two per CU,
// into parts of at least 8 steps.  From the shapes alone.
struct TGeom {
  int wm, nsplit;
  int64_t tiles;
};
TGeom t_geometry(int64_t M, int64_t N, int64_t K, int64_t experts) {
  TGeom g;
  const bool grouped = experts > 0;
  g.wm = M / (grouped ? experts : 1) >= 256 ? 4 : 2;
  const int64_t bm = 64 * g.wm;
  g.tiles = grouped ? max_row_tiles(M, experts, bm) : (M + bm - 1) / bm;
  const int64_t blocks = g.tiles * ((K + kTK - 1) / kTK);
  int64_t ns = blocks > 0 ? 512 / blocks : 1;
  const int64_t most = N / (8 * kTN);
  if (ns > most) ns = most;
  g.nsplit = ns < 1 ? 1 : (int)ns;
  return g;
}

template <int NB, int WM>
void launch_t(const MatmulTParams& P, int64_t tiles, hipStream_t st) {
  const dim3 grid((unsigned)((P.K + kTK - 1) / kTK), (unsigned)tiles, (unsigned)P.nsplit), block(2 * WM * kWave);
  if (P.offsets) hipLaunchKernelGGL((hqq_matmul_t_kernel<NB, WM, true>), grid, block, 0, st, P);
  else hipLaunchKernelGGL((hqq_matmul_t_kernel<NB, WM, false>), grid, block, 0, st, P);
}

template <int NB>
hipError_t launch_t_nb(MatmulTParams P, hipStream_t st) {
  const TGeom g = t_geometry(P.M, P.N, P.K, P.offsets ? P.experts : 0);
  P.nsplit = g.nsplit;
  if (g.wm == 4) launch_t<NB, 4>(P, g.tiles, st);
  else launch_t<NB, 2>(P, g.tiles, st);
  if (g.nsplit > 1) {
    int64_t blocks = (P.M * P.K + 4 * kBlock - 1) / (4 * kBlock);
    if (blocks > 4096) blocks = 4096;
    hipLaunchKernelGGL(hqq_matmul_t_reduce_kernel, dim3((unsigned)blocks), dim3(kBlock), 0, st, P);
  }
  return hipGetLastError();
}

}  // namespace

int64_t matmul_t_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t experts) {
  const TGeom g = t_geometry(M, N, K, experts);
  return g.nsplit > 1 ? (int64_t)g.nsplit * M * K * (int64_t)sizeof(float) : 0;
}

hipError_t launch_matmul_t(MatmulTParams prm, hipStream_t stream) {
  switch (prm.nbits) {
    case 2: return launch_t_nb<2>(prm, stream);
    case 3: return launch_t_nb<3>(prm, stream);
    case 4: return launch_t_nb<4>(prm, stream);
    case 8: return launch_t_nb<8>(prm, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace hqq
