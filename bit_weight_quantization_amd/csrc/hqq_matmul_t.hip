// hqq_matmul_t.hip -- gfx950 kernels of the gradient of the product with a quantized weight,
// dX = dY Q^-1(W_q), for one weight or for rows sorted by expert with a weight each.
//
// dX[m][k] = sum over n of dY[m][n] s[n][k/g] (q[n][k] - z[n][k/g]): the contraction runs over
// the weight's rows, while codes are packed along k.  The weight tile is dequantized once per
// block into LDS as it is stored (rows n, binary16, as in the forward kernels), and the matrix
// operand, which needs 8 consecutive n of one k in a lane, is read with gfx950's transposing LDS
// read (ds_read_b64_tr_b16: of each 16 lanes' 4 x 16 block of halves lane i gets column i).
// For many rows no unit is busy for more than about a quarter of the time (counters: matrix cores 24%,
// LDS 24%, VALU 22%): the waits within a step bound it.  2048 rows, 4096 x 4096 (4 bits) with adapters of rank 32 take
// 105 us (124 with every operand read right before its use), 4002 rows of 8 such experts 250-260 us
// (280), 530-650 TFLOP/s; dY in 128-byte pieces of a row (8 threads a row) instead of 16-byte ones of
// 64 rows, and 16 columns a lane in the epilogue, took the first from 150 us.
// For few rows bound by the latency of one block's walk over n, which is split over blocks and joined
// in a fixed order (place_tile).
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
constexpr int kTUnit = 8;            // steps in a unit of splitting n
constexpr int t_slots(int wm) { return wm == 4 ? 32 : 64; }  // blocks of an XCD at a time (LDS: one or two per CU)
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
// v_mfma_f32_32x32x16_f16), n in steps of 64.  8 threads stage the 128 bytes of a row of dY, and each
// thread 16 codes of one or two weight rows per step (32 of one row, 64 bytes apart in LDS between
// lanes, cost bank conflicts in 44% of the LDS cycles).  Codes are loaded two steps ahead in registers,
// LDS is double-buffered, one LDS-only barrier per step.  The weight is the A
// operand and its row 8 a + 4 h + b stands for column 16 h + 4 a + b of the 32, so that a lane ends
// with 16 consecutive columns of one row of dX.
enum Rows : int { kAll = 0, kExperts = 1, kAdapted = 2 };  // rows of one weight, of experts, with adapters

template <int NB, int WM, int ROWS>
__global__ __launch_bounds__(2 * WM * kWave) __attribute__((amdgpu_waves_per_eu(2)))
void hqq_matmul_t_kernel(const MatmulTParams P) {
  constexpr int T = 2 * WM * kWave, BM = 64 * WM;
  constexpr int CB = 16, BP = kTK / CB;  // codes of a weight row per thread, threads per row
  constexpr int BR = T / BP, RB = kTN / BR;  // weight rows per round of loads, rounds
  static_assert(RB == 1 || RB == 2, "one or two weight rows per thread");
  __shared__ __align__(16) _Float16 As[2][BM][kTRowA];
  __shared__ __align__(16) _Float16 Bs[2][kTN][kTRowB];
  const int tid = threadIdx.x, wid = __builtin_amdgcn_readfirstlane(tid / kWave), lane = tid & (kWave - 1);
  const int wm = wid >> 1, wn = wid & 1;

  const int64_t cols = (P.K + kTK - 1) / kTK;
  const int units = (int)((P.N + kTN * kTUnit - 1) / (kTN * kTUnit));
  const int64_t tiles = ROWS == kExperts ? count_row_tiles(P.offsets, P.experts, P.M, BM) : (P.M + BM - 1) / BM;
  const TilePlace place = place_tile(blockIdx.x, tiles, cols, units, t_slots(WM), P.xcd_slabs);
  if (place.tile < 0) return;
  int64_t row0 = place.tile * BM;
  int rows = (int)(P.M - row0 < BM ? P.M - row0 : BM);
  int64_t w0 = 0;                    // first weight row of the expert
  int64_t N = P.N;
  if constexpr (ROWS == kExperts) {
    const RowTile t = find_row_tile(P.offsets, P.experts, P.M, BM, place.tile);
    if (t.rows <= 0) return;
    row0 = t.row0;
    rows = t.rows;
    w0 = (int64_t)t.group * P.N;
    if (t.group == P.experts) N = 0, w0 = 0;  // rows of no expert: zeros
  }
  const int64_t k0 = place.col * kTK;
  const int64_t steps = (N + kTN - 1) / kTN;
  const int64_t st0 = (int64_t)units * place.part / place.parts * kTUnit;
  const int64_t send = (int64_t)units * (place.part + 1) / place.parts * kTUnit;
  const int64_t st1 = send < steps ? send : steps;

  const int xr = tid >> 3, xp = tid & 7;  // 16-byte piece xp of rows xr + T / 8 i (past the tile: its last row)
  const uint16_t* yrow[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m = xr + T / 8 * i;
    int64_t row = row0 + (m < rows ? m : rows - 1);
    if constexpr (ROWS == kAdapted) {
      const int32_t o = P.low.order[row];
      row = o < 0 ? ~o : o;
    }
    yrow[i] = P.dY + row * P.N + 8 * xp;
  }
  const int br = tid / BP, bp = tid % BP;
  const int64_t kc = k0 + CB * bp < P.K ? k0 + CB * bp : 0;  // (columns past K are not stored)
  const int64_t row_bytes = (P.K >> 3) * NB, gpr = P.K >> P.group_shift;

  uint4 ar[4];
  uint32_t cw[2][RB][Codes16<NB>::kWords];
  uint32_t s16[2][RB], z16[2][RB];
  auto load_rows = [&](int64_t step) {
    const int64_t nb = step * kTN;
    if (nb + kTN <= N) {
#pragma unroll
      for (int i = 0; i < 4; ++i) ar[i] = load8(yrow[i] + nb);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) ar[i] = load8_part(yrow[i] + nb, N - nb - 8 * xp);
    }
  };
  auto load_codes = [&](auto st_const, int64_t step) {
    constexpr int S = decltype(st_const)::value;
#pragma unroll
    for (int j = 0; j < RB; ++j) {
      const int64_t m = step * kTN + br + BR * j, n = w0 + (m < N ? m : N - 1);
      load_codes16<NB>(P.packed + n * row_bytes + (kc >> 4) * (2 * NB), cw[S][j]);
      const int64_t g = n * gpr + (kc >> P.group_shift);
      s16[S][j] = P.scale16[g];
      z16[S][j] = P.zero16[g];
    }
  };
  auto write_rows = [&](int buf) {
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(&As[buf][xr + T / 8 * i][8 * xp]) = ar[i];
  };
  // half of the thread's codes decoded and written; rows past N enter as zeros
  auto write_weights = [&](auto st_const, int buf, int64_t step, int half) {
    constexpr int S = decltype(st_const)::value;
#pragma unroll
    for (int u = half * RB; u < (half + 1) * RB; ++u) {  // 8 codes each
      const int j = u / 2, i = u % 2;
      const bool ok = step * kTN + br + BR * j < N;
      const float sv = ok ? h2f(s16[S][j]) : 0.f;
      const PairScale sc = {sv * kSub, ok ? -sv * h2f(z16[S][j]) : 0.f};
      *reinterpret_cast<uint4*>(&Bs[buf][br + BR * j][CB * bp + 8 * i]) =
          make_uint4(decode_pair<NB>(cw[S][j], i, 0, sc), decode_pair<NB>(cw[S][j], i, 1, sc),
                     decode_pair<NB>(cw[S][j], i, 2, sc), decode_pair<NB>(cw[S][j], i, 3, sc));
    }
  };

  float16_t acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;

  // the lane's place in a transposing read: group lane / 16 = 2 (n half) + (a half), rows n 8 (lane /
  // 32) .. + 4 (a second read: + 4 .. + 8); lane l of a group supplies row l / 4 and the 4 columns
  // that lanes 4 (l % 4) .. + 4 of the group take: 16 (l & 1) + 4 (2 (a half) + (l & 3) / 2)
  const int tr_row = 8 * (lane >> 5) + ((lane & 15) >> 2);
  const int tr_col = 16 * (lane & 1) + 4 * (2 * ((lane >> 4) & 1) + ((lane & 3) >> 1));
  // operands of matrix step ks of a buffer
  struct Frags {
    half8_t a[2], b[2];
  };
  auto read_frags = [&](int buf, int ks, Frags& f) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      f.a[i] = *reinterpret_cast<const half8_t*>(&As[buf][wm * 64 + i * 32 + (lane & 31)][ks * 16 + (lane >> 5) * 8]);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const _Float16* src = &Bs[buf][ks * 16 + tr_row][wn * 64 + j * 32 + tr_col];
      const short4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4*)src);
      const short4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4*)(src + 4 * kTRowB));
      f.b[j] = __builtin_bit_cast(half8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  };
  auto products = [&](const Frags& f) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f.b[j], f.a[i], acc[i][j], 0, 0, 0);
  };
  // One step: four matrix steps, each behind the LDS reads of the next one.  The next tile is written
  // (its weights decoded) under the first two; the barrier stands before the fourth, whose operands are in
  // registers by then, so that the next tile's first reads run under it.
  Frags fr[2];
  auto step = [&](auto st_const, auto used_const, int64_t c) {
    constexpr int S = decltype(st_const)::value;
    constexpr bool USED = decltype(used_const)::value;
    constexpr std::integral_constant<int, S ^ 1> other{};
    const int64_t c1 = c + 1 < st1 ? c + 1 : st0, c2 = c + 2 < st1 ? c + 2 : st0;  // (past the end: unused)
    if constexpr (USED) read_frags(S, 1, fr[1]);
    write_rows(S ^ 1);
    load_rows(c2);
    load_codes(st_const, c2);
    __builtin_amdgcn_sched_barrier(0);
    write_weights(other, S ^ 1, c1, 0);
    if constexpr (USED) products(fr[0]);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (USED) read_frags(S, 2, fr[0]);
    write_weights(other, S ^ 1, c1, 1);
    if constexpr (USED) {
      products(fr[1]);
      __builtin_amdgcn_sched_barrier(0);
      read_frags(S, 3, fr[1]);
      products(fr[0]);
      __builtin_amdgcn_sched_barrier(0);
    }
    lds_barrier();
    if constexpr (USED) {
      read_frags(S ^ 1, 0, fr[0]);
      products(fr[1]);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto walk = [&](auto used_const) {
    constexpr std::integral_constant<int, 0> s0{};
    constexpr std::integral_constant<int, 1> s1{};
    const int64_t second = st0 + 1 < st1 ? st0 + 1 : st0;
    load_rows(st0);
    load_codes(s0, st0);
    load_codes(s1, second);
    write_rows(0);
    load_rows(second);
    write_weights(s0, 0, st0, 0);
    write_weights(s0, 0, st0, 1);
    lds_barrier();
    if constexpr (decltype(used_const)::value) read_frags(0, 0, fr[0]);
    for (int64_t c = st0; c < st1; c += 2) {
      step(s0, used_const, c);
      if (c + 1 >= st1) break;
      step(s1, used_const, c + 1);
    }
  };
  // a wavefront whose rows are all past the tile only stages (wave-uniform; as many barriers)
  const bool used = wm * 64 < rows;
  if constexpr (ROWS != kAdapted) {
    if (!used) {
      if (st0 < st1) walk(std::false_type{});
      return;
    }
    if (st0 < st1) walk(std::true_type{});
  } else {
    if (st0 < st1) {
      if (used) walk(std::true_type{});
      else walk(std::false_type{});
    }
    lds_barrier();  // (the buffers are used again below)
  }

  float back[2] = {1.f, 1.f};
  if constexpr (ROWS == kAdapted) {
    static_assert(low_halves(BM) <= 2 * BM * kTRowA, "the parts fit the buffers of dY");
    if (place.part == 0) {
      __shared__ float scale_up[BM];
      __shared__ int row_group[BM];
      const int l = lane & 31;
      int64_t col[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) col[j] = k0 + wn * 64 + j * 32 + 16 * ((l >> 2) & 1) + 4 * (l >> 3) + (l & 3);
      add_low<BM, T>(acc, back, P.low, row0, rows, wm * 64, col, &As[0][0][0], scale_up, row_group);
    }
  }

  // lane: row lane % 32 of fragment i, columns 32 j + 16 (lane / 32) .. + 16 (K is a multiple of 32)
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int m = wm * 64 + i * 32 + (lane & 31);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int c = wn * 64 + j * 32 + 16 * (lane >> 5);
      float v[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = back[i] * acc[i][j][e];
      if (place.parts > 1) {  // a part of the sum, in the block's own slab
        __builtin_memcpy(P.slabs + ((int64_t)place.slot * BM + m) * kTK + c, v, 64);
        continue;
      }
      if (m >= rows || k0 + c >= P.K) continue;
      int64_t row = row0 + m;
      if constexpr (ROWS == kAdapted) {
        const int32_t o = P.low.order[row];
        row = o < 0 ? ~o : o;
      }
      const int64_t at = row * P.K + k0 + c;
      if (P.out_f32) {
        __builtin_memcpy(static_cast<float*>(P.dX) + at, v, 64);
      } else {
        _Float16 y[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) y[e] = (_Float16)v[e];
        __builtin_memcpy(static_cast<_Float16*>(P.dX) + at, y, 32);
      }
    }
  }
}

// Tiles that were split: the sum of their parts in order.  A block per split tile and 8 rows.
constexpr int kTJoinRows = 8;
template <int WM, int ROWS>
__global__ __launch_bounds__(kBlock) void hqq_matmul_t_join_kernel(const MatmulTParams P) {
  constexpr int BM = 64 * WM;
  const int64_t cols = (P.K + kTK - 1) / kTK;
  const int64_t tiles = ROWS == kExperts ? count_row_tiles(P.offsets, P.experts, P.M, BM) : (P.M + BM - 1) / BM;
  const int xcd = blockIdx.x % kXcds, rest = blockIdx.x / kXcds;
  const TileShare s = tile_share(xcd, tiles * cols, (int)((P.N + kTN * kTUnit - 1) / (kTN * kTUnit)), t_slots(WM));
  if (rest >= s.rest || (rest + 1) * s.parts > P.xcd_slabs) return;
  const TilePlace place = place_at(s.first + s.full + rest, tiles, cols);
  int64_t row0 = place.tile * BM;
  int rows = (int)(P.M - row0 < BM ? P.M - row0 : BM);
  if constexpr (ROWS == kExperts) {
    const RowTile t = find_row_tile(P.offsets, P.experts, P.M, BM, place.tile);
    row0 = t.row0;
    rows = t.rows;
  }
  const int c = threadIdx.x % kTK;
  const int64_t k = place.col * kTK + c;
  if (k >= P.K) return;
  const float* slab = P.slabs + (int64_t)(xcd * P.xcd_slabs + rest * s.parts) * BM * kTK + c;
  const int m0 = blockIdx.y * kTJoinRows;
#pragma unroll
  for (int u = 0; u < kTJoinRows; u += kBlock / kTK) {
    const int m = m0 + u + threadIdx.x / kTK;
    if (m >= rows) break;
    float part[kMaxParts];
#pragma unroll
    for (int p = 0; p < kMaxParts; ++p) part[p] = p < s.parts ? slab[((int64_t)p * BM + m) * kTK] : 0.f;
    float y = part[0];
#pragma unroll
    for (int p = 1; p < kMaxParts; ++p) y += part[p];
    int64_t row = row0 + m;
    if constexpr (ROWS == kAdapted) {
      const int32_t o = P.low.order[row];
      row = o < 0 ? ~o : o;
    }
    const int64_t at = row * P.K + k;
    if (P.out_f32) static_cast<float*>(P.dX)[at] = y;
    else static_cast<_Float16*>(P.dX)[at] = (_Float16)y;
  }
}

// Tiles of 256 rows from a mean of 1024 rows an expert on (each weight tile is dequantized once per 256
// rows), else of 128 (a group's last tile is half full on average: mean 500 rows, 267 us against 284 us
// with 256, before the read-ahead).
int t_wm(int64_t M, int64_t experts) { return M / (experts > 0 ? experts : 1) >= 1024 ? 4 : 2; }
int64_t t_most(int64_t M, int64_t K, int64_t experts, int64_t bm) {
  return (K + kTK - 1) / kTK * (experts > 0 ? max_row_tiles(M, experts, bm) : (M + bm - 1) / bm);
}

// Whether tiles may be split (one weight: whether any is; groups' tiles are counted on the device; one
// unit of n is never split).
bool t_splits(int64_t M, int64_t N, int64_t K, int64_t experts, int wm) {
  const int64_t units = (N + kTN * kTUnit - 1) / (kTN * kTUnit);
  if (units <= 1) return false;
  return experts > 0 || place_splits(t_most(M, K, 0, 64 * wm), (int)(units < kMaxParts ? units : kMaxParts), t_slots(wm));
}

template <int NB, int WM, int ROWS>
hipError_t launch_t(MatmulTParams P, hipStream_t st) {
  const int64_t most = t_most(P.M, P.K, ROWS == kExperts ? P.experts : 0, 64 * WM), blocks = place_blocks(most, t_slots(WM));
  if (blocks * 2 * WM * kWave > UINT32_MAX) return hipErrorInvalidValue;  // threads of a grid
  P.xcd_slabs = place_slabs(most, t_slots(WM));
  hipLaunchKernelGGL((hqq_matmul_t_kernel<NB, WM, ROWS>), dim3((unsigned)blocks), dim3(2 * WM * kWave), 0, st, P);
  if (t_splits(P.M, P.N, P.K, ROWS == kExperts ? P.experts : 0, WM)) {  // (split tiles: at most half of an XCD's slots)
    const dim3 join(kXcds * t_slots(WM) / 2, 64 * WM / kTJoinRows);
    hipLaunchKernelGGL((hqq_matmul_t_join_kernel<WM, ROWS>), join, dim3(kBlock), 0, st, P);
  }
  return hipGetLastError();
}

template <int NB>
hipError_t launch_t_nb(const MatmulTParams& P, hipStream_t st) {
  const bool tall = t_wm(P.M, P.offsets ? P.experts : 0) == 4;
  if (P.offsets) return tall ? launch_t<NB, 4, kExperts>(P, st) : launch_t<NB, 2, kExperts>(P, st);
  if (P.low.low) return tall ? launch_t<NB, 4, kAdapted>(P, st) : launch_t<NB, 2, kAdapted>(P, st);
  return tall ? launch_t<NB, 4, kAll>(P, st) : launch_t<NB, 2, kAll>(P, st);
}

}  // namespace

int64_t matmul_t_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t experts) {
  const int wm = t_wm(M, experts);
  if (!t_splits(M, N, K, experts, wm)) return 0;
  return (int64_t)kXcds * place_slabs(t_most(M, K, experts, 64 * wm), t_slots(wm)) * 64 * wm * kTK *
         (int64_t)sizeof(float);
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
