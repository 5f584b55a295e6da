// hqq_low_tile.h -- the adapters' low-rank product of a tile of sorted rows, added to the
// accumulators of the tile's large product (hqq_group_gemm.hip, hqq_matmul_t.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "hqq_codes.h"
#include "hqq_internal.h"

namespace hqq {

// Row i of the sorted rows (row order[i] of X; negative: of no adapter, behind all others) of
// adapter g gets scales[g] low[i] factor[g]^T added.
struct LowRank {
  const float* low;         // M x rank, sorted; null: nothing is added
  const uint16_t* factor;   // adapters x width x rank binary16
  const float* scales;
  const int32_t* ids;       // adapter of every row of X
  const int32_t* order;
  const int32_t* offsets;   // first sorted row of every adapter, adapters + 1 values
  int64_t width;
  int rank, adapters;
};

// The product's accumulators take the sum: no fp32 base goes through memory (with a pass of its own the
// gradient of 2048 rows, 4096 x 4096, rank 32 took 182 instead of 172 us).
namespace {

constexpr int kLowRound = 64;                // low-rank values per round
constexpr int kLowRow = kLowRound + 8;       // halves per LDS row
constexpr int low_halves(int bm) { return 2 * bm * kLowRow; }

// acc[a][j] (row frag0 + 32 a + lane % 32 of the tile; weight row col[j] of the lane as A operand of
// v_mfma_f32_32x32x16_f16) += the low-rank product, all scaled by 1 / back[a].  s low[i] enters as
// two binary16 parts of the row scaled by a power of two (22 bits below the row's largest value);
// the accumulators of the row are scaled alike (exact), the caller scales back.  A tile may hold rows
// of several adapters: each in turn, with the parts of the other rows left out.  The whole block of T
// threads calls it; parts: low_halves(BM) halves, scale_up and row_group: BM values of LDS, free.
template <int BM, int T, int TA, int TJ>
__device__ __forceinline__ void add_low(float16_t (&acc)[TA][TJ], float (&back)[TA], const LowRank& L,
                                        int64_t row0, int rows, int frag0, const int64_t (&col)[TJ],
                                        _Float16* parts, float* scale_up, int* row_group) {
  constexpr int XP = BM * 8 / T, XT = T / 8;  // 8 threads share a row
  const int tid = threadIdx.x, lane = tid & (kWave - 1), i = lane & 31, h = lane >> 5;
  const int xp = tid & 7, xr = tid >> 3;
  if (row0 >= L.offsets[L.adapters]) return;  // uniform: no row of an adapter
#pragma unroll
  for (int p = 0; p < XP; ++p) {
    const int m = xr + XT * p;
    int g = -1;
    if (m < rows) {
      const int32_t o = L.order[row0 + m];
      g = o < 0 ? -1 : L.ids[o];
    }
    float largest = 0.f;
    if (g >= 0)
      for (int r = xp; r < L.rank; r += 8) {
        const float v = L.scales[g] * L.low[(row0 + m) * L.rank + r];
        largest = __builtin_isfinite(v) ? __builtin_fmaxf(largest, __builtin_fabsf(v)) : largest;
      }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) largest = __builtin_fmaxf(largest, __shfl_xor(largest, o, kWave));
    // 2^x: the largest comes to [2^13, 2^14); x within -114 .. 40, so that the accumulators stay
    // finite (smaller rows then lose what lies below 2^-64)
    int x = 13 - ((int)((__builtin_bit_cast(uint32_t, largest) >> 23) & 255) - 127);
    x = x > 40 ? 40 : x < -114 ? -114 : x;
    if (xp == 0) {
      scale_up[m] = g >= 0 ? __builtin_bit_cast(float, (uint32_t)(127 + x) << 23) : 1.f;
      row_group[m] = g;
    }
  }
  __syncthreads();
#pragma unroll
  for (int a = 0; a < TA; ++a) {
    const float up = scale_up[frag0 + 32 * a + i];
    back[a] = __builtin_bit_cast(float, (uint32_t)(254 << 23) - __builtin_bit_cast(uint32_t, up));  // 1 / up
#pragma unroll
    for (int j = 0; j < TJ; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[a][j][v] *= up;
  }
  for (int m0 = 0; m0 < rows;) {  // uniform: the tile's adapters
    const int g = __builtin_amdgcn_readfirstlane(row_group[m0]);
    if (g < 0) break;
    const int64_t gend = L.offsets[g + 1] - row0;
    const int m1 = gend <= m0 ? m0 + 1 : gend < rows ? (int)gend : rows;  // (past m0 in any case)
    const float s = L.scales[g];
    for (int r0 = 0; r0 < L.rank; r0 += kLowRound) {
      // thread: rows xr + XT p, low-rank values 8 xp .. + 8 of the round
#pragma unroll
      for (int p = 0; p < XP; ++p) {
        const int m = xr + XT * p, r = r0 + 8 * xp;
        half8_t hi = {}, lo = {};
        if (m >= m0 && m < m1 && r < L.rank) {
          const float up = s * scale_up[m];
          const float* low = L.low + (row0 + m) * L.rank + r;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float v = up * low[e];
            hi[e] = (_Float16)v;
            lo[e] = __builtin_isfinite((float)hi[e]) ? (_Float16)(v - (float)hi[e]) : (_Float16)0.f;
          }
        }
        *reinterpret_cast<half8_t*>(parts + m * kLowRow + 8 * xp) = hi;
        *reinterpret_cast<half8_t*>(parts + (BM + m) * kLowRow + 8 * xp) = lo;
      }
      __syncthreads();
#pragma unroll 1
      for (int st = 0; st < kLowRound / 16; ++st) {
        const int r = r0 + 16 * st + 8 * h;
        if (r0 + 16 * st >= L.rank) break;  // uniform
        half8_t wl[TJ];
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
          wl[j] = (half8_t){};
          if (col[j] < L.width && r < L.rank)
            wl[j] = *reinterpret_cast<const half8_t*>(L.factor + ((int64_t)g * L.width + col[j]) * L.rank + r);
        }
#pragma unroll
        for (int a = 0; a < TA; ++a) {
          const int f = frag0 + 32 * a;
          if (f >= m1 || f + 32 <= m0) continue;  // wave-uniform: no row of this adapter
          const _Float16* src = parts + (f + i) * kLowRow + 16 * st + 8 * h;
          const half8_t hi = *reinterpret_cast<const half8_t*>(src);
          const half8_t lo = *reinterpret_cast<const half8_t*>(src + BM * kLowRow);
          // a lane's sums are one row's: rows of another adapter keep theirs, also where this one's
          // factor holds an infinity or a NaN (times their zeros)
          const bool mine = f + i >= m0 && f + i < m1;
#pragma unroll
          for (int j = 0; j < TJ; ++j) {
            float16_t sum = __builtin_amdgcn_mfma_f32_32x32x16_f16(wl[j], hi, acc[a][j], 0, 0, 0);
            sum = __builtin_amdgcn_mfma_f32_32x32x16_f16(wl[j], lo, sum, 0, 0, 0);
            if (f >= m0 && f + 32 <= m1) {  // uniform
              acc[a][j] = sum;
            } else {
#pragma unroll
              for (int v = 0; v < 16; ++v) acc[a][j][v] = mine ? sum[v] : acc[a][j][v];
            }
          }
        }
      }
      __syncthreads();
    }
    m0 = m1;
  }
}

}  // namespace
}  // namespace hqq
