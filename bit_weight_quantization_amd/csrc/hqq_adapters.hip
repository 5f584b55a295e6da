// hqq_adapters.hip -- gfx950 kernels of low-rank adapters of many requests beside a shared
// projection, and of their gradients.
//
// Row m of X belongs to adapter a = ids[m] (outside [0, adapters): to none):
//   v_m = A_a x_m,  y_m = base_m + s_a B_a v_m
//   u_m = B_a^T dy_m,  dx_m = base_m + s_a A_a^T u_m,
//   dA_a = s_a sum_m u_m x_m^T,  dB_a = s_a sum_m dy_m v_m^T
// v and u (rank numbers a row) stay in fp32.  Where they meet 16-bit factors or rows on the
// matrix cores they enter as a sum of 16-bit parts: two binary16 parts of the value scaled by a
// power of two (22 bits below the largest value of the row, or of a piece of the adapter's rows), or two or
// three bfloat16 parts (16 or 24 bits), so the products lose nothing that fp32 sums keep.
//
// Bound by HBM: rows of X, dY, base and Y once or twice each, used factors once; 2 rank
// operations per byte at most.  Few rows (decode) take a wavefront's dot products over the
// row's own factors; more rows are sorted by adapter and go through tiles of one adapter.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "hqq_adapters.h"
#include "hqq_group_gemm.h"
#include "hqq_internal.h"
#include "hqq_matmul.h"
#include "hqq_matmul_t.h"
#include "hqq_route.h"
#include "hqq_tiles.h"

namespace hqq {
namespace {

typedef float float4_t __attribute__((ext_vector_type(4)));
typedef short short4_t __attribute__((ext_vector_type(4)));
typedef short short8_t __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) short4_t lds_short4;

struct F16 {
  typedef _Float16 vec8 __attribute__((ext_vector_type(8)));
  static __device__ __forceinline__ float up(uint16_t v) { return (float)__builtin_bit_cast(_Float16, v); }
  static __device__ __forceinline__ uint16_t down(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }
  static __device__ __forceinline__ float4_t mfma(short8_t a, short8_t b, float4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(vec8, a), __builtin_bit_cast(vec8, b), c, 0, 0, 0);
  }
  static constexpr bool kScaled = true;   // parts of a scaled value (binary16 has 5 exponent bits)
  static constexpr int kParts = 2, kPartsOut16 = 2;
};
struct Bf16 {
  typedef __bf16 vec8 __attribute__((ext_vector_type(8)));
  static __device__ __forceinline__ float up(uint16_t v) { return __builtin_bit_cast(float, (uint32_t)v << 16); }
  static __device__ __forceinline__ uint16_t down(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
  static __device__ __forceinline__ float4_t mfma(short8_t a, short8_t b, float4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(vec8, a), __builtin_bit_cast(vec8, b), c, 0, 0, 0);
  }
  static constexpr bool kScaled = false;
  static constexpr int kParts = 3, kPartsOut16 = 2;  // 16 bits suffice under a bfloat16 result
};

// v as a sum of PARTS 16-bit numbers, each the nearest to what the ones before leave.
template <typename D, int PARTS>
__device__ __forceinline__ void split(float v, uint16_t (&part)[PARTS]) {
#pragma unroll
  for (int p = 0; p < PARTS; ++p) {
    part[p] = D::down(v);
    const float back = D::up(part[p]);
    v = __builtin_isfinite(back) ? v - back : 0.f;  // (an infinity is its first part alone)
  }
}

// |v|, or 0 for what no scale can serve (infinities and NaN keep their own way through split).
__device__ __forceinline__ float finite_abs(float v) {
  return __builtin_isfinite(v) ? __builtin_fabsf(v) : 0.f;
}

// Exponent x with 2^x largest in [2^13, 2^14), 0 < x's range cut so that 2^x and 2^-x are
// normal numbers.
__device__ __forceinline__ int scale_exponent(float largest) {
  const int e = (int)((__builtin_bit_cast(uint32_t, largest) >> 23) & 255) - 127;
  return min(13 - e, 126);
}
__device__ __forceinline__ float exp2i(int x) { return __builtin_bit_cast(float, (uint32_t)(127 + x) << 23); }

// 8 16-bit numbers from p (2-byte aligned) of which the first `valid` exist, the others zero.
__device__ __forceinline__ short8_t load8(const uint16_t* p, int64_t valid) {
  short8_t v;
  if (valid >= 8) {
    __builtin_memcpy(&v, p, 16);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < valid ? (short)p[i] : (short)0;
  }
  return v;
}

// The sum of n values `stride` apart, in order, 8 loads in flight (one by one each add would wait for
// its load: the second step of 64 rows, 8192 x 8192 of 16 splits took 8.2 us).
__device__ __forceinline__ float sum_strided(const float* p, int64_t stride, int n) {
  float y = 0.f;
  for (int i0 = 0; i0 < n; i0 += 8) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i0 + i < n ? p[(i0 + i) * stride] : 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) y += v[i];
  }
  return y;
}

__device__ __forceinline__ float read_base(const AdapterParams& P, int64_t at);

// ---------------------------------------------------------------- few rows --

constexpr int64_t kFewRows = 64;
constexpr int kFewK = kWave * 8;    // values of k per block
constexpr int kFewRank = 16;        // rows of A per block: four per wavefront
constexpr int kFewN = 128;          // outputs per block

// part[split][m][r] = the part of v_m[r] over 512 values of k.
template <typename D>
__global__ __launch_bounds__(kBlock) void hqq_adapter_shrink_few_kernel(const AdapterParams P, float* part) {
  const int lane = threadIdx.x & (kWave - 1), wid = threadIdx.x / kWave;
  const int64_t m = blockIdx.y;
  const int a = P.ids[m];
  if ((uint32_t)a >= (uint32_t)P.adapters) return;
  const int64_t k = (int64_t)blockIdx.x * kFewK + 8 * lane;
  const bool on = k < P.K;  // K is a multiple of 8
  const int r0 = blockIdx.z * kFewRank + wid * 4;
  const uint16_t* Ar = P.A + (int64_t)a * P.rank * P.K;
  short8_t x = {}, f[4] = {};
  if (on) {
    x = load8(P.X + m * P.K + k, 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + i < P.rank ? r0 + i : P.rank - 1;
      f[i] = load8(Ar + r * P.K + k, 8);
    }
  }
  float dot[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) dot[i] = __builtin_fmaf(D::up((uint16_t)x[e]), D::up((uint16_t)f[i][e]), dot[i]);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int o = kWave / 2; o > 0; o >>= 1) dot[i] += __shfl_xor(dot[i], o, kWave);
  if (lane < 4 && r0 + lane < P.rank) {
    const float v = lane == 0 ? dot[0] : lane == 1 ? dot[1] : lane == 2 ? dot[2] : dot[3];
    part[((int64_t)blockIdx.x * P.M + m) * P.rank + r0 + lane] = v;
  }
}

// A thread per output: y = base + s sum_r v[r] B[n][r].
template <typename D>
__global__ __launch_bounds__(kFewN) void hqq_adapter_expand_few_kernel(const AdapterParams P, const float* part,
                                                                       int splits) {
  __shared__ float v[kMaxAdapterRank];
  const int64_t m = blockIdx.y, n = (int64_t)blockIdx.x * kFewN + threadIdx.x;
  const int a = P.ids[m];
  const bool has = (uint32_t)a < (uint32_t)P.adapters;
  float y = n < P.N ? read_base(P, m * P.N + n) : 0.f;  // (in flight with what follows)
  if (has) {
    const float s = P.scales[a];
    for (int r = threadIdx.x; r < P.rank; r += kFewN) {
      v[r] = s * sum_strided(part + m * P.rank + r, P.M * P.rank, splits);
    }
  }
  __syncthreads();
  if (n >= P.N) return;
  if (has) {
    const uint16_t* b = P.B + ((int64_t)a * P.N + n) * P.rank;
    float t = 0.f;
    for (int r = 0; r < P.rank; r += 8) {
      const short8_t w = load8(b + r, 8);
#pragma unroll
      for (int e = 0; e < 8; ++e) t = __builtin_fmaf(v[r + e], D::up((uint16_t)w[e]), t);
    }
    y += t;
  }
  if (P.out_f32) static_cast<float*>(P.out)[m * P.N + n] = y;
  else static_cast<uint16_t*>(P.out)[m * P.N + n] = D::down(y);
}

__device__ __forceinline__ float read_base(const AdapterParams& P, int64_t at) {
  if (!P.base) return 0.f;
  if (P.base_slabs > 0) {
    return sum_strided(static_cast<const float*>(P.base) + at, P.base_stride, P.base_slabs);
  }
  if (P.base_f32) return static_cast<const float*>(P.base)[at];
  const uint16_t v = static_cast<const uint16_t*>(P.base)[at];
  return P.dtype == 0 ? F16::up(v) : Bf16::up(v);
}

// --------------------------------------------------------- sorted row tiles --

// One side of the low-rank step: rows (M x width, 16-bit, 2-byte aligned) times the adapters'
// factor rows (rank x stride, 16-byte aligned, zeros behind width): out[i][r], i sorted.
struct ShrinkSide {
  const uint16_t* rows;
  const uint16_t* factor;   // adapters x rank x stride
  int64_t width, stride;
  float* out;               // M x rank
  float* largest;           // the largest finite |out| of every tile of 16 rows (null: not kept)
};
struct ShrinkParams {
  ShrinkSide side[2];       // blockIdx.z
  const int32_t* order;
  const int32_t* offsets;
  int64_t M;
  int rank, adapters;
};

// Wavefronts of a block: as many as the registers and the LDS of the rank allow (their loads in flight
// are what hides the latency of the few chunks each has).
constexpr int shrink_waves(int rt) { return rt <= 4 ? 16 : 8; }
constexpr int kShrinkRows = 16;

// 8190 rows of X (4096) and dY (11008), bfloat16, rank 16: 247 MB in 65 us, 3.8 TB/s; 4096 x 8192,
// rank 64: 41-44 us, the 1 MB of a factor read from L2 by each block of 16 rows.
//
// A block per 16 sorted rows of one adapter; its W wavefronts take every W-th chunk of 128 of
// the width and their tiles are added in LDS in order.  Lane i + 16 q holds 8 values (8 q ..) of row
// i of both operands for each of a chunk's four matrix steps, so that one load covers 64 contiguous
// bytes of 16 rows (with 32 consecutive values per lane each load touched 64 pieces of 64 bytes, and
// the address unit bound the kernel).  The factor rows are the A operand, so a lane ends with 4
// consecutive r of one row.
template <typename D, int RT>
__global__ __launch_bounds__(shrink_waves(RT) * kWave) void hqq_adapter_shrink_kernel(const ShrinkParams P) {
  constexpr int kShrinkWaves = shrink_waves(RT);
  __shared__ float red[kShrinkWaves][RT * 4][kWave];
  __shared__ float wave_largest[kShrinkWaves];
  const ShrinkSide S = P.side[blockIdx.z];
  const RowTile t = find_row_tile(P.offsets, P.adapters, P.M, kShrinkRows, blockIdx.x);
  if (t.rows <= 0 || t.group == P.adapters) return;
  const int wid = threadIdx.x / kWave, lane = threadIdx.x & (kWave - 1);
  const int i = lane & 15, q = lane >> 4;
  const int32_t slot = P.order[t.row0 + (i < t.rows ? i : t.rows - 1)];
  const uint16_t* x = S.rows + slot * S.width;
  const uint16_t* f[RT];
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    const int r = 16 * j + i;
    f[j] = S.factor + ((int64_t)t.group * P.rank + (r < P.rank ? r : P.rank - 1)) * S.stride;
  }
  float4_t acc[RT];
#pragma unroll
  for (int j = 0; j < RT; ++j) acc[j] = (float4_t){0.f, 0.f, 0.f, 0.f};
  // The next chunk is in flight during this one's products (up to rank 16 its factors too: two sets
  // of registers); whole chunks take plain loads, the last one may end anywhere.
  const int64_t chunks = (S.width + 127) >> 7;
  constexpr int FD = RT <= 1 ? 2 : 1;
  short8_t xv[2][4], fv[FD][4][RT];
  auto load_x = [&](int64_t c, short8_t (&o)[4]) {
    const int64_t k = c * 128 + 8 * q;
    if ((c + 1) * 128 <= S.width) {  // uniform
#pragma unroll
      for (int s = 0; s < 4; ++s) __builtin_memcpy(&o[s], x + k + 32 * s, 16);
    } else {
#pragma unroll
      for (int s = 0; s < 4; ++s) o[s] = load8(x + k + 32 * s, S.width - k - 32 * s);
    }
  };
  auto load_f = [&](int64_t c, short8_t (&o)[4][RT]) {
    const int64_t k = c * 128 + 8 * q;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      // past the width (a stride holds it rounded up to 8): any values, X has zeros there; the row's first
      const int64_t at = k + 32 * s < S.width ? k + 32 * s : 0;
#pragma unroll
      for (int j = 0; j < RT; ++j) o[s][j] = *reinterpret_cast<const short8_t*>(f[j] + at);
    }
  };
  auto products = [&](const short8_t (&xo)[4], const short8_t (&fo)[4][RT]) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int j = 0; j < RT; ++j) acc[j] = D::mfma(fo[s][j], xo[s], acc[j]);
  };
  auto chunk = [&](int64_t c, int cur) {
    const int64_t cn = c + kShrinkWaves;
    if (cn < chunks) load_x(cn, xv[cur ^ 1]);
    if constexpr (FD == 2) {
      if (cn < chunks) load_f(cn, fv[cur ^ 1]);
      __builtin_amdgcn_sched_barrier(0);
      products(xv[cur], fv[cur]);
    } else {
      load_f(c, fv[0]);
      products(xv[cur], fv[0]);
    }
  };
  if (wid < chunks) {
    load_x(wid, xv[0]);
    if constexpr (FD == 2) load_f(wid, fv[0]);
    for (int64_t c = wid; c < chunks; c += 2 * kShrinkWaves) {
      chunk(c, 0);
      if (c + kShrinkWaves < chunks) chunk(c + kShrinkWaves, 1);
    }
  }
#pragma unroll
  for (int j = 0; j < RT; ++j)
#pragma unroll
    for (int v = 0; v < 4; ++v) red[wid][4 * j + v][lane] = acc[j][v];
  __syncthreads();
  float largest = 0.f;
  for (int j = wid; j < RT; j += kShrinkWaves) {
    float4_t sum;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      float y = red[0][4 * j + v][lane];
#pragma unroll
      for (int w = 1; w < kShrinkWaves; ++w) y += red[w][4 * j + v][lane];
      sum[v] = y;
    }
    const int r = 16 * j + 4 * q;
    if (i < t.rows && r < P.rank) {
      *reinterpret_cast<float4_t*>(S.out + (t.row0 + i) * P.rank + r) = sum;
#pragma unroll
      for (int v = 0; v < 4; ++v) largest = __builtin_fmaxf(largest, finite_abs(sum[v]));
    }
  }
  if (S.largest) {
#pragma unroll
    for (int o = kWave / 2; o > 0; o >>= 1) largest = __builtin_fmaxf(largest, __shfl_xor(largest, o, kWave));
    if (lane == 0) wave_largest[wid] = largest;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
      for (int w = 1; w < kShrinkWaves; ++w) largest = __builtin_fmaxf(largest, wave_largest[w]);
      S.largest[blockIdx.x] = largest;
    }
  }
}

struct ExpandParams {
  const float* low;         // M x rank, sorted
  const uint16_t* factor;   // adapters x width x rank
  const float* scales;
  const int32_t* order;
  const int32_t* offsets;
  const void* base;
  void* out;
  int64_t M, width;
  int rank, adapters, base_f32, out_f32;
};

constexpr int kExpandRows = 32;
constexpr int kExpandCols = 64;  // outputs per wavefront
constexpr int kExpandWaves = 4;

// Bound by HBM: 8190 x 4096 bfloat16 with a base, 134 MB and 4 MB of low in 47 us, 2.9 TB/s (rows are
// scattered in sorted order; row pieces of 64 bytes instead of 128 took 57-64 us).
//
// out = base + s low factor^T.  A block per 32 sorted rows of one adapter and 256 outputs; a
// wavefront keeps its 64 factor rows in registers for the tile's rows.  The factor rows are the
// A operand, and row 4 q + v of its tile t stands for output 16 q + 4 t + v of the 64, so a lane
// holds 16 consecutive outputs of one row: base and out move in 16-byte pieces, 64 outputs of a
// row together.
template <typename D, int RS, int PARTS>
__global__ __launch_bounds__(kExpandWaves * kWave) void hqq_adapter_expand_kernel(const ExpandParams P) {
  const RowTile t = find_row_tile(P.offsets, P.adapters, P.M, kExpandRows, blockIdx.y);
  if (t.rows <= 0) return;
  const int wid = threadIdx.x / kWave, lane = threadIdx.x & (kWave - 1);
  const int i = lane & 15, q = lane >> 4;
  const int64_t n0 = ((int64_t)blockIdx.x * kExpandWaves + wid) * kExpandCols;
  if (n0 >= P.width) return;  // wave-uniform; no barrier below
  const bool has = t.group < P.adapters;
  const bool whole = n0 + kExpandCols <= P.width;
  const float s = has ? P.scales[t.group] : 0.f;
  short8_t f[RS][4];
#pragma unroll
  for (int c = 0; c < RS; ++c)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t n = n0 + 16 * (i >> 2) + 4 * j + (i & 3);
      const int r = 32 * c + 8 * q;
      f[c][j] = (short8_t){};
      if (has && n < P.width && r < P.rank)
        f[c][j] = *reinterpret_cast<const short8_t*>(P.factor + ((int64_t)t.group * P.width + n) * P.rank + r);
    }
  const int64_t n = n0 + 16 * q;
  for (int m0 = 0; m0 < t.rows; m0 += 16) {
    const int m = m0 + i;
    const bool on = m < t.rows;
    // the base first: in flight during the products
    const int32_t o = P.order[t.row0 + (on ? m : 0)];
    const int64_t at = (int64_t)(o < 0 ? ~o : o) * P.width + n, left = P.width - n;
    float y[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) y[e] = 0.f;
    if (P.base && whole) {  // uniform
      if (P.base_f32) {
        __builtin_memcpy(y, static_cast<const float*>(P.base) + at, 64);
      } else {
        short8_t w[2];
        __builtin_memcpy(w, static_cast<const uint16_t*>(P.base) + at, 32);
#pragma unroll
        for (int e = 0; e < 16; ++e) y[e] = D::up((uint16_t)w[e >> 3][e & 7]);
      }
    } else if (P.base) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        if (e >= left) continue;
        y[e] = P.base_f32 ? static_cast<const float*>(P.base)[at + e] : D::up(static_cast<const uint16_t*>(P.base)[at + e]);
      }
    }
    float4_t acc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = (float4_t){0.f, 0.f, 0.f, 0.f};
    float back = s;
    if (has) {  // wave-uniform
      float4_t v[RS][2];
      float largest = 0.f;
#pragma unroll
      for (int c = 0; c < RS; ++c) {
        const int r = 32 * c + 8 * q;
        v[c][0] = v[c][1] = (float4_t){0.f, 0.f, 0.f, 0.f};
        if (on && r < P.rank) {
          const float4_t* p = reinterpret_cast<const float4_t*>(P.low + (t.row0 + m) * P.rank + r);
          v[c][0] = p[0];
          v[c][1] = p[1];
        }
        if constexpr (D::kScaled) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            largest = __builtin_fmaxf(largest, __builtin_fmaxf(finite_abs(v[c][0][e]), finite_abs(v[c][1][e])));
        }
      }
      float up = 1.f;
      if constexpr (D::kScaled) {
        largest = __builtin_fmaxf(largest, __shfl_xor(largest, 16, kWave));
        largest = __builtin_fmaxf(largest, __shfl_xor(largest, 32, kWave));
        const int x = scale_exponent(largest);
        up = exp2i(x);
        back = s * exp2i(-x);
      }
#pragma unroll
      for (int c = 0; c < RS; ++c) {
        short8_t part[PARTS];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          uint16_t h[PARTS];
          split<D>(up * v[c][e >> 2][e & 3], h);
#pragma unroll
          for (int p = 0; p < PARTS; ++p) part[p][e] = (short)h[p];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int p = 0; p < PARTS; ++p) acc[j] = D::mfma(f[c][j], part[p], acc[j]);
      }
    }
    if (!on || n >= P.width) continue;
    if (has) {
#pragma unroll
      for (int e = 0; e < 16; ++e) y[e] = __builtin_fmaf(back, acc[e >> 2][e & 3], y[e]);
    }
    if (P.out_f32) {
      float* p = static_cast<float*>(P.out) + at;
      if (left >= 16) {
        __builtin_memcpy(p, y, 64);
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (e < left) p[e] = y[e];
      }
    } else {
      uint16_t* p = static_cast<uint16_t*>(P.out) + at;
      uint16_t h[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) h[e] = D::down(y[e]);
      if (left >= 16) {
        __builtin_memcpy(p, h, 32);
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (e < left) p[e] = h[e];
      }
    }
  }
}

// ------------------------------------------------------------ the gradients --

struct TransposeParams {
  const uint16_t* A;        // adapters x rank x K -> At: adapters x K x rank
  uint16_t* At;
  const uint16_t* B;        // adapters x N x rank -> Bt: adapters x rank x Np, zeros behind N
  uint16_t* Bt;
  const int32_t* offsets;
  int64_t N, K, Np;
  int rank, adapters;
};

constexpr int kTransTile = 64;

// The used adapters' factors transposed, so that the gradients run the forward kernels with the
// factors' places swapped: 64 x 64 tiles through LDS; blockIdx.z 0: A, 1: B.
__global__ __launch_bounds__(kBlock) void hqq_adapter_transpose_kernel(const TransposeParams P) {
  __shared__ __align__(16) uint16_t tile[kTransTile][kTransTile + 8];  // [column][row]
  const int a = blockIdx.y;
  const bool of_b = blockIdx.z == 1;
  if (P.offsets[a + 1] == P.offsets[a]) return;
  const int64_t rows = of_b ? P.N : P.rank, cols = of_b ? P.rank : P.K;
  const int64_t stride = of_b ? P.Np : P.rank;  // of the output's rows
  const int64_t rt = (stride + kTransTile - 1) / kTransTile, ct = (cols + kTransTile - 1) / kTransTile;
  if (blockIdx.x >= rt * ct) return;
  const int64_t r0 = blockIdx.x / ct * kTransTile, c0 = blockIdx.x % ct * kTransTile;
  const uint16_t* in = (of_b ? P.B : P.A) + (int64_t)a * rows * cols;
  uint16_t* out = (of_b ? P.Bt : P.At) + (int64_t)a * cols * stride;
  // 16-byte pieces both ways (cols and stride are multiples of 8): piece x of row y, then y + 32
  const int x = threadIdx.x % 8, y = threadIdx.x / 8;
#pragma unroll
  for (int j = y; j < kTransTile; j += kBlock / 8) {
    const int64_t r = r0 + j, c = c0 + 8 * x;
    short8_t v = {};
    if (r < rows && c < cols) v = *reinterpret_cast<const short8_t*>(in + r * cols + c);
#pragma unroll
    for (int e = 0; e < 8; ++e) tile[8 * x + e][j] = (uint16_t)v[e];
  }
  __syncthreads();
#pragma unroll
  for (int j = y; j < kTransTile; j += kBlock / 8) {
    const int64_t c = c0 + j, r = r0 + 8 * x;
    if (c < cols && r < stride)
      *reinterpret_cast<short8_t*>(out + c * stride + r) = *reinterpret_cast<const short8_t*>(&tile[j][8 * x]);
  }
}

struct OuterSide {
  const uint16_t* rows;     // M x width (X or dY)
  const float* low;         // M x rank, sorted (u or v)
  const float* largest;     // of every tile of kShrinkRows rows
  float* out;               // dA: adapters x rank x width; dB: adapters x width x rank
  float* slabs;             // pieces x rank x width
  int64_t width;
  int64_t blocks;           // column blocks
};
struct OuterParams {
  OuterSide side[2];        // 0: dA, 1: dB
  const float* scales;
  const int32_t* order;
  const int32_t* offsets;
  int64_t M;
  int rank, adapters, piece;
};

constexpr int kOuterCols = 128;
constexpr int kOuterRows = 64;              // sorted rows per step
constexpr int kOuterD = kOuterCols + 16;    // halves per LDS row: 8 rows of a read cover the banks once
constexpr int outer_w(int rt) { return rt == 1 ? 16 : 16 * rt + 16; }

// Bound by the caches' bandwidth: 8190 x (4096 + 11008) bfloat16 at rank 16, 247 MB in 47 us, 5.3 TB/s
// right behind the first step, which has just read the rows (57 us later in the call).
//
// The sum over an adapter's rows of rows^T low: a block takes 128 columns and one piece (at most
// `piece` sorted rows) of one adapter, in steps of 64 rows staged in LDS as they are stored, and
// reads both operands with the transposing LDS read (the contraction runs over rows).  Within a
// step of 32 the lanes of quarter q take rows 4 q .. + 4 and 16 + 4 q .. + 4, so that one read's
// 8 rows (stride an odd multiple of 32 bytes) cover the banks once.  An adapter of one piece is
// written directly, else the piece's slab, added in order afterwards.
template <typename D, int RT>
__global__ __launch_bounds__(kBlock) void hqq_adapter_outer_kernel(const OuterParams P) {
  constexpr int PARTS = D::kParts, WS = outer_w(RT);
  __shared__ __align__(16) uint16_t Ds[kOuterRows][kOuterD];
  __shared__ __align__(16) uint16_t Ws[PARTS][kOuterRows][WS];
  const bool of_b = (int64_t)blockIdx.x >= P.side[0].blocks;
  const OuterSide S = P.side[of_b ? 1 : 0];
  const RowTile t = find_row_tile(P.offsets, P.adapters, P.M, P.piece, blockIdx.y);
  if (t.rows <= 0 || t.group == P.adapters) return;
  const int tid = threadIdx.x, wid = tid / kWave, lane = tid & (kWave - 1);
  const int i = lane & 15, q = lane >> 4;
  const int64_t c0 = ((int64_t)blockIdx.x - (of_b ? P.side[0].blocks : 0)) * kOuterCols;
  float up = 1.f, back = P.scales[t.group];
  if constexpr (D::kScaled) {
    // one power of two for the piece: its largest value (every wavefront finds the same)
    const GroupTiles tiles = find_group_tiles(P.offsets, P.M, kShrinkRows, t.group);
    const float* of_tile = S.largest + tiles.first + (int64_t)t.index * (P.piece / kShrinkRows);
    float largest = 0.f;
    for (int n = lane; n * kShrinkRows < t.rows; n += kWave) largest = __builtin_fmaxf(largest, of_tile[n]);
#pragma unroll
    for (int o = kWave / 2; o > 0; o >>= 1) largest = __builtin_fmaxf(largest, __shfl_xor(largest, o, kWave));
    const int x = scale_exponent(largest);
    up = exp2i(x);
    back *= exp2i(-x);
  }
  // the thread's share of a step: 16-byte column piece tid % 16 of rows tid / 16 + 16 j, and
  // RT pieces of four low-rank values
  const int dc = tid & 15, dr = tid >> 4;
  short8_t dv[4];
  float4_t wv[RT];
  auto load = [&](int m0) {
    const int64_t c = c0 + 8 * dc;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + dr + 16 * j;
      dv[j] = (short8_t){};
      if (m < t.rows) {
        const uint16_t* row = S.rows + P.order[t.row0 + m] * S.width;
        if (c0 + kOuterCols <= S.width) __builtin_memcpy(&dv[j], row + c, 16);  // uniform: whole pieces
        else dv[j] = load8(row + c, S.width - c);
      }
    }
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      const int e = (j * kBlock + tid) * 4, m = m0 + e / (16 * RT), r = e % (16 * RT);
      wv[j] = (float4_t){0.f, 0.f, 0.f, 0.f};
      if (m < t.rows && r < P.rank) wv[j] = *reinterpret_cast<const float4_t*>(S.low + (t.row0 + m) * P.rank + r);
    }
  };
  float4_t acc[2][RT];
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int j = 0; j < RT; ++j) acc[c][j] = (float4_t){0.f, 0.f, 0.f, 0.f};

  load(0);
  for (int m0 = 0; m0 < t.rows; m0 += kOuterRows) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j) *reinterpret_cast<short8_t*>(&Ds[dr + 16 * j][8 * dc]) = dv[j];
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      const int e = (j * kBlock + tid) * 4;
      short4_t part[PARTS];
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        uint16_t h[PARTS];
        split<D>(up * wv[j][v], h);
#pragma unroll
        for (int p = 0; p < PARTS; ++p) part[p][v] = (short)h[p];
      }
#pragma unroll
      for (int p = 0; p < PARTS; ++p)
        *reinterpret_cast<short4_t*>(&Ws[p][e / (16 * RT)][e % (16 * RT)]) = part[p];
    }
    __syncthreads();
    if (m0 + kOuterRows < t.rows) load(m0 + kOuterRows);
#pragma unroll
    for (int ks = 0; ks < kOuterRows / 32; ++ks) {
      const int row = 32 * ks + 4 * q + (i >> 2), col = 4 * (i & 3);
      auto read = [&](const uint16_t* src, int stride) -> short8_t {
        const short4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4*)src);
        const short4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4*)(src + 16 * stride));
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      };
      short8_t d[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) d[c] = read(&Ds[row][32 * wid + 16 * c + col], kOuterD);
#pragma unroll
      for (int j = 0; j < RT; ++j)
#pragma unroll
        for (int p = 0; p < PARTS; ++p) {
          const short8_t w = read(&Ws[p][row][16 * j + col], WS);
#pragma unroll
          for (int c = 0; c < 2; ++c) acc[c][j] = of_b ? D::mfma(w, d[c], acc[c][j]) : D::mfma(d[c], w, acc[c][j]);
        }
    }
  }

  const int64_t size = S.width * P.rank;
  float* out = t.group_rows <= P.piece ? S.out + t.group * size : S.slabs + (int64_t)blockIdx.y * size;
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      const float4_t y = acc[c][j] * back;
      if (of_b) {  // lane: column i of the tile, 4 consecutive r
        const int64_t col = c0 + 32 * wid + 16 * c + i;
        const int r = 16 * j + 4 * q;
        if (col < S.width && r < P.rank) *reinterpret_cast<float4_t*>(out + col * P.rank + r) = y;
      } else {     // lane: r = i of the tile, 4 consecutive columns (the width is a multiple of 8)
        const int64_t col = c0 + 32 * wid + 16 * c + 4 * q;
        const int r = 16 * j + i;
        if (col < S.width && r < P.rank) *reinterpret_cast<float4_t*>(out + r * S.width + col) = y;
      }
    }
}

// Adapters of no row: zeros.  Of more than one piece: the sum of their slabs in order.
__global__ __launch_bounds__(kBlock) void hqq_adapter_join_kernel(const OuterParams P) {
  const OuterSide S = P.side[blockIdx.z];
  const int a = blockIdx.y;
  const GroupTiles g = find_group_tiles(P.offsets, P.M, P.piece, a);
  if (g.count == 1) return;
  const int64_t size = S.width * P.rank;  // a multiple of 8
  for (int64_t e = ((int64_t)blockIdx.x * kBlock + threadIdx.x) * 4; e < size; e += (int64_t)gridDim.x * kBlock * 4) {
    float4_t y = {0.f, 0.f, 0.f, 0.f};
    for (int p = 0; p < g.count; ++p) y += *reinterpret_cast<const float4_t*>(S.slabs + (g.first + p) * size + e);
    *reinterpret_cast<float4_t*>(S.out + a * size + e) = y;
  }
}

// -------------------------------------------------------------------- host --

int64_t up256(int64_t b) { return (b + 255) & ~(int64_t)255; }

// A workspace laid out piece by piece, each 256-byte aligned.
struct Layout {
  char* base;
  int64_t used = 0;
  template <typename T>
  T* take(int64_t n) {
    T* p = reinterpret_cast<T*>(base + used);
    used += up256(n * (int64_t)sizeof(T));
    return p;
  }
};

struct SortedPlan {
  int32_t* order;
  int32_t* position;
  int32_t* offsets;
  int32_t* sort_ws;
  float* v;
  explicit SortedPlan(Layout& l, int64_t M, int rank, int adapters) {
    order = l.take<int32_t>(M);
    position = l.take<int32_t>(M);
    offsets = l.take<int32_t>(adapters + 1);
    sort_ws = l.take<int32_t>(route_sort_workspace_bytes(M, adapters) / 4);
    v = l.take<float>(M * rank);
  }
};

// Rows of one piece of the gradient sums: about 1024 blocks in all, 256 rows at least.
int64_t outer_piece(int64_t M, int64_t N, int64_t K) {
  const int64_t cols = (N + kOuterCols - 1) / kOuterCols + (K + kOuterCols - 1) / kOuterCols;
  const int64_t rows = (M * cols / 1024 + kOuterRows - 1) / kOuterRows * kOuterRows;
  return rows < 256 ? 256 : rows;
}

struct BackwardPlan {
  SortedPlan s;
  float* u;
  float* largest[2];        // of u and v
  uint16_t* At;
  uint16_t* Bt;
  float* slabs_a;
  float* slabs_b;
  int64_t Np, piece, pieces;
  BackwardPlan(Layout& l, int64_t M, int64_t N, int64_t K, int rank, int adapters) : s(l, M, rank, adapters) {
    Np = (N + 7) & ~(int64_t)7;
    piece = outer_piece(M, N, K);
    pieces = max_row_tiles(M, adapters, piece);
    u = l.take<float>(M * rank);
    for (float*& p : largest) p = l.take<float>(max_row_tiles(M, adapters, kShrinkRows));
    At = l.take<uint16_t>((int64_t)adapters * K * rank);
    Bt = l.take<uint16_t>((int64_t)adapters * Np * rank);
    const int64_t slabs = M > piece ? pieces : 0;  // (else every adapter is one piece)
    slabs_a = l.take<float>(slabs * rank * K);
    slabs_b = l.take<float>(slabs * rank * N);
  }
};

template <typename D>
hipError_t launch_shrink(const ShrinkParams& p, int sides, hipStream_t st) {
  const dim3 grid((unsigned)max_row_tiles(p.M, p.adapters, kShrinkRows), 1, (unsigned)sides), block(shrink_waves(p.rank <= 64 ? 4 : 16) * kWave);
  if (p.rank <= 16) hipLaunchKernelGGL((hqq_adapter_shrink_kernel<D, 1>), grid, block, 0, st, p);
  else if (p.rank <= 32) hipLaunchKernelGGL((hqq_adapter_shrink_kernel<D, 2>), grid, block, 0, st, p);
  else if (p.rank <= 64) hipLaunchKernelGGL((hqq_adapter_shrink_kernel<D, 4>), grid, block, 0, st, p);
  else if (p.rank <= 128) hipLaunchKernelGGL((hqq_adapter_shrink_kernel<D, 8>), grid, block, 0, st, p);
  else hipLaunchKernelGGL((hqq_adapter_shrink_kernel<D, 16>), grid, block, 0, st, p);
  return hipGetLastError();
}

template <typename D, int PARTS>
hipError_t launch_expand_parts(const ExpandParams& p, hipStream_t st) {
  constexpr int kCols = kExpandWaves * kExpandCols;
  const dim3 grid((unsigned)((p.width + kCols - 1) / kCols), (unsigned)max_row_tiles(p.M, p.adapters, kExpandRows));
  const dim3 block(kExpandWaves * kWave);
  if (p.rank <= 32) hipLaunchKernelGGL((hqq_adapter_expand_kernel<D, 1, PARTS>), grid, block, 0, st, p);
  else if (p.rank <= 64) hipLaunchKernelGGL((hqq_adapter_expand_kernel<D, 2, PARTS>), grid, block, 0, st, p);
  else if (p.rank <= 128) hipLaunchKernelGGL((hqq_adapter_expand_kernel<D, 4, PARTS>), grid, block, 0, st, p);
  else hipLaunchKernelGGL((hqq_adapter_expand_kernel<D, 8, PARTS>), grid, block, 0, st, p);
  return hipGetLastError();
}

template <typename D>
hipError_t launch_expand(const ExpandParams& p, hipStream_t st) {
  if constexpr (D::kParts != D::kPartsOut16) {
    if (p.out_f32) return launch_expand_parts<D, D::kParts>(p, st);
  }
  return launch_expand_parts<D, D::kPartsOut16>(p, st);
}

template <typename D>
hipError_t launch_outer(const OuterParams& p, hipStream_t st) {
  const dim3 grid((unsigned)(p.side[0].blocks + p.side[1].blocks), (unsigned)max_row_tiles(p.M, p.adapters, p.piece));
  const dim3 block(kBlock);
  if (p.rank <= 16) hipLaunchKernelGGL((hqq_adapter_outer_kernel<D, 1>), grid, block, 0, st, p);
  else if (p.rank <= 32) hipLaunchKernelGGL((hqq_adapter_outer_kernel<D, 2>), grid, block, 0, st, p);
  else if (p.rank <= 64) hipLaunchKernelGGL((hqq_adapter_outer_kernel<D, 4>), grid, block, 0, st, p);
  else if (p.rank <= 128) hipLaunchKernelGGL((hqq_adapter_outer_kernel<D, 8>), grid, block, 0, st, p);
  else hipLaunchKernelGGL((hqq_adapter_outer_kernel<D, 16>), grid, block, 0, st, p);
  return hipGetLastError();
}

int few_splits(int64_t K) { return (int)((K + kFewK - 1) / kFewK); }

template <typename D>
hipError_t launch_shrink_few(const AdapterParams& p, float* part, hipStream_t st) {
  const dim3 grid((unsigned)few_splits(p.K), (unsigned)p.M, (unsigned)((p.rank + kFewRank - 1) / kFewRank));
  hipLaunchKernelGGL((hqq_adapter_shrink_few_kernel<D>), grid, dim3(kBlock), 0, st, p, part);
  return hipGetLastError();
}

template <typename D>
hipError_t launch_expand_few(const AdapterParams& p, const float* part, hipStream_t st) {
  const dim3 grid((unsigned)((p.N + kFewN - 1) / kFewN), (unsigned)p.M);
  hipLaunchKernelGGL((hqq_adapter_expand_few_kernel<D>), grid, dim3(kFewN), 0, st, p, part, few_splits(p.K));
  return hipGetLastError();
}

// Sort and first step of the sorted path.
template <typename D>
hipError_t launch_sorted_shrink(const AdapterParams& p, const SortedPlan& w, hipStream_t st) {
  const hipError_t e = launch_route_sort(p.ids, p.M, p.adapters, w.order, w.position, w.offsets, w.sort_ws, st);
  if (e != hipSuccess) return e;
  ShrinkParams s = {};
  s.side[0] = {p.X, p.A, p.K, p.K, w.v, nullptr};
  s.order = w.order;
  s.offsets = w.offsets;
  s.M = p.M;
  s.rank = p.rank;
  s.adapters = p.adapters;
  return launch_shrink<D>(s, 1, st);
}

template <typename D>
hipError_t launch_forward(const AdapterParams& p, hipStream_t st) {
  if (p.M <= kFewRows) {
    float* part = static_cast<float*>(p.workspace);
    const hipError_t e = launch_shrink_few<D>(p, part, st);
    return e != hipSuccess ? e : launch_expand_few<D>(p, part, st);
  }
  Layout l{static_cast<char*>(p.workspace)};
  const SortedPlan w(l, p.M, p.rank, p.adapters);
  const hipError_t e = launch_sorted_shrink<D>(p, w, st);
  if (e != hipSuccess) return e;
  return launch_expand<D>({w.v, p.B, p.scales, w.order, w.offsets, p.base, p.out, p.M, p.N, p.rank,
                           p.adapters, p.base_f32, p.out_f32}, st);
}

// `t` null: dX is base + the low-rank product; else the weight's product `t` makes it with the low-rank
// product added (binary16).
template <typename D>
hipError_t launch_backward(const AdapterParams& p, MatmulTParams* t, hipStream_t st) {
  Layout l{static_cast<char*>(p.workspace)};
  const BackwardPlan w(l, p.M, p.N, p.K, p.rank, p.adapters);
  hipError_t e = launch_route_sort(p.ids, p.M, p.adapters, w.s.order, w.s.position, w.s.offsets, w.s.sort_ws, st);
  if (e != hipSuccess) return e;
  if (p.M > 0) {
    const auto tiles = [](int64_t n) { return (n + kTransTile - 1) / kTransTile; };
    const int64_t of_a = tiles(p.rank) * tiles(p.K), of_b = tiles(w.Np) * tiles(p.rank);
    TransposeParams tr = {p.A, w.At, p.B, w.Bt, w.s.offsets, p.N, p.K, w.Np, p.rank, p.adapters};
    const int64_t most = of_a > of_b ? of_a : of_b;
    hipLaunchKernelGGL(hqq_adapter_transpose_kernel, dim3((unsigned)(most > 0 ? most : 1), (unsigned)p.adapters, 2),
                       dim3(kBlock), 0, st, tr);
    ShrinkParams s = {};
    s.side[0] = {p.X, p.A, p.K, p.K, w.s.v, D::kScaled ? w.largest[1] : nullptr};
    s.side[1] = {p.dY, w.Bt, p.N, w.Np, w.u, D::kScaled ? w.largest[0] : nullptr};
    s.order = w.s.order;
    s.offsets = w.s.offsets;
    s.M = p.M;
    s.rank = p.rank;
    s.adapters = p.adapters;
    e = launch_shrink<D>(s, 2, st);
    if (e != hipSuccess) return e;
  }
  OuterParams o = {};
  const auto blocks = [](int64_t n) { return (n + kOuterCols - 1) / kOuterCols; };
  o.side[0] = {p.X, w.u, w.largest[0], p.dA, w.slabs_a, p.K, blocks(p.K)};
  o.side[1] = {p.dY, w.s.v, w.largest[1], p.dB, w.slabs_b, p.N, blocks(p.N)};
  o.scales = p.scales;
  o.order = w.s.order;
  o.offsets = w.s.offsets;
  o.M = p.M;
  o.rank = p.rank;
  o.adapters = p.adapters;
  o.piece = (int)w.piece;
  if (p.M > 0) {
    // right behind the first step, while the cache may still hold the rows it read
    e = launch_outer<D>(o, st);
    if (e != hipSuccess) return e;
    if (t) {
      t->low = {w.u, w.At, p.scales, p.ids, w.s.order, w.s.offsets, p.K, p.rank, p.adapters};
      e = launch_matmul_t(*t, st);
    } else {
      e = launch_expand<D>({w.u, w.At, p.scales, w.s.order, w.s.offsets, p.base, p.out, p.M, p.K, p.rank,
                            p.adapters, p.base_f32, p.out_f32}, st);
    }
    if (e != hipSuccess) return e;
  }
  const int64_t most_elems = (p.N > p.K ? p.N : p.K) * p.rank;
  int64_t jb = (most_elems + 4 * kBlock - 1) / (4 * kBlock);
  if (jb > 256) jb = 256;
  hipLaunchKernelGGL(hqq_adapter_join_kernel, dim3((unsigned)jb, (unsigned)p.adapters, 2), dim3(kBlock), 0, st, o);
  return hipGetLastError();
}

}  // namespace

int64_t adapters_workspace_bytes(int64_t M, int64_t N, int64_t K, int rank, int adapters) {
  if (M <= kFewRows) return up256(few_splits(K) * M * rank * (int64_t)sizeof(float));
  Layout l{nullptr};
  const SortedPlan w(l, M, rank, adapters);
  return l.used;
}

int64_t adapters_backward_workspace_bytes(int64_t M, int64_t N, int64_t K, int rank, int adapters) {
  Layout l{nullptr};
  const BackwardPlan w(l, M, N, K, rank, adapters);
  return l.used;
}

hipError_t launch_adapters(const AdapterParams& p, hipStream_t stream) {
  return p.dtype == 0 ? launch_forward<F16>(p, stream) : launch_forward<Bf16>(p, stream);
}

hipError_t launch_adapters_backward(const AdapterParams& p, hipStream_t stream) {
  return p.dtype == 0 ? launch_backward<F16>(p, nullptr, stream) : launch_backward<Bf16>(p, nullptr, stream);
}

// The workspace of a projection with adapters: the adapters' own, then the base in fp32 and the
// product's workspace (few rows), or the tiles' (more rows, backward).
int64_t matmul_adapters_workspace_bytes(const MatmulParams& q, const AdapterParams& p) {
  const int64_t own = adapters_workspace_bytes(p.M, p.N, p.K, p.rank, p.adapters);
  if (p.M > kFewRows) return own + group_gemm_workspace_bytes(p.M, p.N, p.K, p.adapters, true);
  return own + up256(p.M * p.N * (int64_t)sizeof(float)) +
         up256(matmul_workspace_bytes(p.M, p.N, p.K, q.nbits, q.group_size));
}

hipError_t launch_matmul_adapters(MatmulParams q, AdapterParams p, int cus, hipStream_t st) {
  q.X = p.X;
  q.M = p.M;
  if (p.M > kFewRows) {
    Layout l{static_cast<char*>(p.workspace)};
    const SortedPlan w(l, p.M, p.rank, p.adapters);
    const hipError_t e = launch_sorted_shrink<F16>(p, w, st);
    if (e != hipSuccess) return e;
    GroupGemmParams g = {};
    g.X = p.X;
    g.packed = q.packed;
    g.scale16 = q.scale16;
    g.zero16 = q.zero16;
    g.Y = p.out;
    g.M = p.M;
    g.N = p.N;
    g.K = p.K;
    g.nbits = q.nbits;
    g.group_shift = q.group_shift;
    g.out_f32 = p.out_f32;
    g.offsets = w.offsets;
    g.order = w.order;
    g.groups = p.adapters;
    g.topk = 1;
    g.low = {w.v, p.B, p.scales, p.ids, w.order, w.offsets, p.N, p.rank, p.adapters};
    g.slabs = l.take<float>(0);
    return launch_group_gemm(g, st);
  }
  Layout l{static_cast<char*>(p.workspace)};
  float* part = l.take<float>(few_splits(p.K) * p.M * p.rank);
  float* base = l.take<float>(p.M * p.N);
  hipError_t e = launch_shrink_few<F16>(p, part, st);
  if (e != hipSuccess) return e;
  if (matmul_adds_low(q)) {
    q.Y = p.out;
    q.out_f32 = p.out_f32;
    q.low = part;
    q.low_splits = few_splits(p.K);
    q.rank = p.rank;
    q.adapters = p.adapters;
    q.factor = p.B;
    q.ids = p.ids;
    q.scales = p.scales;
    return launch_matmul(q, cus, st);
  }
  q.Y = base;
  q.part = l.take<float>(0);
  MatmulBase b;
  e = launch_matmul_base(q, cus, &b, st);
  if (e != hipSuccess) return e;
  p.base = b.slabs > 0 ? q.part : base;
  p.base_f32 = 1;
  p.base_slabs = b.slabs;
  p.base_stride = b.stride;
  return launch_expand_few<F16>(p, part, st);
}

int64_t matmul_adapters_backward_workspace_bytes(const MatmulParams& q, const AdapterParams& p) {
  return adapters_backward_workspace_bytes(p.M, p.N, p.K, p.rank, p.adapters) +
         up256(matmul_t_workspace_bytes(p.M, p.N, p.K, 0));
}

hipError_t launch_matmul_adapters_backward(const MatmulParams& q, const AdapterParams& p, hipStream_t st) {
  MatmulTParams t = {};
  t.dY = p.dY;
  t.packed = q.packed;
  t.scale16 = q.scale16;
  t.zero16 = q.zero16;
  t.dX = p.out;
  t.M = p.M;
  t.N = p.N;
  t.K = p.K;
  t.nbits = q.nbits;
  t.group_size = q.group_size;
  t.group_shift = q.group_shift;
  t.out_f32 = p.out_f32;
  t.slabs = reinterpret_cast<float*>(static_cast<char*>(p.workspace) +
                                     adapters_backward_workspace_bytes(p.M, p.N, p.K, p.rank, p.adapters));
  return launch_backward<F16>(p, &t, st);
}

}  // namespace hqq
