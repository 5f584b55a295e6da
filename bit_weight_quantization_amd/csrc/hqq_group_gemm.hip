// hqq_group_gemm.hip -- gfx950 kernels of the tiled products of sorted rows with quantized
// weights, Y[i] = X[i] Q^-1(W)^T: with every expert's own weight, or with one weight and every
// adapter's low-rank product added to the same accumulators.
//
// A block's four wavefronts share 32 TI rows of X through LDS, and each takes 32 TJ weight rows
// of its own: it decodes its codes straight into the matrix operand (no LDS for the weight, and
// no weight is decoded twice in a block), so an LDS read feeds TJ matrix instructions.
//
// Bound by the matrix cores, the decoding and the power they draw together: 4096 rows of 8 experts of
// 11008 x 4096 (4 bits, g = 64) in 500 us, 740 TFLOP/s at about 2.0 GHz; without the loads of X, without
// those of the codes or without the decoding it is 10-18% faster each.  Tiles as the shared-weight kernel
// has them, 64 x 64 per wavefront with both operands in LDS, took 650 us.  256 rows (spills), 8 wavefronts
// of 128 x 512 and three buffers of X took 520 us.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "hqq_codes.h"
#include "hqq_group_gemm.h"
#include "hqq_internal.h"
#include "hqq_tiles.h"

namespace hqq {
namespace {

constexpr int kGK = 64;            // k per step
constexpr int kGRow = kGK + 8;     // halves per LDS row of X (rows 4 banks apart)
constexpr int kGWaves = 4;
constexpr int kGSlots = 64;        // blocks of an XCD at a time: two per CU
constexpr int kGUnit = 512;        // unit of splitting k: whole tables of scales for every group size
constexpr int kGTables = 4;        // ring of the scales' LDS tables, of 4 groups each

// Lane i + 32 h holds, per step of 64, the values 32 h .. + 32 of row i of both operands; the
// four matrix steps (v_mfma_f32_32x32x16_f16) take 8 of them each, the instruction's k order
// being the same for both.  The weight is the A operand and row 8 a + 4 h + b of tile j stands
// for weight row 32 h + 16 j + 4 a + b (TJ = 2) of the wavefront's, so that a lane ends with 16 TJ
// consecutive outputs of one row of X.  X goes through LDS one step ahead, double-buffered; codes
// and X are loaded a step ahead in registers, two wavefronts per SIMD.
template <int NB, int TI, int TJ, bool G16, bool ADAPTERS>
__global__ __launch_bounds__(kGWaves * kWave) __attribute__((amdgpu_waves_per_eu(2)))
void hqq_group_gemm_kernel(const GroupGemmParams P) {
  constexpr int BM = 32 * TI;
  constexpr int T = kGWaves * kWave;
  constexpr int XP = BM * kGK / 8 / T;      // 16-byte pieces of X per thread and step
  constexpr int XT = T / (kGK / 8);         // rows of X per round of loads
  static_assert(XP >= 1 && XP * T * 8 == BM * kGK && 4 * TJ % TI == 0, "a piece per thread at least, decoding in whole pairs");
  constexpr int BN = 32 * TJ * kGWaves;     // weight rows: one per thread
  static_assert(BN == T, "a thread loads the scales of one weight row");
  __shared__ __align__(16) _Float16 As[2][BM][kGRow];
  __shared__ uint32_t Sz[kGTables][4][BN];   // s and z (binary16) of the block's rows
  const int64_t cols = (P.N + BN - 1) / BN;
  const int units = (int)((P.K + kGUnit - 1) / kGUnit);
  const int64_t tiles = ADAPTERS ? (P.M + BM - 1) / BM : count_row_tiles(P.offsets, P.groups, P.M, BM);
  const TilePlace place = place_tile(blockIdx.x, tiles, cols, units, kGSlots, P.xcd_slabs);
  if (place.tile < 0) return;
  RowTile t;
  if constexpr (ADAPTERS) {  // tiles of the sorted rows, across adapters
    t.group = 0;
    t.row0 = place.tile * BM;
    t.rows = (int)(P.M - t.row0 < BM ? P.M - t.row0 : BM);
  } else {
    t = find_row_tile(P.offsets, P.groups, P.M, BM, place.tile);
    if (t.rows <= 0) return;
  }
  const int tid = threadIdx.x;
  const int wid = __builtin_amdgcn_readfirstlane(tid / kWave), lane = tid & (kWave - 1);
  const int i = lane & 31, h = lane >> 5;
  const int64_t n0 = place.col * BN + wid * (32 * TJ);
  // fragments of 32 rows that hold any (none in a wavefront past the last weight row)
  const int used = n0 < P.N ? (t.rows + 31) >> 5 : 0;
  const bool none = !ADAPTERS && t.group == P.groups;
  const int64_t w0 = ADAPTERS || none ? 0 : (int64_t)t.group * P.N;
  const int K = none ? 0 : (int)P.K;  // rows of no expert: zeros
  // the block's part of the inner size, in whole units
  const int kfirst = units * place.part / place.parts * kGUnit;
  const int kend = units * (place.part + 1) / place.parts * kGUnit;
  const int klast = kend < K ? kend : K;
  const int64_t row_bytes = (P.K >> 3) * NB, gpr = P.K >> P.group_shift;

  // rows past the tile read its last row; weight rows past N the last one (results not stored)
  const int xp = tid & 7, xr = tid >> 3;
  const uint16_t* xrow[XP];
#pragma unroll
  for (int p = 0; p < XP; ++p) {
    const int m = xr + XT * p;
    const int64_t row = t.row0 + (m < t.rows ? m : t.rows - 1);
    int64_t src = row;
    if constexpr (ADAPTERS) {
      const int32_t o = P.order[row];
      src = o < 0 ? ~o : o;
    } else if (P.order) {
      src = P.order[row] / P.topk;
      if (src < 0) src = 0;  // (rows of no expert read nothing)
    }
    xrow[p] = P.X + src * P.K;
  }
  // the wavefront's first weight row, and the lane's rows as 32-bit offsets from it (64 rows of
  // K <= 2^24 codes)
  const int64_t wave_row = w0 + (n0 < P.N ? n0 : P.N - 1);
  const uint8_t* wbase = P.packed + wave_row * row_bytes;
  uint32_t woff[TJ];
  int srow[TJ];  // the lane's rows in the scales' table
#pragma unroll
  for (int j = 0; j < TJ; ++j) {
    const int r = 16 * TJ * ((i >> 2) & 1) + 16 * j + 4 * (i >> 3) + (i & 3);
    srow[j] = wid * (32 * TJ) + r;
    woff[j] = (uint32_t)(w0 + (n0 + r < P.N ? n0 + r : P.N - 1) - wave_row) * (uint32_t)row_bytes;
  }
  const int64_t trow = place.col * BN + tid;
  const int64_t sfirst = (w0 + (trow < P.N ? trow : P.N - 1)) * gpr;
  // The scales of 4 groups of a row are 8 contiguous bytes, loaded at once by the row's thread two
  // tables ahead and put into LDS a step later.  (Loaded by the lanes that decode, step by step, each
  // 2-byte load touched 32 lines and the address unit bound the kernel: 1147 instead of 601 us for
  // 4096 rows, 8 experts of 11008 x 4096.)  The load stays inside the arrays: at their end it starts
  // earlier and is shifted back.
  const int tk = 4 << P.group_shift;  // k of a table
  const int64_t sgroups = (ADAPTERS ? P.N : P.N * P.groups) * gpr;
  uint64_t s4, z4;
  auto load_scales = [&](int k0) {
    const int64_t want = sfirst + (k0 < K ? k0 >> P.group_shift : 0);
    if (sgroups >= 4) {  // uniform
      const int64_t at = want < sgroups - 4 ? want : sgroups - 4;
      __builtin_memcpy(&s4, P.scale16 + at, 8);
      __builtin_memcpy(&z4, P.zero16 + at, 8);
      const int shift = 16 * (int)(want - at);
      s4 >>= shift;
      z4 >>= shift;
    } else {             // a weight of less than four groups in all
      s4 = z4 = 0;
      for (int e = 0; e < 4; ++e) {
        const int64_t at = want + e < sgroups ? want + e : sgroups - 1;
        s4 |= (uint64_t)P.scale16[at] << (16 * e);
        z4 |= (uint64_t)P.zero16[at] << (16 * e);
      }
    }
  };
  auto write_scales = [&](int k0) {
    const int table = (k0 >> (P.group_shift + 2)) & (kGTables - 1);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      Sz[table][c][tid] = ((uint32_t)(s4 >> (16 * c)) & 0xffffu) | ((uint32_t)(z4 >> (16 * c)) << 16);
    }
  };

  uint4 xv[XP];
  struct Codes {
    uint32_t w[TJ][NB];
  };
  auto load_x = [&](int k0) {
    const int k = k0 + 8 * xp;
#pragma unroll
    for (int p = 0; p < XP; ++p) xv[p] = *reinterpret_cast<const uint4*>(xrow[p] + (k < K ? k : 0));
  };
  auto write_x = [&](int buf, int k0) {
    if (k0 + kGK > K && k0 + 8 * xp >= K) {  // the last step's upper half
#pragma unroll
      for (int p = 0; p < XP; ++p) xv[p] = make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int p = 0; p < XP; ++p) *reinterpret_cast<uint4*>(&As[buf][xr + XT * p][8 * xp]) = xv[p];
  };
  auto load_codes = [&](int k0, Codes& c) {
    const uint32_t kk = k0 + 32 * h < K ? k0 + 32 * h : 0;  // K is a multiple of 32
#pragma unroll
    for (int j = 0; j < TJ; ++j) load_codes32<NB>(wbase + (uint64_t)(woff[j] + (kk >> 5) * (4 * NB)), c.w[j]);
  };

  float16_t acc[TI][TJ];
#pragma unroll
  for (int a = 0; a < TI; ++a)
#pragma unroll
    for (int j = 0; j < TJ; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[a][j][v] = 0.f;

  // the lane's scales of the step at k0: of codes 0-15 and 16-31 (different groups only when g = 16)
  struct Scales {
    PairScale p[TJ][2];
  };
  auto read_scales = [&](int k0, Scales& o) {
    const int g = (k0 + 32 * h) >> P.group_shift;
    auto scales = [&](uint32_t v) -> PairScale {
      const float f = h2f(v & 0xffffu);
      return {f * kSub, -f * h2f(v >> 16)};
    };
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      o.p[j][0] = scales(Sz[(g >> 2) & (kGTables - 1)][g & 3][srow[j]]);
      o.p[j][1] = G16 ? scales(Sz[(g >> 2) & (kGTables - 1)][(g & 3) + 1][srow[j]]) : o.p[j][0];
    }
    if (k0 + kGK > K && k0 + 32 * h >= K) {  // the last step's upper half: weights of zero
#pragma unroll
      for (int j = 0; j < TJ; ++j) o.p[j][0] = o.p[j][1] = {0.f, 0.f};
    }
  };
  uint32_t wf[2][TJ][4];  // decoded weights of a matrix step and of the next one
  // One step: the loads of the next one first, then 4 matrix steps of TI slots each.  A slot is the
  // products of one X fragment, the read of the fragment that takes its place one matrix step later
  // (4 slots ahead: the products between cover the LDS latency) and a slice of the decoding of the
  // next matrix step's weights (after the last one, of the next step's first); the scheduling
  // barriers keep this order.
  auto step = [&](int buf, int k0, const Codes& cur, Codes& nxt, const Scales& sc, Scales& sn) {
    const int kn = k0 + kGK < klast ? k0 + kGK : kfirst;  // (past the end: unused)
    half8_t xf[TI];
    auto read_x = [&](int s, int a) {
      xf[a] = *reinterpret_cast<const half8_t*>(&As[buf][32 * a + i][32 * h + 8 * s]);
    };
#pragma unroll
    for (int a = 0; a < TI; ++a)
      if (a < used) read_x(0, a);
    load_x(kn);
    load_codes(kn, nxt);
    const bool refill = (k0 & (tk - 1)) == 0;  // a new table began: load the one after the next
    if (refill) load_scales(k0 + 2 * tk);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (s == 2) read_scales(kn, sn);  // (its table was written a barrier ago at least)
      mfma_distance();
#pragma unroll
      for (int a = 0; a < TI; ++a) {
        if (a < used) {  // uniform: fragments of rows past the tile's cost nothing
#pragma unroll
          for (int j = 0; j < TJ; ++j)
            acc[a][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
                __builtin_bit_cast(half8_t, make_uint4(wf[s & 1][j][0], wf[s & 1][j][1], wf[s & 1][j][2], wf[s & 1][j][3])),
                xf[a], acc[a][j], 0, 0, 0);
          if (s < 3) read_x(s + 1, a);
        }
#pragma unroll
        for (int q = a * (4 * TJ / TI); q < (a + 1) * (4 * TJ / TI); ++q) {
          const int j = q % TJ, e = q / TJ;
          wf[(s + 1) & 1][j][e] = s < 3 ? decode_pair<NB>(cur.w[j], s + 1, e, sc.p[j][(s + 1) >> 1])
                                        : decode_pair<NB>(nxt.w[j], 0, e, sn.p[j][0]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    write_x(buf ^ 1, k0 + kGK);
    if (refill) write_scales(k0 + 2 * tk);
    lds_barrier();
  };
  if (kfirst < klast) {
    Codes ca, cb;
    Scales sa, sb;
    load_x(kfirst);
    load_codes(kfirst, ca);
    load_scales(kfirst);
    write_x(0, kfirst);
    write_scales(kfirst);
    load_scales(kfirst + tk);
    write_scales(kfirst + tk);
    lds_barrier();
    read_scales(kfirst, sa);
#pragma unroll
    for (int j = 0; j < TJ; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) wf[0][j][e] = decode_pair<NB>(ca.w[j], 0, e, sa.p[j][0]);
    int k0 = kfirst;
    for (; k0 + kGK < klast; k0 += 2 * kGK) {
      step(0, k0, ca, cb, sa, sb);
      step(1, k0 + kGK, cb, ca, sb, sa);
    }
    if (k0 < klast) step(0, k0, ca, cb, sa, sb);
  }

  float back[TI];
#pragma unroll
  for (int a = 0; a < TI; ++a) back[a] = 1.f;
  if constexpr (ADAPTERS) {
    static_assert(low_halves(BM) <= 2 * BM * kGRow, "the parts fit the X buffers");
    if (place.part == 0) {
      __shared__ float scale_up[BM];
      __shared__ int row_group[BM];
      int64_t col[TJ];
#pragma unroll
      for (int j = 0; j < TJ; ++j) col[j] = n0 + 16 * TJ * ((i >> 2) & 1) + 16 * j + 4 * (i >> 3) + (i & 3);
      add_low<BM, T>(acc, back, P.low, t.row0, t.rows, 0, col, &As[0][0][0], scale_up, row_group);
    }
  }

  // lane: row 32 a + i of the tile, outputs n0 + 16 TJ h .. + 16 TJ (element 4 a' + b of tile j:
  // register 4 a' + b)
  const int64_t n = n0 + 16 * TJ * h;
#pragma unroll
  for (int a = 0; a < TI; ++a) {
    const int m = 32 * a + i;
    if (place.parts > 1) {  // a part of the sum (rows past the tile too: the slab is the block's own)
      float* y = P.slabs + ((int64_t)place.slot * BM + m) * BN + wid * (32 * TJ) + 16 * TJ * h;
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        float v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = back[a] * acc[a][j][e];
        __builtin_memcpy(y + 16 * j, v, 64);
      }
      continue;
    }
    if (m >= t.rows || n >= P.N) continue;
    int64_t row = t.row0 + m;
    if constexpr (ADAPTERS) {
      const int32_t o = P.order[row];
      row = o < 0 ? ~o : o;
    }
    const int64_t at = row * P.N + n, left = P.N - n;
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      if (P.out_f32) {
        float* y = static_cast<float*>(P.Y) + at + 16 * j;
        float v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = back[a] * acc[a][j][e];
        if (left >= 16 * (j + 1)) {
          __builtin_memcpy(y, v, 64);
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (16 * j + e < left) y[e] = v[e];
        }
      } else {
        _Float16* y = static_cast<_Float16*>(P.Y) + at + 16 * j;
        _Float16 v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = (_Float16)(back[a] * acc[a][j][e]);
        if (left >= 16 * (j + 1)) {
          __builtin_memcpy(y, v, 32);
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (16 * j + e < left) y[e] = v[e];
        }
      }
    }
  }
}

// Tiles that were split: the sum of their parts in order.  A block per split tile and 4 rows.
constexpr int kJoinRows = 4;
template <int TI, bool ADAPTERS>
__global__ __launch_bounds__(64 * kGWaves) void hqq_group_gemm_join_kernel(const GroupGemmParams P) {
  constexpr int BM = 32 * TI, BN = 64 * kGWaves;  // a thread per column
  const int64_t cols = (P.N + BN - 1) / BN;
  const int64_t tiles = ADAPTERS ? (P.M + BM - 1) / BM : count_row_tiles(P.offsets, P.groups, P.M, BM);
  const int xcd = blockIdx.x % kXcds, rest = blockIdx.x / kXcds;
  const TileShare s = tile_share(xcd, tiles * cols, (int)((P.K + kGUnit - 1) / kGUnit), kGSlots);
  if (rest >= s.rest || (rest + 1) * s.parts > P.xcd_slabs) return;
  const TilePlace place = place_at(s.first + s.full + rest, tiles, cols);
  int64_t row0 = place.tile * BM;
  int rows = (int)(P.M - row0 < BM ? P.M - row0 : BM);
  if constexpr (!ADAPTERS) {
    const RowTile t = find_row_tile(P.offsets, P.groups, P.M, BM, place.tile);
    row0 = t.row0;
    rows = t.rows;
  }
  const int64_t n = place.col * BN + threadIdx.x;
  if (n >= P.N) return;
  const float* slab = P.slabs + (int64_t)(xcd * P.xcd_slabs + rest * s.parts) * BM * BN + threadIdx.x;
  for (int m = blockIdx.y * kJoinRows; m < (int)(blockIdx.y + 1) * kJoinRows && m < rows; ++m) {
    float part[kMaxParts];
#pragma unroll
    for (int p = 0; p < kMaxParts; ++p) part[p] = p < s.parts ? slab[((int64_t)p * BM + m) * BN] : 0.f;
    float y = part[0];
#pragma unroll
    for (int p = 1; p < kMaxParts; ++p) y += part[p];
    int64_t row = row0 + m;
    if constexpr (ADAPTERS) {
      const int32_t o = P.order[row];
      row = o < 0 ? ~o : o;
    }
    if (P.out_f32) static_cast<float*>(P.Y)[row * P.N + n] = y;
    else static_cast<_Float16*>(P.Y)[row * P.N + n] = (_Float16)y;
  }
}

// 128 rows a tile where the groups' mean reaches beyond 64, else 64 (a group of up to 64 rows would
// leave half of a 128-row tile's matrix instructions empty and pay for its registers all the same).
bool tall_tiles(int64_t M, int64_t groups) { return M / groups > 64; }
int64_t most_tiles(int64_t M, int64_t N, int64_t groups, bool adapters, int64_t bm) {
  return (N + 64 * kGWaves - 1) / (64 * kGWaves) * (adapters ? (M + bm - 1) / bm : max_row_tiles(M, groups, bm));
}

// Whether tiles may be split (adapters: whether any is; experts' tiles are counted on the device; one
// unit of k is never split).
bool tiles_split(int64_t M, int64_t N, int64_t K, int64_t groups, bool adapters, int64_t bm) {
  const int64_t units = (K + kGUnit - 1) / kGUnit;
  if (units <= 1) return false;
  return !adapters || place_splits(most_tiles(M, N, groups, true, bm), (int)(units < kMaxParts ? units : kMaxParts), kGSlots);
}

template <int NB, int TI, bool ADAPTERS>
hipError_t launch_tile(GroupGemmParams p, hipStream_t st) {
  const int64_t most = most_tiles(p.M, p.N, p.groups, ADAPTERS, 32 * TI), blocks = place_blocks(most, kGSlots);
  p.xcd_slabs = place_slabs(most, kGSlots);
  if (blocks * kGWaves * kWave > UINT32_MAX) return hipErrorInvalidValue;  // threads of a grid
  const dim3 grid((unsigned)blocks), block(kGWaves * kWave);
  if (p.group_shift == 4) hipLaunchKernelGGL((hqq_group_gemm_kernel<NB, TI, 2, true, ADAPTERS>), grid, block, 0, st, p);
  else hipLaunchKernelGGL((hqq_group_gemm_kernel<NB, TI, 2, false, ADAPTERS>), grid, block, 0, st, p);
  if (tiles_split(p.M, p.N, p.K, p.groups, ADAPTERS, 32 * TI)) {  // (split tiles: at most half of an XCD's slots)
    const dim3 join(kXcds * kGSlots / 2, 32 * TI / kJoinRows);
    hipLaunchKernelGGL((hqq_group_gemm_join_kernel<TI, ADAPTERS>), join, dim3(64 * kGWaves), 0, st, p);
  }
  return hipGetLastError();
}

template <int NB>
hipError_t launch_nb(const GroupGemmParams& p, hipStream_t st) {
  if (p.low.low) return launch_tile<NB, 4, true>(p, st);
  return tall_tiles(p.M, p.groups) ? launch_tile<NB, 4, false>(p, st) : launch_tile<NB, 2, false>(p, st);
}

}  // namespace

int64_t group_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t groups, bool adapters) {
  const int64_t bm = adapters || tall_tiles(M, groups) ? 128 : 64;
  if (!tiles_split(M, N, K, groups, adapters, bm)) return 0;
  return (int64_t)kXcds * place_slabs(most_tiles(M, N, groups, adapters, bm), kGSlots) * bm * 64 * kGWaves *
         (int64_t)sizeof(float);
}

hipError_t launch_group_gemm(GroupGemmParams p, hipStream_t stream) {
  switch (p.nbits) {
    case 2: return launch_nb<2>(p, stream);
    case 3: return launch_nb<3>(p, stream);
    case 4: return launch_nb<4>(p, stream);
    case 8: return launch_nb<8>(p, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace hqq
