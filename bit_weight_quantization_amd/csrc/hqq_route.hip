// hqq_route.hip -- gfx950 kernels that order the (token, choice) slots of a routed layer by
// expert, bring rows into that order, and bring them back with weights, with the gradient.
//
// Slot s = t topk + j is choice j of token t; ids outside [0, experts) are dropped.  The
// order is a stable counting sort: row i of the sorted rows is slot order[i], the kept slots
// by expert and then the dropped ones (as ~slot); position is its inverse (~row for dropped
// slots), so that every row and every slot is named exactly once and each kernel below
// writes every output element exactly once: no atomics on results, no separate clearing.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "hqq_internal.h"
#include "hqq_route.h"

namespace hqq {
namespace {

// The sort is bound by launches and latency: one block sorts up to 4096 slots in 3.3 us (2 slots) to
// 5 us (4096); beyond, a count and a sort launch: 11 us for 16384 slots of 8 experts, 16 us for 32760
// of 64.
constexpr int kSortWaves = 16;
constexpr int kSortBlock = kSortWaves * kWave;
constexpr int64_t kSortOneBlock = 4096;  // slots that one block sorts in one launch
constexpr int64_t kSortChunk = 2048;     // slots per block above that
constexpr int64_t kSortMaxBlocks = 512;  // every block reads every block's counts

struct SortParams {
  const int32_t* ids;
  int32_t* order;
  int32_t* position;
  int32_t* offsets;
  int32_t* counts;   // blocks x (experts + 1), or null (one block)
  int64_t slots;
  int64_t chunk;     // slots per block, a multiple of kSortBlock
  int experts;
  int bits;          // of experts (the dropped slots' key)
};

__device__ __forceinline__ int sort_key(const SortParams& P, int64_t s) {
  const int id = P.ids[s];
  return (uint32_t)id < (uint32_t)P.experts ? id : P.experts;
}

// Lanes of the wavefront with this lane's key (among `active` lanes): one ballot per key bit.
__device__ __forceinline__ uint64_t same_key(int key, int bits, uint64_t active) {
  uint64_t m = active;
  for (int b = 0; b < bits; ++b) {
    const uint64_t set = __ballot((key >> b) & 1);
    m &= (key >> b) & 1 ? set : ~set;
  }
  return m;
}

__global__ __launch_bounds__(kSortBlock) void hqq_route_count_kernel(const SortParams P) {
  __shared__ int32_t hist[kMaxExperts + 1];
  for (int e = threadIdx.x; e <= P.experts; e += kSortBlock) hist[e] = 0;
  __syncthreads();
  const int64_t s0 = (int64_t)blockIdx.x * P.chunk;
  const int64_t s1 = s0 + P.chunk < P.slots ? s0 + P.chunk : P.slots;
  for (int64_t s = s0 + threadIdx.x; s < s1; s += kSortBlock) atomicAdd(&hist[sort_key(P, s)], 1);
  __syncthreads();
  int32_t* out = P.counts + (int64_t)blockIdx.x * (P.experts + 1);
  for (int e = threadIdx.x; e <= P.experts; e += kSortBlock) out[e] = hist[e];
}

// Wavefront w of a block owns a contiguous part of the block's slots, so the sorted place of
// a slot is: its key's first row + the slots of that key in earlier blocks + in earlier
// wavefronts + earlier in its own wavefront.  The first three are prefix sums of counts, the
// last one the rank among the lanes of equal key (ballots), so the result is stable and
// does not depend on the order in which wavefronts run.
__global__ __launch_bounds__(kSortBlock) void hqq_route_sort_kernel(const SortParams P) {
  __shared__ int32_t next[kSortWaves][kMaxExperts + 1];  // counts, then next rows
  __shared__ int32_t scan[kSortWaves];
  const int tid = threadIdx.x, wid = tid / kWave, lane = tid & (kWave - 1);
  const int E = P.experts;
  for (int w = 0; w < kSortWaves; ++w)
    for (int e = tid; e <= E; e += kSortBlock) next[w][e] = 0;
  __syncthreads();
  const int64_t s0 = (int64_t)blockIdx.x * P.chunk;
  const int64_t s1 = s0 + P.chunk < P.slots ? s0 + P.chunk : P.slots;
  const int64_t per = P.chunk / kSortWaves;
  const int64_t w0 = s0 + wid * per;
  const int64_t w1 = w0 + per < s1 ? w0 + per : s1;
  for (int64_t s = w0 + lane; s < w1; s += kWave) atomicAdd(&next[wid][sort_key(P, s)], 1);
  __syncthreads();

  // thread e: the slots of expert e in this block, in all blocks, in the blocks before
  int32_t total = 0, before = 0;
  if (tid < E) {
    if (P.counts) {
      for (int b = 0; b < (int)gridDim.x; ++b) {
        const int32_t c = P.counts[(int64_t)b * (E + 1) + tid];
        total += c;
        before += b < (int)blockIdx.x ? c : 0;
      }
    } else {
      for (int w = 0; w < kSortWaves; ++w) total += next[w][tid];
    }
  }
  // exclusive sums of the totals over the experts
  int32_t inc = total;
  for (int o = 1; o < kWave; o <<= 1) {
    const int32_t v = __shfl_up(inc, o, kWave);
    if (lane >= o) inc += v;
  }
  if (lane == kWave - 1) scan[wid] = inc;
  __syncthreads();
  int32_t pre = 0, kept = 0;
  for (int w = 0; w < kSortWaves; ++w) {
    pre += w < wid ? scan[w] : 0;
    kept += scan[w];
  }
  const int32_t first = pre + inc - total;
  if (tid < E) {
    if (blockIdx.x == 0) P.offsets[tid] = first;
    int32_t at = first + before;
    for (int w = 0; w < kSortWaves; ++w) {
      const int32_t c = next[w][tid];
      next[w][tid] = at;
      at += c;
    }
  }
  if (tid == 0) {
    if (blockIdx.x == 0) P.offsets[E] = kept;
    int32_t at = kept;
    if (P.counts)
      for (int b = 0; b < (int)blockIdx.x; ++b) at += P.counts[(int64_t)b * (E + 1) + E];
    for (int w = 0; w < kSortWaves; ++w) {
      const int32_t c = next[w][E];
      next[w][E] = at;
      at += c;
    }
  }
  __syncthreads();

  for (int64_t sb = w0; sb < w1; sb += kWave) {  // wave-uniform
    const int64_t s = sb + lane;
    const bool on = s < w1;
    const int key = on ? sort_key(P, s) : 0;
    const uint64_t active = __ballot(on);
    const uint64_t m = same_key(key, P.bits, active);
    const int leader = m ? __builtin_ctzll(m) : lane;
    int32_t base = 0;
    if (on && lane == leader) base = atomicAdd(&next[wid][key], (int32_t)__builtin_popcountll(m));
    base = __shfl(base, leader, kWave);
    if (on) {
      const int32_t row = base + (int32_t)__builtin_popcountll(m & ((1ull << lane) - 1));
      const bool dropped = key == E;
      P.order[row] = dropped ? ~(int32_t)s : (int32_t)s;
      P.position[s] = dropped ? ~row : row;
    }
  }
}

// ------------------------------------------------------------------- rows --

struct F16 {
  using T = uint16_t;
  static __device__ __forceinline__ float up(uint16_t v) { return (float)__builtin_bit_cast(_Float16, v); }
  static __device__ __forceinline__ uint16_t down(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }
};
struct Bf16 {
  using T = uint16_t;
  static __device__ __forceinline__ float up(uint16_t v) { return __builtin_bit_cast(float, (uint32_t)v << 16); }
  static __device__ __forceinline__ uint16_t down(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
};
struct F32 {
  using T = float;
  static __device__ __forceinline__ float up(float v) { return v; }
  static __device__ __forceinline__ float down(float v) { return v; }
};

// V elements that move as one access: 16 bytes, or one element where the width or a pointer
// does not allow 16.
template <typename D, bool WIDE>
struct Chunk {
  static constexpr int V = WIDE ? 16 / (int)sizeof(typename D::T) : 1;
  typedef typename D::T vec __attribute__((ext_vector_type(V)));
  vec v;
  __device__ __forceinline__ void load(const typename D::T* p) {
    if constexpr (WIDE) v = *reinterpret_cast<const vec*>(p);
    else v[0] = *p;
  }
  __device__ __forceinline__ void store(typename D::T* p) const {
    if constexpr (WIDE) *reinterpret_cast<vec*>(p) = v;
    else *p = v[0];
  }
};

// A block per token: every row is read once and written to the topk places of its slots.
// Bound by HBM: tokens reads and slots writes of a row (8192 x 4096 binary16, topk 2: 201 MB in
// 33-35 us, 5.8 TB/s, a part of the writes still in the 256 MB cache)
template <typename D, bool WIDE>
__global__ __launch_bounds__(kBlock) void hqq_route_gather_kernel(const RouteRows P) {
  using T = typename D::T;
  using C = Chunk<D, WIDE>;
  T* out = static_cast<T*>(P.out);
  for (int64_t t = blockIdx.x; t < P.tokens; t += gridDim.x) {
    const T* in = static_cast<const T*>(P.in) + t * P.width;
    const int32_t* pos = P.position + t * P.topk;
    for (int64_t c = (int64_t)threadIdx.x * C::V; c < P.width; c += (int64_t)blockDim.x * C::V) {
      C x, zero;
      x.load(in + c);
      zero.v = (typename C::vec)(T)0;
      for (int j = 0; j < P.topk; ++j) {
        const int32_t p = pos[j];
        if (p >= 0) x.store(out + p * P.width + c);
        else zero.store(out + (int64_t)~p * P.width + c);  // a dropped slot's row
      }
    }
  }
}

constexpr int kTopkStep = 8;  // choices whose rows are read together

// A block per token: out[t] = sum over its kept choices of weight * row, in fp32 in the order
// of the choices, rounded once.  The rows of up to 8 choices are in flight together.  Bound by HBM:
// 8192 x 4096 binary16 of 2 choices, 201 MB in 48 us, 4.2 TB/s.
template <typename D, bool WIDE>
__global__ __launch_bounds__(kBlock) void hqq_route_combine_kernel(const RouteRows P) {
  using T = typename D::T;
  using C = Chunk<D, WIDE>;
  for (int64_t t = blockIdx.x; t < P.tokens; t += gridDim.x) {
    const T* in = static_cast<const T*>(P.in);
    T* out = static_cast<T*>(P.out) + t * P.width;
    const int32_t* pos = P.position + t * P.topk;
    const float* w = P.weights ? P.weights + t * P.topk : nullptr;
    for (int64_t c = (int64_t)threadIdx.x * C::V; c < P.width; c += (int64_t)blockDim.x * C::V) {
      float acc[C::V];
#pragma unroll
      for (int v = 0; v < C::V; ++v) acc[v] = 0.f;
      for (int j0 = 0; j0 < P.topk; j0 += kTopkStep) {
        C x[kTopkStep];
        int32_t p[kTopkStep];
        float wt[kTopkStep];
#pragma unroll
        for (int j = 0; j < kTopkStep; ++j) {
          p[j] = j0 + j < P.topk ? pos[j0 + j] : -1;
          wt[j] = p[j] >= 0 && w ? w[j0 + j] : 1.f;
          if (p[j] >= 0) x[j].load(in + p[j] * P.width + c);
        }
#pragma unroll
        for (int j = 0; j < kTopkStep; ++j) {
          if (p[j] >= 0) {
#pragma unroll
            for (int v = 0; v < C::V; ++v) acc[v] = __builtin_fmaf(wt[j], D::up(x[j].v[v]), acc[v]);
          }
        }
      }
      C y;
#pragma unroll
      for (int v = 0; v < C::V; ++v) y.v[v] = D::down(acc[v]);
      y.store(out + c);
    }
  }
}

// A block per token: for each kept choice the row's gradient weight * dOut[t] and the
// weight's gradient <dOut[t], row>; zeros for dropped ones.  The gradient is read once for 8
// choices, whose dot products meet in a fixed order (butterfly, then the wavefronts).  Bound by HBM:
// 4095 x 8192 bfloat16 of 8 choices, a tenth dropped, 1.09 GB in 213 us, 5.1 TB/s.
template <typename D, bool WIDE>
__global__ __launch_bounds__(kBlock) void hqq_route_combine_backward_kernel(const RouteRows P) {
  using T = typename D::T;
  using C = Chunk<D, WIDE>;
  __shared__ float part[kBlock / kWave][kTopkStep];
  const int wid = threadIdx.x / kWave, lane = threadIdx.x & (kWave - 1);
  const int waves = blockDim.x / kWave;
  const T* in = static_cast<const T*>(P.in);
  T* out = static_cast<T*>(P.out);
  for (int64_t t = blockIdx.x; t < P.tokens; t += gridDim.x) {
    const T* grad = static_cast<const T*>(P.grad) + t * P.width;
    const int32_t* pos = P.position + t * P.topk;
    for (int j0 = 0; j0 < P.topk; j0 += kTopkStep) {
      int32_t p[kTopkStep];
      float wt[kTopkStep], dot[kTopkStep];
#pragma unroll
      for (int j = 0; j < kTopkStep; ++j) {
        p[j] = j0 + j < P.topk ? pos[j0 + j] : -1;
        wt[j] = p[j] >= 0 && P.weights ? P.weights[t * P.topk + j0 + j] : 1.f;
        dot[j] = 0.f;
      }
      for (int64_t c = (int64_t)threadIdx.x * C::V; c < P.width; c += (int64_t)blockDim.x * C::V) {
        C g, x[kTopkStep];
        g.load(grad + c);
        if (P.dweights) {
#pragma unroll
          for (int j = 0; j < kTopkStep; ++j)
            if (p[j] >= 0) x[j].load(in + p[j] * P.width + c);
        }
#pragma unroll
        for (int j = 0; j < kTopkStep; ++j) {
          if (j0 + j >= P.topk) continue;
          C d;
          if (p[j] >= 0) {
#pragma unroll
            for (int v = 0; v < C::V; ++v) {
              const float gv = D::up(g.v[v]);
              d.v[v] = D::down(wt[j] * gv);
              if (P.dweights) dot[j] = __builtin_fmaf(gv, D::up(x[j].v[v]), dot[j]);
            }
            d.store(out + p[j] * P.width + c);
          } else {
            d.v = (typename C::vec)(T)0;
            d.store(out + (int64_t)~p[j] * P.width + c);
          }
        }
      }
      if (!P.dweights) continue;
#pragma unroll
      for (int j = 0; j < kTopkStep; ++j) {
#pragma unroll
        for (int o = kWave / 2; o > 0; o >>= 1) dot[j] += __shfl_xor(dot[j], o, kWave);
        if (lane == 0) part[wid][j] = dot[j];
      }
      __syncthreads();
      if ((int)threadIdx.x < kTopkStep && j0 + (int)threadIdx.x < P.topk) {
        float sum = 0.f;
        for (int w = 0; w < waves; ++w) sum += part[w][threadIdx.x];
        P.dweights[t * P.topk + j0 + threadIdx.x] = sum;
      }
      __syncthreads();
    }
  }
}

bool wide(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <typename D>
bool wide_rows(const RouteRows& p) {
  return p.width * sizeof(typename D::T) % 16 == 0 && wide(p.in) && wide(p.out) && wide(p.grad);
}

// Threads of a row: a wavefront at least, 256 at most.
int row_threads(int64_t width, int v) {
  const int64_t chunks = (width + v - 1) / v;
  if (chunks >= kBlock) return kBlock;
  return chunks <= kWave ? kWave : (int)((chunks + kWave - 1) / kWave) * kWave;
}

constexpr int64_t kRowBlocks = 1 << 22;

enum class Rows { kGather, kCombine, kBackward };

template <typename D, bool WIDE>
hipError_t launch_rows(const RouteRows& p, Rows what, hipStream_t st) {
  // (a grid may have 2^32 threads; blocks go on to further tokens)
  const dim3 grid((unsigned)(p.tokens < kRowBlocks ? p.tokens : kRowBlocks)), block(row_threads(p.width, Chunk<D, WIDE>::V));
  switch (what) {
    case Rows::kGather: hipLaunchKernelGGL((hqq_route_gather_kernel<D, WIDE>), grid, block, 0, st, p); break;
    case Rows::kCombine: hipLaunchKernelGGL((hqq_route_combine_kernel<D, WIDE>), grid, block, 0, st, p); break;
    default: hipLaunchKernelGGL((hqq_route_combine_backward_kernel<D, WIDE>), grid, block, 0, st, p); break;
  }
  return hipGetLastError();
}

template <typename D>
hipError_t launch_rows_d(const RouteRows& p, Rows what, hipStream_t st) {
  return wide_rows<D>(p) ? launch_rows<D, true>(p, what, st) : launch_rows<D, false>(p, what, st);
}

hipError_t launch_rows_any(const RouteRows& p, int dtype, Rows what, hipStream_t st) {
  switch (dtype) {
    case 0: return launch_rows_d<F16>(p, what, st);
    case 1: return launch_rows_d<Bf16>(p, what, st);
    default: return launch_rows_d<F32>(p, what, st);
  }
}

int64_t sort_chunk(int64_t slots) {
  const int64_t least = (slots + kSortMaxBlocks - 1) / kSortMaxBlocks;
  const int64_t chunk = least > kSortChunk ? least : kSortChunk;
  return (chunk + kSortBlock - 1) / kSortBlock * kSortBlock;
}

}  // namespace

int64_t route_sort_workspace_bytes(int64_t slots, int experts) {
  if (slots <= kSortOneBlock) return 0;
  const int64_t chunk = sort_chunk(slots);
  return (slots + chunk - 1) / chunk * (experts + 1) * (int64_t)sizeof(int32_t);
}

hipError_t launch_route_sort(const int32_t* ids, int64_t slots, int experts, int32_t* order,
                             int32_t* position, int32_t* offsets, int32_t* workspace,
                             hipStream_t stream) {
  SortParams p;
  p.ids = ids;
  p.order = order;
  p.position = position;
  p.offsets = offsets;
  p.slots = slots;
  p.experts = experts;
  p.bits = 32 - __builtin_clz((unsigned)experts);
  p.counts = nullptr;
  p.chunk = kSortOneBlock;
  int64_t blocks = 1;
  if (slots > kSortOneBlock) {
    p.chunk = sort_chunk(slots);
    p.counts = workspace;
    blocks = (slots + p.chunk - 1) / p.chunk;
    hipLaunchKernelGGL(hqq_route_count_kernel, dim3((unsigned)blocks), dim3(kSortBlock), 0, stream, p);
  }
  hipLaunchKernelGGL(hqq_route_sort_kernel, dim3((unsigned)blocks), dim3(kSortBlock), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_route_gather(const RouteRows& p, int dtype, hipStream_t stream) {
  return launch_rows_any(p, dtype, Rows::kGather, stream);
}

hipError_t launch_route_combine(const RouteRows& p, int dtype, hipStream_t stream) {
  return launch_rows_any(p, dtype, Rows::kCombine, stream);
}

hipError_t launch_route_combine_backward(const RouteRows& p, int dtype, hipStream_t stream) {
  return launch_rows_any(p, dtype, Rows::kBackward, stream);
}

}  // namespace hqq
