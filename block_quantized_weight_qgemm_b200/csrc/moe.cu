// moe.cu -- routed tokens: the rows that qgemm_moe_* and qgemm_i8_moe_* read, sorted by expert,
// the way back with the routing weights applied, and the gradients of both (sm_100a).
//
// With slot s = t k + j and e_s its expert (a slot whose expert is outside [0, E) is dropped):
//   row[s]     = #{valid s' : e_s' < e_s} + #{s' < s : e_s' = e_s},   offsets[e] = #{valid s : e_s < e}
//   dispatch   xs[row[s]] = x[t]                       its gradient  dx[t] = sum_j dxs[row[t][j]]
//   combine    y[t] = sum_j w[t][j] ys[row[t][j]]      its gradient  dys[row[s]] = w[s] dy[t],
//                                                                    dw[s] = <dy[t], ys[row[s]]>
// Ranks are counts of integers (no float, no order of arrival), and every float sum runs in a
// fixed order in fp32, so results are the same from call to call.  All of it is bound by memory
// or, for few slots, by the launch.
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "ptx.cuh"

namespace qg {

// ---------------------------------------------------------------------------------------
// Launch helper: every kernel here is a programmatic dependent of what precedes it.  Each waits
// for that grid before it touches memory, and only then lets its own dependents launch.
// ---------------------------------------------------------------------------------------
template <typename... P, typename... A>
static cudaError_t launch_dep(void (*kern)(P...), dim3 grid, dim3 block, size_t smem,
                              cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// ---------------------------------------------------------------------------------------
// Sort
// ---------------------------------------------------------------------------------------
constexpr int kSortThreads = 256;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortChunk = 1024;   // slots per block, while that needs at most kSortBlocks blocks
constexpr int kSortBlocks = 148;

struct SortParams {
  const int* ids;  // [S]
  int S, E, nb, chunk;
  int* hist;       // [nb][E]: slots of each expert in each block's chunk
  int* offsets;    // [E + 1]
  int* row;        // [S]
};

__global__ void __launch_bounds__(kSortThreads) qgemm_moe_count_kernel(const SortParams p) {
  extern __shared__ int sm_hist[];
  griddep_wait();
  griddep_launch_dependents();
  for (int e = threadIdx.x; e < p.E; e += kSortThreads) sm_hist[e] = 0;
  __syncthreads();
  const int64_t s0 = (int64_t)blockIdx.x * p.chunk;
  const int n = (int)min((int64_t)p.chunk, (int64_t)p.S - s0);
  for (int i = threadIdx.x; i < n; i += kSortThreads) {
    const int e = p.ids[s0 + i];
    if ((unsigned)e < (unsigned)p.E) atomicAdd(&sm_hist[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += kSortThreads) p.hist[(size_t)blockIdx.x * p.E + e] = sm_hist[e];
}

// Exclusive prefix sum of v over the block's threads, in thread order; *total gets the sum.
__device__ __forceinline__ int block_excl_scan(int v, int* red, int* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) red[w] = inc;
  __syncthreads();
  int base = 0, sum = 0;
#pragma unroll
  for (int i = 0; i < kSortWarps; ++i) {
    if (i < w) base += red[i];
    sum += red[i];
  }
  __syncthreads();
  *total = sum;
  return base + inc - v;
}

// Rows of one chunk.  Shared memory: the running row of each expert for each warp's share of the
// chunk, [kSortWarps][E].
__global__ void __launch_bounds__(kSortThreads) qgemm_moe_rank_kernel(const SortParams p) {
  extern __shared__ int sm_cnt[];
  __shared__ int red[kSortWarps];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < kSortWarps * p.E; i += kSortThreads) sm_cnt[i] = 0;
  __syncthreads();
  const int64_t s0 = (int64_t)blockIdx.x * p.chunk;
  const int n = (int)min((int64_t)p.chunk, (int64_t)p.S - s0);
  const int share = (n + kSortWarps - 1) / kSortWarps;
  const int i0 = min(n, w * share), i1 = min(n, i0 + share);
  for (int i = i0 + lane; i < i1; i += 32) {
    const int e = p.ids[s0 + i];
    if ((unsigned)e < (unsigned)p.E) atomicAdd(&sm_cnt[w * p.E + e], 1);
  }
  __syncthreads();
  // first row of each expert in this chunk: all slots of smaller experts, then those of this
  // expert in earlier chunks, then in earlier warps
  int carry = 0;
  for (int e0 = 0; e0 < p.E; e0 += kSortThreads) {
    const int e = e0 + threadIdx.x;
    int tot = 0, before = 0;
    if (e < p.E)
      for (int b = 0; b < p.nb; ++b) {
        const int c = p.hist[(size_t)b * p.E + e];
        before += (b < (int)blockIdx.x) ? c : 0;
        tot += c;
      }
    int sum;
    const int first = carry + block_excl_scan(tot, red, &sum);
    carry += sum;
    if (e < p.E) {
      int at = first + before;
#pragma unroll
      for (int i = 0; i < kSortWarps; ++i) {
        const int c = sm_cnt[i * p.E + e];
        sm_cnt[i * p.E + e] = at;
        at += c;
      }
      if (blockIdx.x == 0) p.offsets[e] = first;
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) p.offsets[p.E] = carry;
  __syncthreads();
  // 32 slots at a time, in order: a slot's row is the expert's running row plus the lanes of the
  // same expert before it
  int* cnt = sm_cnt + w * p.E;
  for (int i = i0; i < i1; i += 32) {
    const bool in = i + lane < i1;
    const int e = in ? p.ids[s0 + i + lane] : -1;
    const bool ok = (unsigned)e < (unsigned)p.E;
    const unsigned same = __match_any_sync(0xffffffffu, ok ? e : -1);
    const int rank = __popc(same & ((1u << lane) - 1u));
    const int base = ok ? cnt[e] : 0;
    __syncwarp();
    if (ok && rank == 0) cnt[e] = base + __popc(same);
    __syncwarp();
    if (in) p.row[s0 + i + lane] = ok ? base + rank : -1;
  }
}

// ---------------------------------------------------------------------------------------
// Rows.  A thread block is bx threads along a row (bx a power of two) times by tokens.
// ---------------------------------------------------------------------------------------
constexpr int kRowThreads = 256;

struct RowShape {
  int bx, by;
};
static RowShape row_shape(int64_t nvec) {
  int bx = 1;
  while (bx < kRowThreads && bx < nvec) bx <<= 1;
  return {bx, kRowThreads / bx};
}

template <typename V>
__global__ void __launch_bounds__(kRowThreads) qgemm_moe_gather_kernel(const V* __restrict__ x, int64_t T,
                                                                       int nvec, int k,
                                                                       const int* __restrict__ row,
                                                                       V* __restrict__ xs) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (t >= T) return;
  const int* r = row + t * k;
  for (int v = threadIdx.x; v < nvec; v += blockDim.x) {
    const V a = x[t * nvec + v];
    for (int j = 0; j < k; ++j) {
      const int ro = __ldg(r + j);
      if (ro >= 0) xs[(int64_t)ro * nvec + v] = a;
    }
  }
}

// N elements of a row as fp32, and back with one rounding.
template <typename T, int N>
struct Vec;
template <int N>
struct Vec<float, N> {
  static __device__ __forceinline__ void load(const float* p, float (&f)[N]) {
    if constexpr (N % 4 == 0) {
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const float4 v = *reinterpret_cast<const float4*>(p + i);
        f[i] = v.x, f[i + 1] = v.y, f[i + 2] = v.z, f[i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = p[i];
    }
  }
  static __device__ __forceinline__ void store(float* p, const float (&f)[N]) {
    if constexpr (N % 4 == 0) {
#pragma unroll
      for (int i = 0; i < N; i += 4)
        *reinterpret_cast<float4*>(p + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) p[i] = f[i];
    }
  }
};
template <int N>
struct Vec<__nv_bfloat16, N> {
  static __device__ __forceinline__ void load(const __nv_bfloat16* p, float (&f)[N]) {
    if constexpr (N == 8) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    } else if constexpr (N == 2) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
      f[0] = __uint_as_float(w << 16);
      f[1] = __uint_as_float(w & 0xFFFF0000u);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = __bfloat162float(p[i]);
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&f)[N]) {
    if constexpr (N % 2 == 0) {
      uint32_t w[N / 2];
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
      }
      if constexpr (N == 8) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
      else *reinterpret_cast<uint32_t*>(p) = w[0];
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) p[i] = __float2bfloat16_rn(f[i]);
    }
  }
};

// y[t] = sum_j w[t][j] ys[row[t][j]], j ascending (w absent: 1); a row outside [0, S) is none.
template <typename TI, typename TO, int N>
__global__ void __launch_bounds__(kRowThreads) qgemm_moe_combine_kernel(const TI* __restrict__ ys, int64_t T,
                                                                        int H, int k, int64_t S,
                                                                        const int* __restrict__ row,
                                                                        const float* __restrict__ w,
                                                                        TO* __restrict__ y) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (t >= T) return;
  const int* r = row + t * k;
  for (int h = threadIdx.x * N; h < H; h += blockDim.x * N) {
    float acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.f;
    for (int j = 0; j < k; ++j) {
      const int ro = __ldg(r + j);
      if (ro < 0 || ro >= S) continue;
      const float wj = w ? __ldg(w + t * k + j) : 1.f;
      float f[N];
      Vec<TI, N>::load(ys + (int64_t)ro * H + h, f);
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] = fmaf(wj, f[i], acc[i]);
    }
    Vec<TO, N>::store(y + t * H + h, acc);
  }
}

constexpr int kGradSlots = 8;  // slots of a token whose dot products run together

// dys[row] = w dy and dw = <dy, ys[row]>.  Each thread sums its elements of the row in ascending
// order; lanes, then warps, are added in a fixed tree.
template <typename TD, typename TY, int N>
__global__ void __launch_bounds__(kRowThreads) qgemm_moe_combine_grad_kernel(
    const TD* __restrict__ dy, const TY* __restrict__ ys, int64_t T, int H, int k, int64_t S,
    const int* __restrict__ row, const float* __restrict__ w, TY* __restrict__ dys, float* __restrict__ dw) {
  __shared__ float red[kRowThreads / 32][kGradSlots];
  griddep_wait();
  griddep_launch_dependents();
  const int bx = blockDim.x;
  const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = t < T;  // (every thread takes part in the reductions)
  const int tid = threadIdx.y * bx + threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int j0 = 0; j0 < k; j0 += kGradSlots) {
    int ro[kGradSlots];
    float wj[kGradSlots], part[kGradSlots];
#pragma unroll
    for (int j = 0; j < kGradSlots; ++j) {
      ro[j] = (live && j0 + j < k) ? __ldg(row + t * k + j0 + j) : -1;
      if (ro[j] >= S) ro[j] = -1;
      wj[j] = ro[j] >= 0 ? __ldg(w + t * k + j0 + j) : 0.f;
      part[j] = 0.f;
    }
    if (live)
      for (int h = threadIdx.x * N; h < H; h += bx * N) {
        float d[N];
        Vec<TD, N>::load(dy + t * H + h, d);
#pragma unroll
        for (int j = 0; j < kGradSlots; ++j) {
          if (ro[j] < 0) continue;
          float f[N], g[N];
          Vec<TY, N>::load(ys + (int64_t)ro[j] * H + h, f);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            part[j] = fmaf(d[i], f[i], part[j]);
            g[i] = wj[j] * d[i];
          }
          Vec<TY, N>::store(dys + (int64_t)ro[j] * H + h, g);
        }
      }
    const int width = min(bx, 32);
#pragma unroll
    for (int j = 0; j < kGradSlots; ++j)
      for (int o = width >> 1; o > 0; o >>= 1) part[j] += __shfl_xor_sync(0xffffffffu, part[j], o);
    if (bx > 32) {
      if (lane == 0)
#pragma unroll
        for (int j = 0; j < kGradSlots; ++j) red[warp][j] = part[j];
      __syncthreads();
      const int w0 = threadIdx.y * (bx >> 5);
      if (threadIdx.x < kGradSlots) {
        float s = 0.f;
        for (int i = 0; i < (bx >> 5); ++i) s += red[w0 + i][threadIdx.x];
        if (live && j0 + (int)threadIdx.x < k) dw[t * k + j0 + threadIdx.x] = s;
      }
      __syncthreads();
    } else if (live && threadIdx.x == 0) {
#pragma unroll
      for (int j = 0; j < kGradSlots; ++j)
        if (j0 + j < k) dw[t * k + j0 + j] = part[j];
    }
  }
}

// ---------------------------------------------------------------------------------------
// Host-side launchers
// ---------------------------------------------------------------------------------------
static int sort_chunk(int64_t S) {
  return (int)std::max<int64_t>(kSortChunk, (S + kSortBlocks - 1) / kSortBlocks);
}

size_t moe_sort_bytes(int64_t S, int E) {
  const int64_t c = sort_chunk(S);
  return (size_t)((S + c - 1) / c) * (size_t)E * 4;
}

cudaError_t launch_moe_sort(const int* ids, int64_t S, int E, int* offsets, int* row, int* hist,
                            cudaStream_t stream) {
  SortParams p{};
  p.ids = ids;
  p.S = (int)S;
  p.E = E;
  p.chunk = sort_chunk(S);
  p.nb = (int)((S + p.chunk - 1) / p.chunk);
  p.hist = hist;
  p.offsets = offsets;
  p.row = row;
  const size_t rank_smem = (size_t)kSortWarps * E * 4;
  if (rank_smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(qgemm_moe_rank_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kSmemLimit - 1024);
    if (e != cudaSuccess) return e;
  }
  cudaError_t e = launch_dep(qgemm_moe_count_kernel, dim3(p.nb), dim3(kSortThreads), (size_t)E * 4, stream, p);
  if (e != cudaSuccess) return e;
  return launch_dep(qgemm_moe_rank_kernel, dim3(p.nb), dim3(kSortThreads), rank_smem, stream, p);
}

template <typename V>
static cudaError_t gather_impl(const void* x, int64_t T, int64_t row_bytes, int k, const int* row, void* xs,
                               cudaStream_t stream) {
  const int nvec = (int)(row_bytes / (int64_t)sizeof(V));
  const RowShape s = row_shape(nvec);
  return launch_dep(qgemm_moe_gather_kernel<V>, dim3((unsigned)((T + s.by - 1) / s.by)), dim3(s.bx, s.by), 0,
                    stream, static_cast<const V*>(x), T, nvec, k, row, static_cast<V*>(xs));
}

cudaError_t launch_moe_gather(const void* x, int64_t T, int64_t row_bytes, int k, const int* row, void* xs,
                              cudaStream_t stream) {
  if (row_bytes % 16 == 0) return gather_impl<uint4>(x, T, row_bytes, k, row, xs, stream);
  if (row_bytes % 4 == 0) return gather_impl<uint32_t>(x, T, row_bytes, k, row, xs, stream);
  return gather_impl<uint16_t>(x, T, row_bytes, k, row, xs, stream);
}

// Elements per thread and step: 8 (16 bytes of bf16) where H allows it, else 2, else 1 -- rows
// are contiguous, so H also decides their alignment.
template <typename F>
static cudaError_t by_width(int64_t H, F f) {
  if (H % 8 == 0) return f(std::integral_constant<int, 8>{});
  if (H % 2 == 0) return f(std::integral_constant<int, 2>{});
  return f(std::integral_constant<int, 1>{});
}

template <typename TI, typename TO>
static cudaError_t combine_impl(const void* ys, int64_t T, int64_t H, int k, const int* row, const float* w,
                                void* y, cudaStream_t stream) {
  return by_width(H, [&](auto n) {
    constexpr int N = decltype(n)::value;
    const RowShape s = row_shape(H / N);
    return launch_dep(qgemm_moe_combine_kernel<TI, TO, N>, dim3((unsigned)((T + s.by - 1) / s.by)),
                      dim3(s.bx, s.by), 0, stream, static_cast<const TI*>(ys), T, (int)H, k, T * k, row, w,
                      static_cast<TO*>(y));
  });
}

cudaError_t launch_moe_combine(bool in_bf16, bool out_bf16, const void* ys, int64_t T, int64_t H, int k,
                               const int* row, const float* w, void* y, cudaStream_t stream) {
  using B = __nv_bfloat16;
  if (in_bf16)
    return out_bf16 ? combine_impl<B, B>(ys, T, H, k, row, w, y, stream)
                    : combine_impl<B, float>(ys, T, H, k, row, w, y, stream);
  return out_bf16 ? combine_impl<float, B>(ys, T, H, k, row, w, y, stream)
                  : combine_impl<float, float>(ys, T, H, k, row, w, y, stream);
}

template <typename TD, typename TY>
static cudaError_t combine_grad_impl(const void* dy, const void* ys, int64_t T, int64_t H, int k, const int* row,
                                     const float* w, void* dys, float* dw, cudaStream_t stream) {
  return by_width(H, [&](auto n) {
    constexpr int N = decltype(n)::value;
    const RowShape s = row_shape(H / N);
    return launch_dep(qgemm_moe_combine_grad_kernel<TD, TY, N>, dim3((unsigned)((T + s.by - 1) / s.by)),
                      dim3(s.bx, s.by), 0, stream, static_cast<const TD*>(dy), static_cast<const TY*>(ys), T,
                      (int)H, k, T * k, row, w, static_cast<TY*>(dys), dw);
  });
}

cudaError_t launch_moe_combine_grad(bool dy_bf16, bool ys_bf16, const void* dy, const void* ys, int64_t T,
                                    int64_t H, int k, const int* row, const float* w, void* dys, float* dw,
                                    cudaStream_t stream) {
  using B = __nv_bfloat16;
  if (dy_bf16)
    return ys_bf16 ? combine_grad_impl<B, B>(dy, ys, T, H, k, row, w, dys, dw, stream)
                   : combine_grad_impl<B, float>(dy, ys, T, H, k, row, w, dys, dw, stream);
  return ys_bf16 ? combine_grad_impl<float, B>(dy, ys, T, H, k, row, w, dys, dw, stream)
                 : combine_grad_impl<float, float>(dy, ys, T, H, k, row, w, dys, dw, stream);
}

}  // namespace qg
