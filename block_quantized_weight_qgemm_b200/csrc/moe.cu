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
// for that grid before it touches memory (the gather after the sort reads x ahead: see there), and
// only then, if at all, lets its own dependents launch.
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
constexpr int kSmallSlots = 8192;  // one launch can dispatch up to here
constexpr int kSmallThreads = 256;
constexpr int kSortCtas = 8;       // a portable cluster
constexpr int kIdLoads = 8;        // expert ids a lane of the sort loads together
constexpr int kSmallLoads = 4;     // and a thread of the small dispatch

// Exclusive prefix sum of v over the threads of a block of W warps, in thread order; *total gets the sum.
// red: an int per warp.
template <int W>
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
  for (int i = 0; i < W; ++i) {
    if (i < w) base += red[i];
    sum += red[i];
  }
  __syncthreads();
  *total = sum;
  return base + inc - v;
}

// Few slots: one launch for everything.  A block is a token: the row of each of its slots is a count over
// all slots of those that come before it in the order (expert, slot), read as one integer key; then the
// block copies the token's row to its places.  The last block counts the offsets.  (This kernel does
// not let its dependents launch early: qgemm_moe_run reads the offsets before it waits for the grid
// ahead of it.)
template <typename V, int B>
__global__ void __launch_bounds__(kSmallThreads) qgemm_moe_dispatch_small_kernel(
    const int* __restrict__ ids, int T, int k, int E, const V* __restrict__ x, int nvec, int* __restrict__ offsets,
    int* __restrict__ row, V* __restrict__ xs) {
  extern __shared__ int sm_hist[];
  __shared__ int red[kSmallThreads / 32][8];
  __shared__ int place[8];
  griddep_wait();
  const int S = T * k, tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  if ((int)blockIdx.x == T) {
    for (int e = tid; e < E; e += kSmallThreads) sm_hist[e] = 0;
    __syncthreads();
    for (int i0 = 0; i0 < S; i0 += kSmallLoads * kSmallThreads) {
      int e[kSmallLoads];
#pragma unroll
      for (int q = 0; q < kSmallLoads; ++q) {
        const int i = i0 + q * kSmallThreads + tid;
        e[q] = i < S ? __ldg(ids + i) : -1;
      }
#pragma unroll
      for (int q = 0; q < kSmallLoads; ++q)
        if ((unsigned)e[q] < (unsigned)E) atomicAdd(&sm_hist[e[q]], 1);
    }
    __syncthreads();
    int carry = 0;
    for (int e0 = 0; e0 < E; e0 += kSmallThreads) {
      const int e = e0 + tid;
      int sum;
      const int first = carry + block_excl_scan<kSmallThreads / 32>(e < E ? sm_hist[e] : 0, &red[0][0], &sum);
      carry += sum;
      if (e < E) offsets[e] = first;
    }
    if (tid == 0) offsets[E] = carry;
    return;
  }
  const int t = blockIdx.x;
  V a;
  if (tid < nvec) a = x[(int64_t)t * nvec + tid];
  for (int j0 = 0; j0 < k; j0 += B) {
    int key[B], cnt[B];
#pragma unroll
    for (int j = 0; j < B; ++j) {
      const int e = j0 + j < k ? __ldg(ids + t * k + j0 + j) : -1;
      key[j] = (unsigned)e < (unsigned)E ? e * kSmallSlots + (t * k + j0 + j) : -1;
      cnt[j] = 0;
    }
    for (int i0 = 0; i0 < S; i0 += kSmallLoads * kSmallThreads) {
      int e[kSmallLoads];
#pragma unroll
      for (int q = 0; q < kSmallLoads; ++q) {
        const int i = i0 + q * kSmallThreads + tid;
        e[q] = i < S ? __ldg(ids + i) : -1;
      }
#pragma unroll
      for (int q = 0; q < kSmallLoads; ++q) {
        const int ki = (unsigned)e[q] < (unsigned)E ? e[q] * kSmallSlots + i0 + q * kSmallThreads + tid : 0x7FFFFFFF;
#pragma unroll
        for (int j = 0; j < B; ++j) cnt[j] += ki < key[j] ? 1 : 0;
      }
    }
#pragma unroll
    for (int j = 0; j < B; ++j) {
      cnt[j] = __reduce_add_sync(0xffffffffu, cnt[j]);
      if (lane == j) red[w][j] = cnt[j];
    }
    __syncthreads();
    if (tid < B) {
      int s = 0;
#pragma unroll
      for (int i = 0; i < kSmallThreads / 32; ++i) s += red[i][tid];
      const int e = j0 + tid < k ? __ldg(ids + t * k + j0 + tid) : -1;
      const int ro = (unsigned)e < (unsigned)E ? s : -1;
      place[tid] = ro;
      if (j0 + tid < k) row[t * k + j0 + tid] = ro;
    }
    __syncthreads();
    int ro[B];
#pragma unroll
    for (int j = 0; j < B; ++j) ro[j] = place[j];
    for (int v = tid; v < nvec; v += kSmallThreads) {
      const V b = v == tid ? a : x[(int64_t)t * nvec + v];
#pragma unroll
      for (int j = 0; j < B; ++j)
        if (ro[j] >= 0) xs[(int64_t)ro[j] * nvec + v] = b;
    }
  }
}

// Many slots: one cluster of eight CTAs sorts, each a run of S / 8 slots and each of its W warps a run of
// those.  Every warp counts its run's slots per expert, and the counts become, per expert, the slots of
// the CTA's earlier warps; the CTAs exchange their totals through distributed shared memory, which gives
// each the first row of every expert's slots in it; then each warp walks its run in order, 32 slots at a
// time: a slot's row is its expert's first row, plus the slots of that expert in earlier warps, in the
// warp's earlier slots and in earlier lanes.  Shared memory: [W][E] counts, [E] totals, [E] first rows.
//
// Bound by latencies: 20480 slots of 512 experts take about 7 us, two of them the launch.  The lanes of one
// expert are found by a ballot per bit of its number: __match_any_sync took 1080 cycles per 32 slots of
// mostly different experts, these 580.
struct SortParams {
  const int* ids;  // [S]
  int S, E;
  int* offsets;  // [E + 1]
  int* row;      // [S]
};

// (relaxed: it publishes no writes, and a release would wait for those to global memory)
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

template <int W>
__global__ void __cluster_dims__(kSortCtas, 1, 1) __launch_bounds__(W * 32) qgemm_moe_sort_kernel(const SortParams p) {
  extern __shared__ int sm_cnt[];
  __shared__ int red[W];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, E = p.E;
  const int rank = (int)cluster_ctarank();
  int* tot = sm_cnt + W * E;
  int* base = tot + E;
  for (int i = threadIdx.x; i < W * E; i += W * 32) sm_cnt[i] = 0;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t share = ((int64_t)p.S + kSortCtas * W - 1) / (kSortCtas * W);
  const int s0 = (int)min((int64_t)p.S, share * (rank * W + w)), s1 = (int)min((int64_t)p.S, s0 + share);
  int* cnt = sm_cnt + w * E;
  // an expert outside [0, E) becomes E, which is counted nowhere
  auto load = [&](int s, int (&e)[kIdLoads]) {
#pragma unroll
    for (int q = 0; q < kIdLoads; ++q) {
      e[q] = s1 - s > 32 * q + lane ? __ldg(p.ids + s + 32 * q + lane) : E;
      if ((unsigned)e[q] > (unsigned)E) e[q] = E;
    }
  };
  int id[kIdLoads];
  if (s0 < s1) load(s0, id);
  __syncthreads();
  for (int64_t s = s0; s < s1; s += 32 * kIdLoads) {
    if (s != s0) load((int)s, id);
#pragma unroll
    for (int q = 0; q < kIdLoads; ++q)
      if (id[q] < E) atomicAdd(&cnt[id[q]], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += W * 32) {
    int c[W], sum = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) c[i] = sm_cnt[i * E + e];
#pragma unroll
    for (int i = 0; i < W; ++i) {
      sm_cnt[i * E + e] = sum;
      sum += c[i];
    }
    tot[e] = sum;
  }
  cluster_sync_all();
  int carry = 0;
  for (int e0 = 0; e0 < E; e0 += W * 32) {
    const int e = e0 + threadIdx.x;
    int all = 0, before = 0;
    if (e < E) {
      const uint32_t a = smem_u32(tot + e);
      int c[kSortCtas];
#pragma unroll
      for (int r = 0; r < kSortCtas; ++r)
        asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(c[r]) : "r"(mapa_shared(a, r)) : "memory");
#pragma unroll
      for (int r = 0; r < kSortCtas; ++r) {
        before += r < rank ? c[r] : 0;
        all += c[r];
      }
    }
    int sum;
    const int first = carry + block_excl_scan<W>(all, red, &sum);
    carry += sum;
    if (e < E) {
      base[e] = first + before;
      if (rank == 0) p.offsets[e] = first;
    }
  }
  cluster_arrive();  // this CTA has read the others' totals
  if (rank == 0 && threadIdx.x == 0) p.offsets[E] = carry;
  __syncthreads();
  const int bits = 32 - __clz(E);  // of 0 .. E
  for (int64_t s = s0; s < s1; s += 32 * kIdLoads) {
    if (s1 - s0 > 32 * kIdLoads) load((int)s, id);
    unsigned same[kIdLoads];  // the lanes of the lane's expert
#pragma unroll
    for (int q = 0; q < kIdLoads; ++q) same[q] = 0xffffffffu;
    const int nq = (int)min((int64_t)kIdLoads, (s1 - s + 31) / 32);
    for (int b = 0; b < bits; ++b)
#pragma unroll
      for (int q = 0; q < kIdLoads; ++q) {
        if (q >= nq) break;
        const bool one = (id[q] >> b) & 1;
        const unsigned m = __ballot_sync(0xffffffffu, one);
        same[q] &= one ? m : ~m;
      }
#pragma unroll
    for (int q = 0; q < kIdLoads; ++q) {
      if (q >= nq) break;
      const int64_t at = s + 32 * q + lane;
      const int e = id[q], before = __popc(same[q] & ((1u << lane) - 1u));
      const int run = e < E ? cnt[e] : 0;
      __syncwarp();
      if (e < E && before == 0) cnt[e] = run + __popc(same[q]);
      __syncwarp();
      if (at < s1) p.row[at] = e < E ? base[e] + run + before : -1;
    }
  }
  cluster_wait();  // no CTA leaves while another reads its totals
}

// ---------------------------------------------------------------------------------------
// Rows.  A thread block is bx threads along a row (bx a power of two) times by tokens.
// ---------------------------------------------------------------------------------------
constexpr int kRowThreads = 256;
constexpr int kSMs = 148;  // of a B200, for the rule that spreads few tokens

struct RowShape {
  int bx, by;
};
static RowShape row_shape(int64_t nvec) {
  int bx = 1;
  while (bx < kRowThreads && bx < nvec) bx <<= 1;
  return {bx, kRowThreads / bx};
}

// xs[row[s]] = x[t]: a row is read once and written k times.  Bound by HBM: 2048 tokens top-10 of 4 KB rows
// (92 MB) in 14 us, the measured copy rate.
template <typename V>
__global__ void __launch_bounds__(kRowThreads) qgemm_moe_gather_kernel(const V* __restrict__ x, int64_t T,
                                                                       int nvec, int k,
                                                                       const int* __restrict__ row,
                                                                       V* __restrict__ xs) {
  // x is older than the sort, which let this grid launch after the grids before it had ended: the
  // first piece of the row is loaded under the sort
  const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  V first;
  if (t < T && threadIdx.x < nvec) first = x[t * nvec + threadIdx.x];
  griddep_wait();
  griddep_launch_dependents();
  if (t >= T) return;
  const int* r = row + t * k;
  for (int v = threadIdx.x; v < nvec; v += blockDim.x) {
    const V a = v == threadIdx.x ? first : x[t * nvec + v];
    for (int j = 0; j < k; ++j) {
      const int ro = __ldg(r + j);
      if (ro >= 0) xs[(int64_t)ro * nvec + v] = a;
    }
  }
}

// N elements of a row: raw bits as loaded (so that several rows' loads are in flight before any is
// used), their fp32 values, and back with one rounding.
template <int BYTES>
struct Raw {
  static constexpr int kWords = (BYTES + 3) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ void load(const void* p) {
    if constexpr (BYTES % 16 == 0) {
#pragma unroll
      for (int i = 0; i < BYTES / 16; ++i) {
        const uint4 v = reinterpret_cast<const uint4*>(p)[i];
        w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
      }
    } else if constexpr (BYTES == 8) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x, w[1] = v.y;
    } else if constexpr (BYTES == 4) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
      w[0] = *reinterpret_cast<const uint16_t*>(p);
    }
  }
  __device__ __forceinline__ void store(void* p) const {
    if constexpr (BYTES % 16 == 0) {
#pragma unroll
      for (int i = 0; i < BYTES / 16; ++i)
        reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else if constexpr (BYTES == 8) {
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else if constexpr (BYTES == 4) {
      *reinterpret_cast<uint32_t*>(p) = w[0];
    } else {
      *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[0];
    }
  }
};

template <typename T, int N>
struct Vec;
template <int N>
struct Vec<float, N> {
  using R = Raw<4 * N>;
  static __device__ __forceinline__ void open(const R& r, float (&f)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = __uint_as_float(r.w[i]);
  }
  static __device__ __forceinline__ R close(const float (&f)[N]) {
    R r;
#pragma unroll
    for (int i = 0; i < N; ++i) r.w[i] = __float_as_uint(f[i]);
    return r;
  }
};
template <int N>
struct Vec<__nv_bfloat16, N> {
  using R = Raw<2 * N>;
  static __device__ __forceinline__ void open(const R& r, float (&f)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      f[i] = __uint_as_float((i & 1) ? (r.w[i >> 1] & 0xFFFF0000u) : (r.w[i >> 1] << 16));
  }
  static __device__ __forceinline__ R close(const float (&f)[N]) {
    R r;
    if constexpr (N == 1) {
      r.w[0] = __bfloat16_as_ushort(__float2bfloat16_rn(f[0]));
    } else {
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        r.w[i] = *reinterpret_cast<const uint32_t*>(&b);
      }
    }
    return r;
  }
};

// y[t] = sum_j w[t][j] ys[row[t][j]], j ascending (w absent: 1); a row outside [0, S) is none.
// The loads of B slots go together.  Bound by HBM: 2048 tokens top-10 of 2048 bf16 in 16.5 us (85 % of the
// measured copy rate), 16384 tokens top-8 of 4096 at it.
template <typename TI, typename TO, int N, int B>
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
  const float* wt = w ? w + t * k : nullptr;
  for (int h = (blockIdx.y * blockDim.x + threadIdx.x) * N; h < H; h += gridDim.y * blockDim.x * N) {
    float acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.f;
    for (int j0 = 0; j0 < k; j0 += B) {
      typename Vec<TI, N>::R raw[B];
      float wj[B];
      bool has[B];
#pragma unroll
      for (int j = 0; j < B; ++j) {
        const int ro = j0 + j < k ? __ldg(r + j0 + j) : -1;
        has[j] = ro >= 0 && ro < S;
        wj[j] = has[j] && wt ? __ldg(wt + j0 + j) : 1.f;
        raw[j].clear();
        if (has[j]) raw[j].load(ys + (int64_t)ro * H + h);
      }
#pragma unroll
      for (int j = 0; j < B; ++j) {
        if (!has[j]) continue;
        float f[N];
        Vec<TI, N>::open(raw[j], f);
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = fmaf(wj[j], f[i], acc[i]);
      }
    }
    Vec<TO, N>::close(acc).store(y + t * H + h);
  }
}

// dys[row] = w dy and dw = <dy, ys[row]>: a warp per slot (the k warps of a token find its dy in L1).
// A lane sums its elements in ascending order, the lanes are added in a fixed tree.  Bound by HBM: 2048 tokens
// top-10 of 2048 bf16 in 30 us (176 MB, 89 % of the measured copy rate); with a block per token and sums
// over its warps it took 55.
constexpr int kGradSteps = 2;  // steps of a row loaded together (34, 30, 34, 33 us with 1, 2, 4, 8: 2048 tokens, bf16)

template <typename TD, typename TY, int N>
__global__ void __launch_bounds__(kRowThreads) qgemm_moe_combine_grad_kernel(
    const TD* __restrict__ dy, const TY* __restrict__ ys, int64_t S, int H, int k, const int* __restrict__ row,
    const float* __restrict__ w, TY* __restrict__ dys, float* __restrict__ dw) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t s = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (s >= S) return;
  const int ro = __ldg(row + s);
  if (ro < 0 || ro >= S) {
    if (lane == 0) dw[s] = 0.f;
    return;
  }
  const float ws = __ldg(w + s);
  const TD* d0 = dy + s / k * H;
  const TY* y0 = ys + (int64_t)ro * H;
  TY* o0 = dys + (int64_t)ro * H;
  float part = 0.f;
  for (int h0 = lane * N; h0 < H; h0 += kGradSteps * 32 * N) {
    typename Vec<TD, N>::R rd[kGradSteps];
    typename Vec<TY, N>::R ry[kGradSteps];
#pragma unroll
    for (int i = 0; i < kGradSteps; ++i) {
      const int h = h0 + i * 32 * N;
      rd[i].clear();
      ry[i].clear();
      if (h < H) {
        rd[i].load(d0 + h);
        ry[i].load(y0 + h);
      }
    }
#pragma unroll
    for (int i = 0; i < kGradSteps; ++i) {
      const int h = h0 + i * 32 * N;
      float d[N], f[N];
      Vec<TD, N>::open(rd[i], d);
      Vec<TY, N>::open(ry[i], f);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        part = fmaf(d[e], f[e], part);
        d[e] *= ws;
      }
      if (h < H) Vec<TY, N>::close(d).store(o0 + h);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
  if (lane == 0) dw[s] = part;
}

// ---------------------------------------------------------------------------------------
// Host-side launchers
// ---------------------------------------------------------------------------------------
template <int W>
static cudaError_t sort_impl(const SortParams& p, cudaStream_t stream) {
  const size_t smem = (size_t)(W + 2) * p.E * 4;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(qgemm_moe_sort_kernel<W>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kSmemLimit - 1024);
    if (e != cudaSuccess) return e;
  }
  return launch_dep(qgemm_moe_sort_kernel<W>, dim3(kSortCtas), dim3(W * 32), smem, stream, p);
}

static cudaError_t launch_moe_sort(const int* ids, int64_t S, int E, int* offsets, int* row, cudaStream_t stream) {
  const SortParams p{ids, (int)S, E, offsets, row};
  // as many warps as have their counts in shared memory
  return (size_t)18 * E * 4 <= kSmemLimit - 1024 ? sort_impl<16>(p, stream) : sort_impl<8>(p, stream);
}

// Whether one launch dispatches: every token then counts over all slots, 6 instructions per slot and pass and
// 2 per slot and own slot, about 0.06 us per million beyond the 3 us of a launch.  The sort and the gather
// after it take 4.5 us for few experts and 7 for 512, so 40 million is the border: 256 tokens top-10 (21
// million) 4.4 against 7 us; 450 (65 million) 8.5 against 7; 1500 tokens top-2 of 8 (45 million) 4.7
// against 4.6 us.
static bool dispatch_small(int64_t T, int k) {
  const int64_t S = T * k;
  return S <= kSmallSlots && T * S * (6 * ((k + 7) / 8) + 2 * k) <= 40000000;
}

// k slots in equal batches of at most b.
static int batch_of(int k, int b) {
  const int n = (k + b - 1) / b;
  return (k + n - 1) / n;
}

template <typename V>
static cudaError_t dispatch_impl(const void* x, int64_t T, int64_t row_bytes, const int* ids, int k, int E,
                                 int* offsets, int* row, void* xs, cudaStream_t stream) {
  const int nvec = (int)(row_bytes / (int64_t)sizeof(V));
  const V* xv = static_cast<const V*>(x);
  V* xsv = static_cast<V*>(xs);
  if (dispatch_small(T, k)) {
    // the slots of a token in equal batches, each counted in one pass over all slots
    auto small = [&](auto b) {
      return launch_dep(qgemm_moe_dispatch_small_kernel<V, decltype(b)::value>, dim3((unsigned)T + 1),
                        dim3(kSmallThreads), (size_t)E * 4, stream, ids, (int)T, k, E, xv, nvec, offsets, row, xsv);
    };
    const int b = batch_of(k, 8);
    if (b == 1) return small(std::integral_constant<int, 1>{});
    if (b == 2) return small(std::integral_constant<int, 2>{});
    if (b <= 4) return small(std::integral_constant<int, 4>{});
    if (b <= 6) return small(std::integral_constant<int, 6>{});
    return small(std::integral_constant<int, 8>{});
  }
  const cudaError_t e = launch_moe_sort(ids, T * k, E, offsets, row, stream);
  if (e != cudaSuccess) return e;
  const RowShape s = row_shape(nvec);
  return launch_dep(qgemm_moe_gather_kernel<V>, dim3((unsigned)((T + s.by - 1) / s.by)), dim3(s.bx, s.by), 0,
                    stream, xv, T, nvec, k, (const int*)row, xsv);
}

cudaError_t launch_moe_dispatch(const void* x, int64_t T, int64_t row_bytes, const int* ids, int k, int E,
                                int* offsets, int* row, void* xs, cudaStream_t stream) {
  if (row_bytes % 16 == 0)
    return dispatch_impl<uint4>(x, T, row_bytes, ids, k, E, offsets, row, xs, stream);
  if (row_bytes % 4 == 0)
    return dispatch_impl<uint32_t>(x, T, row_bytes, ids, k, E, offsets, row, xs, stream);
  return dispatch_impl<uint16_t>(x, T, row_bytes, ids, k, E, offsets, row, xs, stream);
}

// Elements per thread and step: 8 (16 bytes of bf16) where H allows it, else 2, else 1 -- rows
// are contiguous, so H also decides their alignment.
template <typename F>
static cudaError_t by_width(int64_t H, F f) {
  if (H % 8 == 0) return f(std::integral_constant<int, 8>{});
  if (H % 2 == 0) return f(std::integral_constant<int, 2>{});
  return f(std::integral_constant<int, 1>{});
}

template <typename TI, typename TO, int N, int B>
static cudaError_t combine_batch(const void* ys, int64_t T, int64_t H, int k, const int* row, const float* w,
                                 void* y, cudaStream_t stream) {
  const RowShape s = row_shape(H / N);
  const int64_t blocks = (T + s.by - 1) / s.by;
  // few tokens: the pieces of a row go to blocks of their own
  const int64_t pieces = (H / N + s.bx - 1) / s.bx;
  const unsigned gy = (unsigned)(blocks < 2 * kSMs ? std::min<int64_t>(pieces, 64) : 1);
  return launch_dep(qgemm_moe_combine_kernel<TI, TO, N, B>, dim3((unsigned)blocks, gy), dim3(s.bx, s.by), 0, stream,
                    static_cast<const TI*>(ys), T, (int)H, k, T * k, row, w, static_cast<TO*>(y));
}

template <typename TI, typename TO>
static cudaError_t combine_impl(const void* ys, int64_t T, int64_t H, int k, const int* row, const float* w,
                                void* y, cudaStream_t stream) {
  return by_width(H, [&](auto n) {
    constexpr int N = decltype(n)::value;
    const auto go = [&](auto b) {
      return combine_batch<TI, TO, N, decltype(b)::value>(ys, T, H, k, row, w, y, stream);
    };
    // A batch's loop has exactly its slots: ten slots as two batches of five took 16.5 us (2048 tokens, bf16)
    // where loops of eight, five of them used, took 19, and two slots in a loop of eight 66 where 40
    // suffice.  At most eight slots, or five of 32-byte pieces (registers).
    if constexpr (N == 8) {
      const int b = batch_of(k, sizeof(TI) == 2 ? 8 : 5);
      if (b == 1) return go(std::integral_constant<int, 1>{});
      if (b == 2) return go(std::integral_constant<int, 2>{});
      if (b == 3) return go(std::integral_constant<int, 3>{});
      if (b == 5) return go(std::integral_constant<int, 5>{});
      if constexpr (sizeof(TI) == 2) {
        if (b == 6) return go(std::integral_constant<int, 6>{});
        if (b == 7) return go(std::integral_constant<int, 7>{});
        if (b == 8) return go(std::integral_constant<int, 8>{});
      }
    }
    return go(std::integral_constant<int, 4>{});
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
    constexpr int kWarps = kRowThreads / 32;
    return launch_dep(qgemm_moe_combine_grad_kernel<TD, TY, N>, dim3((unsigned)((T * k + kWarps - 1) / kWarps)),
                      dim3(kRowThreads), 0, stream, static_cast<const TD*>(dy), static_cast<const TY*>(ys), T * k,
                      (int)H, k, row, w, static_cast<TY*>(dys), dw);
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
