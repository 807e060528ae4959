// i8.cu -- int8 weights with a scale per output channel, int8 activations with a scale per row
// taken on the fly (W8A8), plain and routed by expert (sm_100a).
//
//   s_m = fp32(max|x_m| * fp32(1/127)),  q_mk = RNE(x_mk / s_m);   W: the same per channel n, ahead of time
//   y[m][n] = (sum_k q_mk p_nk) * sw_n * s_m
//
// The sum is an exact int32 (K <= 131072 keeps it inside), so a row of y depends on that row, W
// and nothing else: not on the tiling, the K split or the width of the call.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "dequant.cuh"
#include "i8.cuh"
#include "ptx.cuh"

namespace qg {

// ---------------------------------------------------------------------------------------
// Activations: one CTA per row
// ---------------------------------------------------------------------------------------
constexpr float kI8Inv = 1.f / 127.f;
constexpr int kI8QuantThreads = 256;
constexpr int kI8QuantRegs = 4;  // 8-element words per thread kept in registers (rows to 8192)

struct I8QuantParams {
  const uint16_t* x;  // bf16 [M][K]
  int K;
  int8_t* codes;  // [M][K]
  float* scales;  // [M]
};

// One rounded quotient.  t = x inv + 1.5 2^23 rounds x / s to an integer (in t's low bits) up to
// the error of inv; r = x - q s then says which side of the half step x lies on.  r is exact:
// where it decides, |x| >= s / 2 makes x and q s multiples of s's last place, and |r| is about
// s / 2.  So the code is the one of the exact quotient, ties to even.
__device__ __forceinline__ int i8_code(float x, float inv, float s, float half) {
  const float magic = 12582912.f;
  const float t = fmaf(x, inv, magic);
  const float q = t - magic;
  const float r = fmaf(-q, s, x);
  int c = __float_as_int(t);
  if (fabsf(r) >= half) {
    const bool odd = c & 1;
    if (fabsf(r) > half || odd) c += r > 0.f ? 1 : -1;
  }
  return c;
}

__device__ __forceinline__ uint2 i8_codes8(const uint4& v, float up, float inv, float s, float half) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t o[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int c[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      c[2 * h] = i8_code(__uint_as_float(w[2 * i + h] << 16) * up, inv, s, half);
      c[2 * h + 1] = i8_code(__uint_as_float(w[2 * i + h] & 0xFFFF0000u) * up, inv, s, half);
    }
    o[i] = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
  }
  return make_uint2(o[0], o[1]);
}

// Per row: the largest |x| as bf16 bits (which order like the magnitudes, infinities and NaN
// above every finite value), the scale, the codes.
__global__ void __launch_bounds__(kI8QuantThreads) qgemm_i8_quant_kernel(const I8QuantParams p) {
  // x may come from the grid before this one; only once that has completed may the GEMM launch,
  // which reads weights, offsets and tables before it waits for this grid
  griddep_wait();
  griddep_launch_dependents();
  const int64_t m = blockIdx.x;
  const uint16_t* xr = p.x + m * p.K;
  __shared__ uint32_t red[kI8QuantThreads / 32];
  uint4 v[kI8QuantRegs];
  uint32_t top = 0;  // two maxima of 16 bits
  auto take = [&](const uint4& a) {
    top = __vmaxu2(top, a.x & 0x7FFF7FFFu);
    top = __vmaxu2(top, a.y & 0x7FFF7FFFu);
    top = __vmaxu2(top, a.z & 0x7FFF7FFFu);
    top = __vmaxu2(top, a.w & 0x7FFF7FFFu);
  };
#pragma unroll
  for (int j = 0; j < kI8QuantRegs; ++j) {
    const int k = (threadIdx.x + j * kI8QuantThreads) * 8;
    v[j] = k < p.K ? *reinterpret_cast<const uint4*>(xr + k) : make_uint4(0u, 0u, 0u, 0u);
    take(v[j]);
  }
  for (int k = (threadIdx.x + kI8QuantRegs * kI8QuantThreads) * 8; k < p.K; k += kI8QuantThreads * 8)
    take(*reinterpret_cast<const uint4*>(xr + k));
  const uint32_t mx = __reduce_max_sync(0xffffffffu, max(top & 0xFFFFu, top >> 16));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = mx;
  __syncthreads();
  uint32_t bits = red[0];
#pragma unroll
  for (int i = 1; i < kI8QuantThreads / 32; ++i) bits = max(bits, red[i]);
  const bool finite = bits < 0x7F80u;
  const float amax = __uint_as_float(bits << 16);
  const float scale = finite ? __fmul_rn(amax, kI8Inv) : __int_as_float(0x7FC00000);
  if (threadIdx.x == 0) p.scales[m] = scale;
  int8_t* cr = p.codes + m * p.K;
  if (!finite || bits == 0) {
    for (int k = threadIdx.x * 8; k < p.K; k += kI8QuantThreads * 8)
      *reinterpret_cast<uint2*>(cr + k) = make_uint2(0u, 0u);
    return;
  }
  // rows near the bottom of the range are lifted by an exact power of two, scale and all, so that
  // the reciprocal is finite and the residual normal
  const float up = amax < 0x1p-60f ? 0x1p64f : 1.f;
  const float s = scale * up, half = 0.5f * s, inv = __frcp_rn(s);
#pragma unroll
  for (int j = 0; j < kI8QuantRegs; ++j) {
    const int k = (threadIdx.x + j * kI8QuantThreads) * 8;
    if (k < p.K) *reinterpret_cast<uint2*>(cr + k) = i8_codes8(v[j], up, inv, s, half);
  }
  for (int k = (threadIdx.x + kI8QuantRegs * kI8QuantThreads) * 8; k < p.K; k += kI8QuantThreads * 8)
    *reinterpret_cast<uint2*>(cr + k) = i8_codes8(*reinterpret_cast<const uint4*>(xr + k), up, inv, s, half);
}

// ---------------------------------------------------------------------------------------
// Weights (not performance critical): one warp per channel; rows past N and K past the end are
// zeroed by the launcher
// ---------------------------------------------------------------------------------------
__global__ void __launch_bounds__(256) qgemm_i8_pack_kernel(const float* __restrict__ W, int64_t N, int64_t K,
                                                            uint8_t* __restrict__ codes,
                                                            float* __restrict__ scales) {
  const int64_t n = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (n >= N) return;
  const int lane = threadIdx.x & 31;
  uint32_t bits = 0;
  for (int64_t k = lane; k < K; k += 32) bits = max(bits, __float_as_uint(W[n * K + k]) & 0x7FFFFFFFu);
  bits = __reduce_max_sync(0xffffffffu, bits);
  const bool finite = bits < 0x7F800000u;
  const float s = finite ? __fmul_rn(__uint_as_float(bits), kI8Inv) : __int_as_float(0x7FC00000);
  if (lane == 0) scales[n] = s;
  if (!finite || !(s > 0.f)) return;
  const int64_t C = k_chunks(FMT_FP8, K);
  for (int64_t k = lane; k < K; k += 32) {
    // two 24-bit significands: an fp64 quotient lands on a half step only where the exact one does
    const double q = fmin(127.0, fmax(-127.0, rint((double)W[n * K + k] / (double)s)));
    codes[code_offset(C, n, k / 128, (int)(k % 128))] = (uint8_t)(int8_t)q;
  }
}

// ---------------------------------------------------------------------------------------
// GEMM.  The weights are the MMA's M operand (128 channels, straight from the tile-major codes,
// whose layout is the 128-byte swizzle the tensor core reads), the rows of x its N operand (TMA
// from the row-major codes).  So a thread of the epilogue holds one channel and walks over rows:
// its weight scale stays in a register and a warp's stores are consecutive channels of one row.
//
// Persistent, one CTA per SM.  A unit is (expert, 128-channel tile, up to NB rows, K range); two
// accumulator sets in tensor memory let the epilogue of a unit run under the MMAs of the next.
// Warp 0 brings each 128-K chunk into a ring of shared-memory stages (one 16 KB bulk copy per
// matrix, one or more boxes of x), warp 1 issues four M128 N(rows) K32 MMAs per chunk and matrix,
// warps 2..5 read the accumulators out.
// ---------------------------------------------------------------------------------------
constexpr int kI8Threads = 6 * 32;
constexpr int kI8MaxStages = 12;

__device__ __forceinline__ void i8_mma(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor, kind::i8: D s32 (2), A and B signed 8-bit (1), M = 128, N = n.
__device__ __forceinline__ uint32_t i8_idesc(int n) {
  return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}
__device__ __forceinline__ void i8_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
               : "memory");
}
__device__ __forceinline__ void i8_tmem_alloc(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void i8_tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// Each lane reads 16 consecutive 32-bit columns of its own TMEM lane.
__device__ __forceinline__ void i8_tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}
// One box of x: `box` rows of 128 bytes into 128-byte-swizzled shared memory.
__device__ __forceinline__ void i8_load_x(uint32_t dst, const CUtensorMap* map, uint32_t bar, int k, int row,
                                          uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(k), "r"(row), "l"(policy)
      : "memory");
}

struct I8Unit {
  int ex, t, row0, rows, c0, c1, s;  // rows row0 .. row0+rows-1 of x, chunks c0 .. c1-1
};

// Rows of expert ex: its first row and how many of them are computed.
__device__ __forceinline__ int i8_expert_rows(const I8Params& p, int ex, int& lo) {
  lo = min(max(__ldg(p.off + ex), 0), p.M);
  return min(min(max(__ldg(p.off + ex + 1), lo), p.M) - lo, p.max_rows);
}

// Unit u.  Routed: pre[e] is the number of units before expert e's.
__device__ __forceinline__ I8Unit i8_unit(const I8Params& p, const int* pre, int u) {
  I8Unit U;
  int bt;
  if (p.off) {
    int a = 0, b = p.E;  // the last e with pre[e] <= u
    while (b - a > 1) {
      const int m = (a + b) >> 1;
      if (pre[m] <= u) a = m;
      else b = m;
    }
    U.ex = a;
    int lo;
    const int n = i8_expert_rows(p, a, lo);
    const int r = u - pre[a], bts = (n + p.NB - 1) / p.NB;
    bt = r % bts;
    U.t = r / bts;
    U.row0 = lo + bt * p.NB;
    U.rows = min(p.NB, n - bt * p.NB);
    U.s = 0;
  } else {
    U.ex = 0;
    bt = u % p.b_tiles;
    u /= p.b_tiles;
    U.s = u % p.S;
    U.t = u / p.S;
    U.row0 = bt * p.NB;
    U.rows = min(p.NB, p.M - bt * p.NB);
  }
  U.c0 = (int)((int64_t)U.s * p.chunks / p.S);
  U.c1 = (int)((int64_t)(U.s + 1) * p.chunks / p.S);
  return U;
}

template <int NMAT>
__global__ void __launch_bounds__(kI8Threads, 1) qgemm_i8_kernel(const __grid_constant__ I8Params p,
                                                                 const __grid_constant__ CUtensorMap tm_x) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const int NST = p.stages;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + (size_t)NST * p.stage_bytes);
  const uint32_t bar_full = smem_u32(bars);
  const uint32_t bar_empty = bar_full + 8 * kI8MaxStages;
  const uint32_t bar_acc = bar_empty + 8 * kI8MaxStages;  // [2] a unit's accumulators are complete
  const uint32_t bar_acc_free = bar_acc + 16;             // [2] the epilogue has read them
  const uint32_t bar_drain = bar_acc_free + 16;
  int* ctl = reinterpret_cast<int*>(bars + 2 * kI8MaxStages + 5);
  volatile int* abort_flag = ctl + 1;
  int* pre = ctl + 4;  // routed: [E + 1]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tm_x);
    for (int s = 0; s < NST; ++s) {
      mbar_init(bar_full + 8 * s, 1);
      mbar_init(bar_empty + 8 * s, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_acc + 8 * i, 1);
      mbar_init(bar_acc_free + 8 * i, 4);
    }
    mbar_init(bar_drain, 1);
    ctl[1] = 0;
    fence_mbar_init();
  }
  if (warp == 1) i8_tmem_alloc(smem_u32(ctl), (uint32_t)p.tmem_cols);
  int units = p.units;
  if (p.off) {
    // Units of each expert; one without rows, or whose table entries cannot be read, has none.
    // (The offsets and tables are complete: the quantisation kernel before this one let it launch
    // only after all earlier grids had ended.)
    __shared__ int red[kI8Threads / 32];
    const int per = (p.E + kI8Threads - 1) / kI8Threads;
    const int e0 = min(p.E, (int)threadIdx.x * per), e1 = min(p.E, e0 + per);
    int sum = 0;
    for (int e = e0; e < e1; ++e) {
      int lo;
      const int n = i8_expert_rows(p, e, lo);
      bool bad = false;
#pragma unroll
      for (int m = 0; m < NMAT; ++m) {
        const uint8_t* c = p.codes_tab[m][e];
        const float* sc = p.scales_tab[m][e];
        bad |= !c || !sc || (reinterpret_cast<uintptr_t>(c) & 15u) || (reinterpret_cast<uintptr_t>(sc) & 3u);
      }
      if (bad && n > 0) atomicExch(p.dev_err, kErrArg);
      pre[e] = sum;
      sum += bad ? 0 : (n + p.NB - 1) / p.NB * p.tiles;
    }
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) red[warp] = inc;
    __syncthreads();
    int base = inc - sum;
    units = 0;
#pragma unroll
    for (int i = 0; i < kI8Threads / 32; ++i) {
      if (i < warp) base += red[i];
      units += red[i];
    }
    for (int e = e0; e < e1; ++e) pre[e] += base;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(ctl[0]);
  const int set = NMAT * p.NB;  // columns of one accumulator set

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      const uint64_t pol_w = p.w_again ? policy_evict_last() : policy_evict_first();
      const uint64_t pol_x = policy_evict_last();
      RingPos sp;
      int issued = 0;
      bool ok = true, waited = false;
      for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
        const I8Unit U = i8_unit(p, pre, u);
        const uint8_t* w[NMAT];
#pragma unroll
        for (int m = 0; m < NMAT; ++m)
          w[m] = (p.off ? p.codes_tab[m][U.ex] : p.codes[m]) + (int64_t)U.t * p.chunks * kWCodeBytes;
        const int boxes = (U.rows + p.box - 1) / p.box;
        const uint32_t bytes = (uint32_t)(NMAT * kWCodeBytes + boxes * p.box * 128);
        for (int c = U.c0; c < U.c1; ++c) {
          if (issued >= NST &&
              !mbar_wait(bar_empty + 8 * sp.slot, sp.phase ^ 1u, abort_flag, p.dev_err, kErrTimeout)) {
            ok = false;
            break;
          }
          const uint32_t fb = bar_full + 8 * sp.slot;
          const uint32_t st = sbase + (uint32_t)(sp.slot * p.stage_bytes);
          mbar_arrive_expect_tx(fb, bytes);
#pragma unroll
          for (int m = 0; m < NMAT; ++m)
            bulk_load(st + m * kWCodeBytes, w[m] + (int64_t)c * kWCodeBytes, kWCodeBytes, fb, pol_w);
          if (!waited) {
            griddep_wait();  // the codes of x come from the preceding grid
            waited = true;
          }
          for (int b = 0; b < boxes; ++b)
            i8_load_x(st + NMAT * kWCodeBytes + (uint32_t)(b * p.box * 128), &tm_x, fb, c * 128,
                      U.row0 + b * p.box, pol_x);
          sp.next(NST);
          ++issued;
        }
      }
      if (!ok) {
        // let the copies in flight land before the CTA leaves
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 200000) __nanosleep(1000);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      RingPos sp;
      bool ok = true;
      int i = 0;
      for (int u = blockIdx.x; u < units && ok; u += gridDim.x, ++i) {
        const I8Unit U = i8_unit(p, pre, u);
        const uint32_t idesc = i8_idesc((U.rows + 15) & ~15);
        const uint32_t d = tmem + (uint32_t)((i & 1) * set);
        if (i >= 2) {
          if (!mbar_wait_spin(bar_acc_free + 8 * (i & 1), (uint32_t)((i >> 1) - 1) & 1u, false, abort_flag,
                              p.dev_err, kErrTimeout)) {
            ok = false;
            break;
          }
          tc_fence_after();
        }
        for (int c = U.c0; c < U.c1; ++c) {
          if (!mbar_wait_spin(bar_full + 8 * sp.slot, sp.phase, false, abort_flag, p.dev_err, kErrTimeout)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t st = sbase + (uint32_t)(sp.slot * p.stage_bytes);
          const uint64_t bd = smem_desc_sw128(st + NMAT * kWCodeBytes);
#pragma unroll
          for (int m = 0; m < NMAT; ++m) {
            const uint64_t ad = smem_desc_sw128(st + m * kWCodeBytes);
#pragma unroll
            for (int kb = 0; kb < 4; ++kb)
              i8_mma(d + (uint32_t)(m * p.NB), ad + (uint64_t)(kb * 2), bd + (uint64_t)(kb * 2), idesc,
                     (c != U.c0 || kb != 0) ? 1u : 0u);
          }
          i8_commit(bar_empty + 8 * sp.slot);
          sp.next(NST);
        }
        if (!ok) break;
        i8_commit(bar_acc + 8 * (i & 1));
      }
      // every MMA has completed before the CTA may free its tensor memory
      i8_commit(bar_drain);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(bar_drain, 0) && globaltimer_ns() - t0 < kWaitLimitNs) {
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;
    const uint32_t lane_base = (uint32_t)(q * 32) << 16;
    griddep_wait();  // the scales of x come from the preceding grid
    griddep_launch_dependents();
    int i = 0;
    for (int u = blockIdx.x; u < units; u += gridDim.x, ++i) {
      const I8Unit U = i8_unit(p, pre, u);
      const int64_t n = (int64_t)U.t * kTileRows + q * 32 + lane;
      const bool in = n < p.N;
      float sw[NMAT];
#pragma unroll
      for (int m = 0; m < NMAT; ++m) {
        const float* sc = p.off ? p.scales_tab[m][U.ex] : p.scales[m];
        sw[m] = in ? __ldg(sc + n) : 0.f;
      }
      bool ok = mbar_wait(bar_acc + 8 * (i & 1), (uint32_t)(i >> 1) & 1u, abort_flag, p.dev_err, kErrTimeout);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tmem + lane_base + (uint32_t)((i & 1) * set);
      for (int cb = 0; cb < U.rows; cb += 16) {
        uint32_t v[NMAT][16];
#pragma unroll
        for (int m = 0; m < NMAT; ++m) i8_tmem_ld16(d + (uint32_t)(m * p.NB + cb), v[m]);
        const int nr = min(16, U.rows - cb);
        const int64_t m0 = U.row0 + cb;
        const float sxl = (lane < nr) ? p.xscales[m0 + lane] : 0.f;
        tmem_ld_wait();
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const float sx = __shfl_sync(0xffffffffu, sxl, r);
          if (r >= nr || !in) continue;
          const size_t at = (size_t)(m0 + r) * p.N + n;
          if (NMAT == 1 && p.S > 1) {
            p.ws[(size_t)U.s * p.M * p.N + at] = (int)v[0][r];
            continue;
          }
          const float y = __int2float_rn((int)v[0][r]) * sw[0] * sx;
          if (NMAT == 2)
            reinterpret_cast<__nv_bfloat16*>(p.out)[at] =
                __float2bfloat16_rn(silu_mul(y, __int2float_rn((int)v[NMAT - 1][r]) * sw[NMAT - 1] * sx));
          else if (p.out_bf16)
            reinterpret_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(y);
          else
            reinterpret_cast<float*>(p.out)[at] = y;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_acc_free + 8 * (i & 1));
    }
  }

  // ------------------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    i8_tmem_dealloc(tmem, (uint32_t)p.tmem_cols);
  }
}

// Sum of the K ranges' partials (integers: any order gives the same bits), scales, output.
__global__ void __launch_bounds__(256) qgemm_i8_reduce_kernel(const I8Params p) {
  griddep_launch_dependents();
  griddep_wait();
  const int64_t MN = (int64_t)p.M * p.N;
  const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (at >= MN) return;
  const int lim = (int)min((int64_t)4, MN - at);
  int acc[4] = {0, 0, 0, 0};
  const bool vec = (MN & 3) == 0;
  for (int s = 0; s < p.S; ++s) {
    const int* src = p.ws + s * MN + at;
    if (vec) {
      const int4 v = __ldcs(reinterpret_cast<const int4*>(src));
      acc[0] += v.x, acc[1] += v.y, acc[2] += v.z, acc[3] += v.w;
    } else {
      for (int e = 0; e < lim; ++e) acc[e] += __ldcs(src + e);
    }
  }
  for (int e = 0; e < lim; ++e) {
    const int64_t m = (at + e) / p.N, n = (at + e) % p.N;
    const float y = __int2float_rn(acc[e]) * p.scales[0][n] * p.xscales[m];
    if (p.out_bf16)
      reinterpret_cast<__nv_bfloat16*>(p.out)[at + e] = __float2bfloat16_rn(y);
    else
      reinterpret_cast<float*>(p.out)[at + e] = y;
  }
}

// ---------------------------------------------------------------------------------------
// Host-side launchers
// ---------------------------------------------------------------------------------------
template <typename P>
static cudaError_t launch_dep(void (*kern)(P), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                              const P& p) {
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
  return cudaLaunchKernelEx(&cfg, kern, p);
}

cudaError_t launch_i8_pack(const float* W, int64_t N, int64_t K, uint8_t* codes, float* scales,
                           cudaStream_t stream) {
  const cudaError_t e = cudaMemsetAsync(codes, 0, (size_t)packed_code_bytes(FMT_FP8, N, K), stream);
  if (e != cudaSuccess) return e;
  qgemm_i8_pack_kernel<<<(unsigned)((N + 7) / 8), 256, 0, stream>>>(W, N, K, codes, scales);
  return cudaGetLastError();
}

cudaError_t launch_i8_quant(const uint16_t* x, int64_t M, int64_t K, int8_t* codes, float* scales,
                            cudaStream_t stream) {
  I8QuantParams p{x, (int)K, codes, scales};
  return launch_dep(qgemm_i8_quant_kernel, dim3((unsigned)M), dim3(kI8QuantThreads), 0, stream, p);
}


// SMs of device `dev`, read once per device (devices beyond 64 read it on every launch).
static int sm_count(int dev) {
  static std::atomic<int> cached[64];
  int v = (dev >= 0 && dev < 64) ? cached[dev].load(std::memory_order_relaxed) : 0;
  if (v > 0) return v;
  if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v < 1) v = 148;
  if (dev >= 0 && dev < 64) cached[dev].store(v, std::memory_order_relaxed);
  return v;
}

// K ranges of a plain product: the smallest S of least cost, in units of the time one SM takes to
// stream a 16 KB chunk at its share of the memory (0.37 us): rounds of units, each its chunks and
// about four more to start and end; the partials' way out and back through L2 (8 bytes per
// element at about 5 TB/s); and the reduction's launch (about eight).
static int i8_split(int64_t T, int64_t b_tiles, int64_t C, int64_t MN) {
  int best = 1;
  double best_cost = 0.0;
  for (int64_t S = 1; S <= std::min<int64_t>(32, C); ++S) {
    const double rounds = double((T * b_tiles * S + kI8SMs - 1) / kI8SMs);
    const double cost = rounds * (double((C + S - 1) / S) + 4.0) +
                        (S > 1 ? 8.0 + double(S) * double(MN) * 8.0 / 5e6 / 0.37 : 0.0);
    if (S == 1 || cost < best_cost - 1e-9) {
      best_cost = cost;
      best = (int)S;
    }
  }
  return best;
}

// Tiling of a call: rows is M, or the most rows an expert has.
void i8_plan(int64_t N, int64_t K, int64_t rows, int nmat, bool routed, I8Params* p) {
  p->tiles = (int)row_tiles(N);
  p->chunks = (int)k_chunks(FMT_FP8, K);
  const int cap = nmat == 2 ? 128 : 256;
  p->NB = (int)std::min<int64_t>(cap, (rows + 15) / 16 * 16);
  // routed: small boxes, so that an expert's rows bring few of its neighbours' with them
  p->box = routed ? std::min(p->NB, 32) : p->NB;
  p->b_tiles = (int)((rows + p->NB - 1) / p->NB);
  p->S = routed ? 1 : i8_split(p->tiles, p->b_tiles, p->chunks, rows * N);
  p->w_again = p->b_tiles > 1;
  p->stage_bytes = nmat * kWCodeBytes + (p->NB + p->box - 1) / p->box * p->box * 128;
  int cols = 32;
  while (cols < 2 * nmat * p->NB) cols <<= 1;
  p->tmem_cols = cols;
}

size_t i8_partial_bytes(int64_t N, int64_t K, int64_t M) {
  I8Params p{};
  i8_plan(N, K, M, 1, false, &p);
  return p.S > 1 ? (size_t)p.S * (size_t)M * (size_t)N * 4 : 0;
}

template <int NMAT>
static cudaError_t launch_i8_impl(const I8Params& p, size_t smem, int grid, const CUtensorMap& map, int dev,
                                  cudaStream_t stream) {
  auto kern = qgemm_i8_kernel<NMAT>;
  static std::atomic<uint64_t> set_mask{0};
  const uint64_t bit = (dev >= 0 && dev < 64) ? (1ull << dev) : 0ull;
  if (bit == 0 || !(set_mask.load(std::memory_order_acquire) & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit - 64);
    if (e != cudaSuccess) return e;
    set_mask.fetch_or(bit, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3(kI8Threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p, map);
}

// p: planned (i8_plan), operands filled in; map: x's codes in boxes of 128 x p.box.
cudaError_t launch_i8_gemm(I8Params p, const CUtensorMap& map, cudaStream_t stream) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const size_t misc = 1024 + 8 * (2 * kI8MaxStages + 5) + 16 + (p.off ? 4 * ((size_t)p.E + 1) : 0) + 64;
  p.stages = (int)std::min<size_t>(kI8MaxStages, (kSmemLimit - 64 - misc) / (size_t)p.stage_bytes);
  if (p.stages < 2) return cudaErrorInvalidValue;
  const int64_t most = (int64_t)p.tiles * p.b_tiles * (p.off ? p.E : p.S);
  if (most > 0x3FFFFFFF) return cudaErrorInvalidValue;
  p.units = (int)most;  // routed: the kernel counts the units that have rows
  const int grid = (int)std::min<int64_t>(most, sm_count(dev));
  const size_t smem = misc + (size_t)p.stages * p.stage_bytes;
  const cudaError_t g = p.nmat == 2 ? launch_i8_impl<2>(p, smem, grid, map, dev, stream)
                                    : launch_i8_impl<1>(p, smem, grid, map, dev, stream);
  if (g != cudaSuccess || p.S == 1) return g;
  const int64_t quads = ((int64_t)p.M * p.N + 3) / 4;
  return launch_dep(qgemm_i8_reduce_kernel, dim3((unsigned)((quads + 255) / 256)), dim3(256), 0, stream, p);
}

}  // namespace qg
