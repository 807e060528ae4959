// i8.cu -- int8 weights with a scale per output channel, int8 activations with a scale per row
// taken on the fly (W8A8), plain and routed by expert (sm_100a).
//
//   s_m = fp32(max|x_m| / 127),  q_mk = RNE(x_mk / s_m);   W: the same per channel n, ahead of time
//   y[m][n] = (sum_k q_mk p_nk) * sw_n * s_m
//
// The sum is an exact int32 (K <= 131072 keeps it inside), so a row of y depends on that row, W
// and nothing else: not on the tiling, the K split or the width of the call.
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "dequant.cuh"
#include "i8.cuh"
#include "ptx.cuh"

namespace qg {

// ---------------------------------------------------------------------------------------
// Activations: one CTA per row
// ---------------------------------------------------------------------------------------
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
  const float scale = finite ? __fdiv_rn(amax, 127.f) : __int_as_float(0x7FC00000);
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
  const float s = finite ? __fdiv_rn(__uint_as_float(bits), 127.f) : __int_as_float(0x7FC00000);
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
// GEMM: one thread per channel of a 128-channel tile, kI8Rows rows of x
// ---------------------------------------------------------------------------------------
constexpr int kI8Rows = 16;

__global__ void __launch_bounds__(128) qgemm_i8_kernel(const I8Params p) {
  griddep_wait();
  int lo = 0, rows = p.M;
  const uint8_t* codes[2] = {p.codes[0], p.codes[1]};
  const float* scales[2] = {p.scales[0], p.scales[1]};
  if (p.off) {
    const int ex = blockIdx.z;
    lo = min(max(p.off[ex], 0), p.M);
    rows = min(min(max(p.off[ex + 1], lo), p.M) - lo, p.max_rows);
    for (int i = 0; i < p.nmat; ++i) {
      codes[i] = p.codes_tab[i][ex];
      scales[i] = p.scales_tab[i][ex];
    }
  }
  const int r0 = blockIdx.y * kI8Rows;
  if (r0 >= rows) return;
  if (p.off)
    for (int i = 0; i < p.nmat; ++i)
      if (!codes[i] || !scales[i] || (reinterpret_cast<uintptr_t>(codes[i]) & 15u) ||
          (reinterpret_cast<uintptr_t>(scales[i]) & 3u)) {
        atomicExch(p.dev_err, kErrArg);
        return;
      }
  const int64_t n = (int64_t)blockIdx.x * kTileRows + threadIdx.x;
  int acc[2][kI8Rows] = {};
  for (int c = 0; c < p.chunks; ++c)
    for (int g = 0; g < 8; ++g) {
      const int k = c * 128 + g * 16;
      if (k >= p.K) break;
      for (int i = 0; i < p.nmat; ++i) {
        const int4 w = *reinterpret_cast<const int4*>(codes[i] + code_offset(p.chunks, n, c, g * 16));
#pragma unroll
        for (int r = 0; r < kI8Rows; ++r) {
          if (r0 + r >= rows) break;
          const int4 a = *reinterpret_cast<const int4*>(p.xcodes + (size_t)(lo + r0 + r) * p.K + k);
          acc[i][r] = __dp4a(w.x, a.x, __dp4a(w.y, a.y, __dp4a(w.z, a.z, __dp4a(w.w, a.w, acc[i][r]))));
        }
      }
    }
  if (n >= p.N) return;
#pragma unroll
  for (int r = 0; r < kI8Rows; ++r) {
    if (r0 + r >= rows) break;
    const size_t m = (size_t)(lo + r0 + r);
    const float sx = p.xscales[m];
    const float a = __int2float_rn(acc[0][r]) * scales[0][n] * sx;
    if (p.nmat == 2)
      reinterpret_cast<__nv_bfloat16*>(p.out)[m * p.N + n] =
          __float2bfloat16_rn(silu_mul(a, __int2float_rn(acc[1][r]) * scales[1][n] * sx));
    else if (p.out_bf16)
      reinterpret_cast<__nv_bfloat16*>(p.out)[m * p.N + n] = __float2bfloat16_rn(a);
    else
      reinterpret_cast<float*>(p.out)[m * p.N + n] = a;
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

cudaError_t launch_i8_gemm(const I8Params& p, cudaStream_t stream) {
  const int rows = p.off ? std::min(p.max_rows, p.M) : p.M;
  const dim3 grid((unsigned)row_tiles(p.N), (unsigned)((rows + kI8Rows - 1) / kI8Rows), (unsigned)(p.off ? p.E : 1));
  return launch_dep(qgemm_i8_kernel, grid, dim3(128), 0, stream, p);
}

}  // namespace qg
