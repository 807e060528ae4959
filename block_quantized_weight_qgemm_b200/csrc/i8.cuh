// i8.cuh -- parameters of the int8 GEMM, shared by its kernels and the host layer.
#pragma once
#include <cuda.h>
#include <cstdint>

namespace qg {

constexpr int64_t kI8MaxK = 131072;  // |sum| <= K * 128 * 127 stays inside int32

struct I8Params {
  int M, N, K, chunks;
  int nmat;                    // 1: y; 2: h = SiLU(g) u from two matrices
  const int8_t* xcodes;        // [M][K]
  const float* xscales;        // [M]
  const uint8_t* codes[2];     // tile-major int8 codes of each matrix
  const float* scales[2];      // [N] of each matrix
  void* out;                   // y [M][N] fp32 or bf16, or h [M][N] bf16
  int out_bf16;
  int* dev_err;
  // Routed: rows off[e] .. off[e+1]-1 (clamped to [0, M], max_rows of them at most) belong to
  // expert e, whose buffers come from the tables
  const int* off;
  int E, max_rows;
  const uint8_t* const* codes_tab[2];
  const float* const* scales_tab[2];
};

}  // namespace qg
