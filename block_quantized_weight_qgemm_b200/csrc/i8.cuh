// i8.cuh -- parameters of the int8 GEMM, shared by its kernels and the host layer.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace qg {

constexpr int kI8SMs = 148;  // of a B200, for the rules that weigh tilings
constexpr int64_t kI8MaxK = 131072;  // |sum| <= K * 128 * 127 stays inside int32
constexpr int kI8MaxUnits = 0x3FFFFFFF;  // of a call: a unit's number plus a grid's step stays an int

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
  int falling;      // with offsets that fall, the experts' units could pass kI8MaxUnits
  const uint8_t* const* codes_tab[2];
  const float* const* scales_tab[2];
  // Tiling (i8_plan)
  int pair;         // CTA pairs: tiles of 256 channels x 256 rows
  int tiles;        // channel tiles
  int NB;           // rows of x per unit at most (MMA N), a multiple of 16
  int box;          // rows per TMA box
  int b_tiles;      // row tiles of a plain call (routed: of an expert, at most)
  int units, full;  // plain: units; the first `full` take all of K, those after write partials
  int S;            // K ranges of a split tile
  int runs;         // above 0: CTAs that all chunks are dealt out to (then units = 2 runs, each with a partial)
  int cs;           // CTAs of a cluster that share a unit's K (then one unit per cluster)
  int fused;        // x is quantised in the product's kernel, from x
  int x_bytes;      // shared memory of its codes
  const uint16_t* x;  // bf16 [M][K] (fused)
  int one_set;      // one accumulator set instead of two (two matrices, tiles of more than 128 rows)
  int stages, stage_bytes, tmem_cols;
  int w_again;      // a weight tile is read by more than one unit
  int* ws;          // partials [units - full][NB][channels of a tile]
};

void i8_plan(int64_t M, int64_t N, int64_t K, int64_t rows, int nmat, int E, I8Params* p);
size_t i8_partial_bytes(const I8Params& p);
size_t i8_partial_bound(int64_t M, int64_t N, int64_t K);  // i8_partial_bytes of a plain call of at most M rows
cudaError_t launch_i8_gemm(I8Params p, const CUtensorMap& map_x, const CUtensorMap& map_w, cudaStream_t stream);

}  // namespace qg
