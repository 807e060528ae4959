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
#include <cmath>

#include "common.cuh"
#include "dequant.cuh"
#include "i8.cuh"
#include "ptx.cuh"

namespace qg {

// ---------------------------------------------------------------------------------------
// Activations: a warp or a block per row
// ---------------------------------------------------------------------------------------
constexpr float kI8Inv = 1.f / 127.f;
constexpr int kI8QuantThreads = 1024;  // at most

struct I8QuantParams {
  const uint16_t* x;  // bf16 [M][K]
  int64_t M;
  int K;
  int8_t* codes;  // [M][K]
  float* scales;  // [M]
  int early;      // the dependent grid reads only weights before it waits
};

// Eight rounded quotients.  t = x inv + 1.5 2^23 rounds x / s to an integer (in t's low bits) up
// to the error of inv; r = x - q s then says which side of the half step x lies on.  r is exact:
// where it decides, |x| >= s / 2 makes x and q s multiples of s's last place, and |r| is about
// s / 2.  So the code is the one of the exact quotient, ties to even.  A quotient that close to a
// half step is rare (ties of short significands apart): the words that hold one are corrected in
// a branch of their own.
template <bool UP>
__device__ __forceinline__ uint2 i8_codes8(const uint4& v, float up, float inv, float s, float half) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  const float magic = 12582912.f;
  float x[8];
  int c[8];
  float far = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = __uint_as_float((i & 1) ? (w[i >> 1] & 0xFFFF0000u) : (w[i >> 1] << 16));
    if (UP) x[i] *= up;
    const float t = fmaf(x[i], inv, magic);
    c[i] = __float_as_int(t);
    far = fmaxf(far, fabsf(fmaf(-(t - magic), s, x[i])));
  }
  if (far >= half) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float r = fmaf(-(__int_as_float(c[i]) - magic), s, x[i]);
      if (fabsf(r) > half || (fabsf(r) == half && (c[i] & 1))) c[i] += r > 0.f ? 1 : -1;
    }
  }
  return make_uint2(__byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410),
                    __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410));
}

// What a row's largest |x| (bf16 bits) makes of it.
struct I8Row {
  float scale;         // as it leaves: NaN for a row that is not finite
  float up;            // a row near the bottom of the range is lifted by this exact power of two, scale and
  float s, half, inv;  // all, so that the reciprocal is finite and the residual normal
  bool none;           // all codes 0
  __device__ __forceinline__ explicit I8Row(uint32_t bits) {
    const float amax = __uint_as_float(bits << 16);
    none = bits >= 0x7F80u || bits == 0;
    scale = bits < 0x7F80u ? __fmul_rn(amax, kI8Inv) : __int_as_float(0x7FC00000);
    up = amax >= 0x1p-60f ? 1.f : 0x1p64f;
    s = scale * up;
    half = 0.5f * s;
    inv = none ? 0.f : __frcp_rn(s);
  }
  __device__ __forceinline__ uint2 codes(const uint4& v) const {
    if (none) return make_uint2(0u, 0u);
    return up == 1.f ? i8_codes8<false>(v, up, inv, s, half) : i8_codes8<true>(v, up, inv, s, half);
  }
};
__device__ __forceinline__ uint32_t i8_max16(uint32_t top, const uint4& a) {  // two maxima of 16 bits
  top = __vmaxu2(top, __vmaxu2(a.x & 0x7FFF7FFFu, a.y & 0x7FFF7FFFu));
  return __vmaxu2(top, __vmaxu2(a.z & 0x7FFF7FFFu, a.w & 0x7FFF7FFFu));
}

// Per row: the largest |x| as bf16 bits (which order like the magnitudes, infinities and NaN above
// every finite value), the scale, the codes.  A row is one warp's (WARP: short rows, eight to a
// block) or a block's, each thread with up to R words of eight elements in registers; what is left of a
// long row is read twice.
// Bound by memory: 2048 x 5120 in 7.7 us (31 MB; a launch's latency and one wave of blocks), 8192 x
// 5120 in 23 us (5.4 TB/s).
template <int R, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : kI8QuantThreads) qgemm_i8_quant_kernel(const I8QuantParams p) {
  // The GEMM that follows starts its set-up and its weight copies before it waits for this grid.  A
  // plain one reads nothing else by then, and may launch at once (weights come from a grid that has
  // ended, as the header says); a routed one also reads offsets and tables, which the grid before
  // this one may have written.
  if (p.early) griddep_launch_dependents();
  griddep_wait();
  if (!p.early) griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t m = WARP ? (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
  if (WARP && m >= p.M) return;
  const int k0 = (WARP ? lane : (int)threadIdx.x) * 8, step = WARP ? 256 : (int)blockDim.x * 8;
  const uint16_t* xr = p.x + m * p.K;
  uint4 v[R];
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const int k = k0 + j * step;
    v[j] = k < p.K ? *reinterpret_cast<const uint4*>(xr + k) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int j = 0; j < R; ++j) top = i8_max16(top, v[j]);
  if (!WARP)
    for (int k = k0 + R * step; k < p.K; k += step) top = i8_max16(top, *reinterpret_cast<const uint4*>(xr + k));
  uint32_t bits = __reduce_max_sync(0xffffffffu, max(top & 0xFFFFu, top >> 16));
  if (!WARP) {
    __shared__ uint32_t red[kI8QuantThreads / 32];
    if (lane == 0) red[threadIdx.x >> 5] = bits;
    __syncthreads();
    bits = __reduce_max_sync(0xffffffffu, lane < (int)(blockDim.x >> 5) ? red[lane] : 0u);
  }
  const I8Row row(bits);
  if (k0 == 0) p.scales[m] = row.scale;
  int8_t* cr = p.codes + m * p.K;
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const int k = k0 + j * step;
    if (k < p.K) *reinterpret_cast<uint2*>(cr + k) = row.codes(v[j]);
  }
  if (!WARP)
    for (int k = k0 + R * step; k < p.K; k += step)
      *reinterpret_cast<uint2*>(cr + k) = row.codes(*reinterpret_cast<const uint4*>(xr + k));
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
// accumulator sets in tensor memory let the epilogue of a unit run under the MMAs of the next (one set
// where i8_plan says so).
// Warp 0 brings each 128-K chunk's weights into a ring of shared-memory stages (one 16 KB bulk copy
// per matrix) and warp 2 the rows of x (one or more boxes); apart, because the weights need not wait
// for the quantisation kernel and fill the ring under it.  Warp 1 issues four M128 N(rows) K32 MMAs
// per chunk and matrix, warps 3..10 read the accumulators out.
//
// Bound by the weights' stream up to about 100 rows: an SM takes 51 GB per ms through a ring of 200 KB, all of
// them 7 TB/s.  17408 x 5120 (89 MB) takes 17.3 us with 1 row and 18.7 with 64, of which 12.6 are the stream
// (its slope in K) and the rest the quantisation's and the launch's start and end; 512 routed experts of
// 2 x 512 x 2048, 64 tokens top-10, run at the measured copy rate.  From there to 256 rows (25 us) by what
// the SMs draw from L2, 11 to 13 TB/s: every tile reads all rows again.
// ---------------------------------------------------------------------------------------
constexpr int kI8EpiWarps = 8;
constexpr int kI8XWarp = 2, kI8EpiWarp0 = 3;
constexpr int kI8Threads = (kI8EpiWarp0 + kI8EpiWarps) * 32;
constexpr int kI8Strip = 128;  // rows per epilogue warp: half of a unit's 256 at most
constexpr int kI8MaxStages = 12;
constexpr int kI8List = 128;  // units of a CTA found ahead (routed)
constexpr int kI8FusedRegs = 8;              // words of a row per lane of the fused quantisation
constexpr int kI8FusedK = kI8FusedRegs * 256;
constexpr int kI8FusedRows = 2 * (kI8Threads / 32 - kI8XWarp);

__device__ __forceinline__ void i8_mma(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor, kind::i8: D s32 (2), A and B signed 8-bit (1).
__device__ __forceinline__ uint32_t i8_idesc(int m, int n) {
  return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
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

// How a kernel finds its units: whole tiles, and tiles of a last round split over K; the same with x quantised
// in the kernel; all tiles' chunks dealt out evenly, a run of them to each CTA; those of the experts.
enum I8Mode { kI8Plain, kI8Fused, kI8Runs, kI8Routed };

// One unit of work: rows row0 .. row0+rows-1 of x, a 128-channel tile (for a CTA pair: its two), chunks
// c0 .. c1-1, and the buffers of each matrix.  part >= 0: the int32 partial it writes.
template <int NMAT>
struct I8Unit {
  int t, row0, rows, c0, c1, part;
  const uint8_t* w[NMAT];  // the matrix's codes
  const float* sc[NMAT];   // its channel scales
};

// Rows of expert ex: its first row and how many of them are computed.
__device__ __forceinline__ int i8_expert_rows(const I8Params& p, int ex, int& lo) {
  lo = min(max(__ldg(p.off + ex), 0), p.M);
  return min(min(max(__ldg(p.off + ex + 1), lo), p.M) - lo, p.max_rows);
}

// First chunk (of all tiles' chunks in a row) of CTA i's run: at most 148 runs of 148 tiles of 1024 chunks, so
// the product fits an int.
__device__ __forceinline__ int i8_run_start(const I8Params& p, int i) {
  return (int)((unsigned)(i * (p.tiles * p.b_tiles * p.chunks)) / (unsigned)p.runs);
}

// Unit u.  Routed: pre[e] is the number of units before expert e's.  Plain: the first `full` units
// take all of K, the tiles after them are split in S ranges each.  Runs: units i and runs + i are the parts of
// CTA i's run in its first tile and in the next (a run is no longer than a tile).
template <int NMAT, int MODE>
__device__ __forceinline__ I8Unit<NMAT> i8_unit(const I8Params& p, const int* pre, int u) {
  I8Unit<NMAT> U;
  U.c0 = 0;
  U.c1 = p.chunks;
  U.part = -1;
  if constexpr (MODE == kI8Routed) {
    int a = 0, b = p.E;  // the last e with pre[e] <= u
    while (b - a > 1) {
      const int m = (a + b) >> 1;
      if (pre[m] <= u) a = m;
      else b = m;
    }
    int lo;
    const int n = i8_expert_rows(p, a, lo);
    const int r = u - pre[a], bts = (n + p.NB - 1) / p.NB;
    const int bt = r % bts, nb = ((n + bts - 1) / bts + 15) & ~15;  // tiles of like size
    U.t = r / bts;
    U.row0 = lo + bt * nb;
    U.rows = min(nb, n - bt * nb);
#pragma unroll
    for (int m = 0; m < NMAT; ++m) {
      U.w[m] = p.codes_tab[m][a];
      U.sc[m] = p.scales_tab[m][a];
    }
  } else {
    if constexpr (MODE == kI8Runs) {
      const int i = u < p.runs ? u : u - p.runs;
      const int b0 = i8_run_start(p, i), b1 = i8_run_start(p, i + 1);
      const int tile = b0 / p.chunks, at = tile * p.chunks;
      U.part = 2 * i + (u < p.runs ? 0 : 1);
      U.c0 = u < p.runs ? b0 - at : 0;
      U.c1 = u < p.runs ? min(b1 - at, p.chunks) : b1 - at - p.chunks;
      u = tile + (u < p.runs ? 0 : 1);
    } else if (u >= p.full) {
      const int r = u - p.full, s = r % p.S;
      U.part = r;
      U.c0 = (int)((int64_t)s * p.chunks / p.S);
      U.c1 = (int)((int64_t)(s + 1) * p.chunks / p.S);
      u = p.full + r / p.S;
    }
    const int bt = u % p.b_tiles;
    U.t = u / p.b_tiles;
    U.row0 = bt * p.NB;
    U.rows = min(p.NB, p.M - bt * p.NB);
#pragma unroll
    for (int m = 0; m < NMAT; ++m) {
      U.w[m] = p.codes[m];
      U.sc[m] = p.scales[m];
    }
  }
  return U;
}

// The scales of one epilogue warp's part of a unit: its lane's channel n, and the rows of its
// 16-row blocks (block b of the warp is block 2 b + hw of the unit; entry 16 b + r is its row r).
template <int NMAT>
struct I8Scales {
  float sw[NMAT], sx[kI8Strip / 32];
  __device__ __forceinline__ void fetch(const I8Params& p, const float* xscales, const I8Unit<NMAT>& U, int64_t n,
                                        int hw, int lane) {
#pragma unroll
    for (int m = 0; m < NMAT; ++m) sw[m] = n < p.N ? __ldg(U.sc[m] + n) : 0.f;
#pragma unroll
    for (int e = 0; e < kI8Strip / 32; ++e) {
      const int row = (2 * (2 * e + (lane >> 4)) + hw) * 16 + (lane & 15);
      sx[e] = row < U.rows ? xscales[U.row0 + row] : 0.f;
    }
  }
};

// A unit that a cluster of cs CTAs splits over K (one unit per cluster): 16-row block b is summed and
// written by rank b % cs.  The others send it their sums through distributed shared memory, into the ring
// of its stages, which is free by then: [source][own block][matrix][16 rows / 4][128 channels][4 rows].
constexpr uint32_t kI8Block = 16 * kTileRows * 4;

template <int NMAT>
__device__ __forceinline__ uint32_t i8_block_at(int rows, int cs, int source, int b, int m) {
  const int own = ((rows + 15) / 16 + cs - 1) / cs;  // blocks a rank owns at most
  return (uint32_t)((source * own + b / cs) * NMAT + m) * kI8Block;
}

template <int NMAT>
__device__ __forceinline__ void i8_send(const I8Params& p, const I8Unit<NMAT>& V, uint32_t d, int hw, int ch,
                                        uint32_t ring, int rank) {
  for (int cb = hw * 16; cb < V.rows; cb += 32) {
    const int owner = (cb >> 4) % p.cs;
    if (owner == rank) continue;
    uint32_t v[NMAT][16];
#pragma unroll
    for (int m = 0; m < NMAT; ++m) i8_tmem_ld16(d + (uint32_t)(m * p.NB + cb), v[m]);
    tmem_ld_wait();
#pragma unroll
    for (int m = 0; m < NMAT; ++m) {
      const uint32_t at = mapa_shared(
          ring + i8_block_at<NMAT>(V.rows, p.cs, rank < owner ? rank : rank - 1, cb >> 4, m) + (uint32_t)ch * 16,
          (uint32_t)owner);
#pragma unroll
      for (int r = 0; r < 16; r += 4)
        asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + (uint32_t)(r / 4) * kTileRows * 16),
                     "r"(v[m][r]), "r"(v[m][r + 1]), "r"(v[m][r + 2]), "r"(v[m][r + 3])
                     : "memory");
    }
  }
}

// The read-out of one warp's part of a unit's accumulators (d: its lane quarter's first column).
// ch: the lane's channel within the unit, of `width`; ring: where a cluster's other CTAs have sent their
// sums for this rank's blocks (CL).
template <int NMAT, bool CL, bool PARTS>
__device__ __forceinline__ void i8_read_out(const I8Params& p, const I8Unit<NMAT>& V, uint32_t d, int hw, int64_t n,
                                            int ch, int width, const float (&sw)[NMAT],
                                            const float (&sxl)[kI8Strip / 32], const uint8_t* ring, int rank) {
  const bool in = n < p.N;
  for (int cb = hw * 16; cb < V.rows; cb += 32) {
    if (CL && (cb >> 4) % p.cs != rank) continue;
    __syncwarp();
    uint32_t v[NMAT][16];
#pragma unroll
    for (int m = 0; m < NMAT; ++m) i8_tmem_ld16(d + (uint32_t)(m * p.NB + cb), v[m]);
    // the block's 16 row scales, of which lane 16 (b & 1) + r of entry b >> 1 holds r
    const int b = cb >> 5;
    const float sxb = b < 4 ? (b < 2 ? sxl[0] : sxl[1]) : (b < 6 ? sxl[2] : sxl[3]);
    float sx[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) sx[r] = __shfl_sync(0xffffffffu, sxb, ((b & 1) << 4) + r);
    tmem_ld_wait();
    for (int o = 0; CL && o < p.cs - 1; ++o)
#pragma unroll
      for (int m = 0; m < NMAT; ++m) {
        const uint8_t* at = ring + i8_block_at<NMAT>(V.rows, p.cs, o, cb >> 4, m) + ch * 16;
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
          const uint4 a = *reinterpret_cast<const uint4*>(at + (r / 4) * kTileRows * 16);
          v[m][r] += a.x, v[m][r + 1] += a.y, v[m][r + 2] += a.z, v[m][r + 3] += a.w;
        }
      }
    const int nr = min(16, V.rows - cb);
    // 16 rows of one channel: a full block without a branch per row, so that its stores follow one
    // another
    auto store = [&](auto* out, size_t pitch, auto f) {
      if (nr == 16) {
#pragma unroll
        for (int r = 0; r < 16; ++r) out[(size_t)r * pitch] = f(r);
      } else {
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (r < nr) out[(size_t)r * pitch] = f(r);
      }
    };
    auto y = [&](int m, int r) { return __int2float_rn((int)v[m][r]) * sw[m] * sx[r]; };
    const size_t at = (size_t)(V.row0 + cb) * p.N + n;
    if (!in) continue;
    if (NMAT == 2)
      store(reinterpret_cast<__nv_bfloat16*>(p.out) + at, p.N,
            [&](int r) { return __float2bfloat16_rn(silu_mul(y(0, r), y(NMAT - 1, r))); });
    else if (PARTS && V.part >= 0)
      store(p.ws + ((size_t)V.part * p.NB + cb) * width + ch, width, [&](int r) { return (int)v[0][r]; });
    else if (p.out_bf16)
      store(reinterpret_cast<__nv_bfloat16*>(p.out) + at, p.N, [&](int r) { return __float2bfloat16_rn(y(0, r)); });
    else
      store(reinterpret_cast<float*>(p.out) + at, p.N, [&](int r) { return y(0, r); });
  }
}

__device__ __forceinline__ void prefetch_l2(const void* a) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(a));
}

// MODE and CL (clusters share units) are template parameters because the code that a launch does not run
// costs it time all the same: with all of it in one kernel, 64 rows by 17408 x 5120 took 20.2 us for 18.7.
template <int NMAT, int MODE, bool CL>
__global__ void __launch_bounds__(kI8Threads, 1) qgemm_i8_kernel(const __grid_constant__ I8Params p,
                                                                 const __grid_constant__ CUtensorMap tm_x) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  // fused: the codes of x, [chunk][NB][128] in the 128-byte swizzle; then the ring of stages
  uint8_t* ring = smem + p.x_bytes;
  const uint32_t xbase = smem_u32(smem), sbase = smem_u32(ring);
  const int NST = p.stages;
  uint64_t* bars = reinterpret_cast<uint64_t*>(ring + (size_t)NST * p.stage_bytes);
  const uint32_t bar_full = smem_u32(bars);
  const uint32_t bar_empty = bar_full + 8 * kI8MaxStages;
  const uint32_t bar_acc = bar_empty + 8 * kI8MaxStages;  // [2] a unit's accumulators are complete
  const uint32_t bar_acc_free = bar_acc + 16;             // [2] the epilogue has read them
  const uint32_t bar_drain = bar_acc_free + 16;
  const uint32_t bar_x = bar_drain + 8;                   // fused: the codes of x are written
  int* ctl = reinterpret_cast<int*>(bars + 2 * kI8MaxStages + 6);
  volatile int* abort_flag = ctl + 1;
  // routed: the CTA's first units, then [E] the units before each expert's
  I8Unit<NMAT>* list = reinterpret_cast<I8Unit<NMAT>*>(ctl + 4);
  int* pre = reinterpret_cast<int*>(list + kI8List);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the CTA's (or its cluster's) place among the units
  const int rank = CL ? (int)cluster_ctarank() : 0;
  const int first = CL ? (int)blockIdx.x / p.cs : (int)blockIdx.x;
  const int stride = CL ? (int)gridDim.x / p.cs : (int)gridDim.x;

  if (warp == 0 && lane == 0) {
    if (MODE != kI8Fused) prefetch_tmap(&tm_x);
    for (int s = 0; s < NST; ++s) {
      mbar_init(bar_full + 8 * s, MODE == kI8Fused ? 1 : 2);  // the producers
      mbar_init(bar_empty + 8 * s, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_acc + 8 * i, 1);
      mbar_init(bar_acc_free + 8 * i, kI8EpiWarps);
    }
    mbar_init(bar_drain, 1);
    mbar_init(bar_x, kI8Threads / 32 - kI8XWarp);
    ctl[1] = 0;
    fence_mbar_init();
  }
  if (warp == 1) i8_tmem_alloc(smem_u32(ctl), (uint32_t)p.tmem_cols);
  int units = p.units;
  if constexpr (MODE == kI8Runs) {
    // this CTA's run lies in one tile or two (or is empty: fewer chunks than CTAs)
    const int b0 = i8_run_start(p, first), b1 = i8_run_start(p, first + 1);
    units = b1 <= b0 ? 0 : (b1 - 1) / p.chunks > b0 / p.chunks ? 2 * p.runs : p.runs;
  }
  if constexpr (MODE == kI8Routed) {
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
    // Falling offsets give rows to several experts: where that makes more units than there are clusters, which take one
    // each, or (calls of hundreds of millions of rows) than an int counts, the call computes nothing.
    bool many = CL && units > stride;
    if (!CL && p.falling) {
      int64_t all = 0;
      for (int e = lane; e < p.E; e += 32) {
        int lo;
        all += (int64_t)((i8_expert_rows(p, e, lo) + p.NB - 1) / p.NB) * p.tiles;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
      many = all > kI8MaxUnits;
    }
    if (many) {
      if (threadIdx.x == 0) atomicExch(p.dev_err, kErrArg);
      units = 0;
    }
    __syncthreads();
    // every thread finds one unit of this CTA, so that the roles below read it in one step
    for (int i = threadIdx.x; i < kI8List; i += kI8Threads) {
      const int64_t u = (int64_t)first + (int64_t)i * stride;
      if (u < units) list[i] = i8_unit<NMAT, MODE>(p, pre, (int)u);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(ctl[0]);
  const int set = NMAT * p.NB;  // columns of one accumulator set
  // use i of the accumulators: the set, and how often that has been used before
  auto acc = [&](int i) { return NMAT == 2 && p.one_set ? 0 : i & 1; };
  auto turn = [&](int i) { return NMAT == 2 && p.one_set ? i : i >> 1; };
  auto unit = [&](int i, int u) {
    I8Unit<NMAT> U =
        MODE == kI8Routed && i < kI8List ? list[i] : i8_unit<NMAT, MODE>(p, pre, u);
    if (CL) {
      U.c0 = (int)((int64_t)rank * p.chunks / p.cs);
      U.c1 = (int)((int64_t)(rank + 1) * p.chunks / p.cs);
    }
    return U;
  };
  I8Unit<NMAT> V;  // (epilogue) the unit at hand
  I8Scales<NMAT> vs;
  bool held = false;  // (epilogue, clusters) its accumulators are complete and not read out yet
  const int q = warp & 3, hw = (warp - kI8EpiWarp0) >> 2, ch = q * 32 + lane;

  // ------------------------------------------------------------ fused: quantise x
  // The producer and the issuer go ahead; the other nine warps take two rows each.  Row r's byte k of
  // a chunk goes to group (k / 16) ^ (r & 7) of its 128 bytes.
  float* sx_own = reinterpret_cast<float*>(list);  // (a plain call has no list)
  if (MODE == kI8Fused && warp >= kI8XWarp) {
    griddep_wait();
    const int c0 = CL ? rank * p.chunks / p.cs : 0;  // chunks of this CTA's range
    const int c1 = CL ? (rank + 1) * p.chunks / p.cs : p.chunks;
    constexpr int kWarps = kI8FusedRows / 2;  // a warp takes two rows at once
    uint4 v[2][kI8FusedRegs];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < kI8FusedRegs; ++j) {
        const int r = warp - kI8XWarp + i * kWarps, at = (j * 32 + lane) * 8;
        v[i][j] = r < p.M && at < p.K ? *reinterpret_cast<const uint4*>(p.x + (size_t)r * p.K + at)
                                      : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = warp - kI8XWarp + i * kWarps;
      if (r >= p.M) break;
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < kI8FusedRegs; ++j) top = i8_max16(top, v[i][j]);
      const I8Row row(__reduce_max_sync(0xffffffffu, max(top & 0xFFFFu, top >> 16)));
      if (lane == 0) sx_own[r] = row.scale;
#pragma unroll
      for (int j = 0; j < kI8FusedRegs; ++j) {
        const int at = (j * 32 + lane) * 8, c = at >> 7, g = (at & 127) >> 4;
        if (at < p.K && c >= c0 && c < c1)
          *reinterpret_cast<uint2*>(smem + (size_t)((c - c0) * p.NB + r) * 128 + ((g ^ (r & 7)) << 4) + (at & 8)) =
              row.codes(v[i][j]);
      }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the MMAs read the codes
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_x);
  }

  if (warp == 0 || (warp == kI8XWarp && MODE != kI8Fused)) {
    // ------------------------------------------------------------ producers: weights, rows of x
    if (lane == 0) {
      const bool x = warp == kI8XWarp;
      const uint64_t pol = x || p.w_again ? policy_evict_last() : policy_evict_first();
      RingPos sp;
      int issued = 0, i = 0;
      bool ok = true;
      if (x) griddep_wait();  // the codes of x come from the preceding grid
      for (int u = first; u < units && ok; u += stride, ++i) {
        const I8Unit<NMAT> U = unit(i, u);
        const int boxes = (U.rows + p.box - 1) / p.box;
        const uint32_t bytes = x ? (uint32_t)(boxes * p.box * 128) : (uint32_t)(NMAT * kWCodeBytes);
        for (int c = U.c0; c < U.c1; ++c) {
          if (issued >= NST &&
              !mbar_wait(bar_empty + 8 * sp.slot, sp.phase ^ 1u, abort_flag, p.dev_err, kErrTimeout)) {
            ok = false;
            break;
          }
          const uint32_t fb = bar_full + 8 * sp.slot;
          const uint32_t st = sbase + (uint32_t)(sp.slot * p.stage_bytes);
          mbar_arrive_expect_tx(fb, bytes);
          if (x) {
            for (int b = 0; b < boxes; ++b)
              i8_load_x(st + NMAT * kWCodeBytes + (uint32_t)(b * p.box * 128), &tm_x, fb, c * 128,
                        U.row0 + b * p.box, pol);
          } else {
#pragma unroll
            for (int m = 0; m < NMAT; ++m)
              bulk_load(st + m * kWCodeBytes, U.w[m] + ((int64_t)U.t * p.chunks + c) * kWCodeBytes, kWCodeBytes, fb,
                        pol);
            if (c == U.c0) {
              // the unit's channel scales, into L2 ahead of the epilogue
              const int64_t n0 = (int64_t)U.t * kTileRows;
#pragma unroll
              for (int m = 0; m < NMAT; ++m)
                for (int64_t n = n0; n < n0 + kTileRows && n < p.N; n += 32) prefetch_l2(U.sc[m] + n);
            }
          }
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
      for (int u = first; u < units && ok; u += stride, ++i) {
        const I8Unit<NMAT> U = unit(i, u);
        const uint32_t idesc = i8_idesc(128, (U.rows + 15) & ~15);
        if (MODE == kI8Fused && i == 0 && !mbar_wait_spin(bar_x, 0, false, abort_flag, p.dev_err, kErrTimeout)) {
          ok = false;
          break;
        }
        const uint32_t d = tmem + (uint32_t)(acc(i) * set);
        if (turn(i) > 0) {
          if (!mbar_wait_spin(bar_acc_free + 8 * acc(i), (uint32_t)(turn(i) - 1) & 1u, false, abort_flag,
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
          const uint64_t bd = smem_desc_sw128(MODE == kI8Fused ? xbase + (uint32_t)((c - U.c0) * p.NB * 128)
                                                      : st + NMAT * kWCodeBytes);
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
        i8_commit(bar_acc + 8 * acc(i));
      }
      // every MMA has completed before the CTA may free its tensor memory
      i8_commit(bar_drain);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(bar_drain, 0) && globaltimer_ns() - t0 < kWaitLimitNs) {
      }
    }
    __syncwarp();
  } else if (warp >= kI8EpiWarp0) {
    // ------------------------------------------------------------ epilogue
    // Two warps per lane quarter take alternate 16-row blocks of a unit.  A unit's scales are
    // loaded while the unit before it is computed and read out.
    const uint32_t lane_base = (uint32_t)(q * 32) << 16;
    griddep_wait();  // the scales of x come from the preceding grid
    griddep_launch_dependents();
    // fused: they come from these warps (and from warp 2, which has none of its own work here)
    if (MODE == kI8Fused &&
        !__all_sync(0xffffffffu, mbar_wait(bar_x, 0, abort_flag, p.dev_err, kErrTimeout))) units = 0;
    I8Unit<NMAT> U;
    I8Scales<NMAT> sc;
    auto fetch = [&](int i, int u) {
      U = unit(i, u);
      sc.fetch(p, MODE == kI8Fused ? sx_own : p.xscales, U, (int64_t)U.t * kTileRows + ch, hw, lane);
    };
    if (first < units) fetch(0, first);
    int i = 0;
    for (int u = first; u < units; u += stride, ++i) {
      V = U;
      vs = sc;
      if (u + stride < units) fetch(i + 1, u + stride);
      bool ok = mbar_wait(bar_acc + 8 * acc(i), (uint32_t)turn(i) & 1u, abort_flag, p.dev_err, kErrTimeout);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      if (CL) {
        held = true;
        break;
      }
      i8_read_out<NMAT, false, MODE == kI8Plain || MODE == kI8Runs>(p, V, tmem + lane_base + (uint32_t)(acc(i) * set), hw,
                                                 (int64_t)V.t * kTileRows + ch, ch, kTileRows, vs.sw, vs.sx, nullptr, 0);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_acc_free + 8 * acc(i));
    }
  }

  // ------------------------------------------------------------ sum over the cluster
  if (CL) {
    // every CTA has all its sums: the rings hold nothing any more
    cluster_sync_all();
    const uint32_t d = tmem + ((uint32_t)(q * 32) << 16);
    if (held) i8_send<NMAT>(p, V, d, hw, ch, sbase, rank);
    cluster_sync_all();
    if (held)
      i8_read_out<NMAT, true, false>(p, V, d, hw, (int64_t)V.t * kTileRows + ch, ch, kTileRows, vs.sw, vs.sx, ring,
                                     rank);
  }

  // ------------------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    i8_tmem_dealloc(tmem, (uint32_t)p.tmem_cols);
  }
}

// ---------------------------------------------------------------------------------------
// Wide plain calls (more than kI8PairRows rows, see i8_plan): the same roles on CTA pairs.  A tile is 256 channels (128 in
// each CTA's tensor memory) x 256 rows; each CTA loads its own 128 channels and half of the rows,
// 32 KB per 128-K chunk where a lone CTA's 128 x 256 tile takes 48 KB for the same MMA time.  All
// loads of a stage count on the even CTA's barrier (the tile-major codes by a tensor map too), so no
// thread stands between the copies and the MMAs.
//
// Bound by the tensor pipe and the power cap: 2048 rows by 17408 x 5120 take 120 us (3.0 POP/s) without the
// quantisation, the pipe 79 % busy while the SMs are, at 1.63 GHz; run for seconds on end 150 us, where
// cuBLAS takes 288 for the same product in bf16.
// ---------------------------------------------------------------------------------------
constexpr int kI8PairStage = 2 * kWCodeBytes;
constexpr int kI8PairStages = 7;

__device__ __forceinline__ void i8_mma_pair(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kI8Threads, 1)
    qgemm_i8_pair_kernel(const __grid_constant__ I8Params p, const __grid_constant__ CUtensorMap tm_x,
                         const __grid_constant__ CUtensorMap tm_w) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  constexpr int NST = kI8PairStages;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + NST * kI8PairStage);
  const uint32_t bar_full = smem_u32(bars);       // (even CTA) both CTAs' loads of the stage
  const uint32_t bar_empty = bar_full + 8 * NST;  // the stage's MMAs are done
  const uint32_t bar_acc = bar_empty + 8 * NST;   // [2] a tile's accumulators are complete
  const uint32_t bar_acc_free = bar_acc + 16;     // [2] (even CTA) both epilogues have read them
  const uint32_t bar_drain = bar_acc_free + 16;
  int* ctl = reinterpret_cast<int*>(bars + 2 * NST + 6);
  volatile int* abort_flag = ctl + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pid = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tm_x);
    prefetch_tmap(&tm_w);
    for (int s = 0; s < NST; ++s) {
      mbar_init(bar_full + 8 * s, 2);  // both producers
      mbar_init(bar_empty + 8 * s, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_acc + 8 * i, 1);
      mbar_init(bar_acc_free + 8 * i, 2 * kI8EpiWarps);
    }
    mbar_init(bar_drain, 1);
    ctl[1] = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(ctl), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers are initialised before any load or commit counts on them
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(ctl[0]);

  if (warp == 0 || warp == kI8XWarp) {
    // ------------------------------------------------------------ producers (of this CTA's half)
    if (lane == 0) {
      const bool x = warp == kI8XWarp;
      const uint64_t pol = policy_evict_last();
      const uint32_t full0 = mapa_shared(bar_full, 0);
      RingPos sp;
      int issued = 0;
      bool ok = true;
      if (x) griddep_wait();  // the codes of x come from the preceding grid
      for (int u = pid; u < p.units && ok; u += pairs) {
        const I8Unit<1> U = i8_unit<1, kI8Plain>(p, nullptr, u);
        const int64_t t = 2 * (int64_t)U.t + rank;
        const int half = ((U.rows + 31) & ~31) >> 1;  // rows of the MMA's N that each CTA holds
        for (int c = U.c0; c < U.c1; ++c) {
          if (issued >= NST &&
              !mbar_wait(bar_empty + 8 * sp.slot, sp.phase ^ 1u, abort_flag, p.dev_err, kErrTimeout)) {
            ok = false;
            break;
          }
          const uint32_t st = sbase + (uint32_t)(sp.slot * kI8PairStage), fb = full0 + 8u * (uint32_t)sp.slot;
          if (rank == 0)  // both halves
            mbar_arrive_expect_tx(bar_full + 8 * sp.slot, x ? (uint32_t)p.box * 256u : 2u * kWCodeBytes);
          if (x)
            tma_load_2d_pair(st + kWCodeBytes, &tm_x, fb, c * 128, U.row0 + (int)rank * half, pol);
          else  // (a tile past the matrix reads zeros)
            tma_load_2d_pair(st, &tm_w, fb, 0, (int)((t * p.chunks + c) * kTileRows), pol);
          sp.next(NST);
          ++issued;
        }
      }
      if (!ok) {
        // the copies in flight count on the even CTA's barrier: give them a fixed grace period
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 200000) __nanosleep(1000);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    if (rank == 0 && lane == 0) {
      RingPos sp;
      bool ok = true;
      int i = 0;
      for (int u = pid; u < p.units && ok; u += pairs, ++i) {
        const I8Unit<1> U = i8_unit<1, kI8Plain>(p, nullptr, u);
        const uint32_t idesc = i8_idesc(256, (U.rows + 31) & ~31);
        const uint32_t d = tmem + (uint32_t)((i & 1) * 256);
        if (i >= 2) {
          if (!mbar_wait_spin(bar_acc_free + 8 * (i & 1), (uint32_t)((i >> 1) - 1) & 1u, true, abort_flag,
                              p.dev_err, kErrTimeout)) {
            ok = false;
            break;
          }
          tc_fence_after();
        }
        for (int c = U.c0; c < U.c1; ++c) {
          if (!mbar_wait_spin(bar_full + 8 * sp.slot, sp.phase, true, abort_flag, p.dev_err, kErrTimeout)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t st = sbase + (uint32_t)(sp.slot * kI8PairStage);
          const uint64_t ad = smem_desc_sw128(st), bd = smem_desc_sw128(st + kWCodeBytes);
#pragma unroll
          for (int kb = 0; kb < 4; ++kb)
            i8_mma_pair(d, ad + (uint64_t)(kb * 2), bd + (uint64_t)(kb * 2), idesc, (c != U.c0 || kb != 0) ? 1u : 0u);
          mma_commit_pair(bar_empty + 8 * sp.slot);
          sp.next(NST);
        }
        if (!ok) break;
        mma_commit_pair(bar_acc + 8 * (i & 1));
      }
      mma_commit_pair(bar_drain);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(bar_drain, 0) && globaltimer_ns() - t0 < kWaitLimitNs) {
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue (of this CTA's channels)
    const int q = warp & 3, hw = (warp - kI8EpiWarp0) >> 2, ch = (int)rank * kTileRows + q * 32 + lane;
    const uint32_t lane_base = (uint32_t)(q * 32) << 16;
    const uint32_t free0 = mapa_shared(bar_acc_free, 0);
    griddep_wait();  // the scales of x come from the preceding grid
    griddep_launch_dependents();
    I8Unit<1> U;
    I8Scales<1> sc;
    auto fetch = [&](int u) {
      U = i8_unit<1, kI8Plain>(p, nullptr, u);
      sc.fetch(p, p.xscales, U, (int64_t)U.t * 2 * kTileRows + ch, hw, lane);
    };
    if (pid < p.units) fetch(pid);
    int i = 0;
    for (int u = pid; u < p.units; u += pairs, ++i) {
      const I8Unit<1> V = U;
      const I8Scales<1> vs = sc;
      if (u + pairs < p.units) fetch(u + pairs);
      bool ok = mbar_wait(bar_acc + 8 * (i & 1), (uint32_t)(i >> 1) & 1u, abort_flag, p.dev_err, kErrTimeout);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      i8_read_out<1, false, true>(p, V, tmem + lane_base + (uint32_t)((i & 1) * 256), hw,
                                  (int64_t)V.t * 2 * kTileRows + ch, ch, 2 * kTileRows, vs.sw, vs.sx, nullptr, 0);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (rank == 0) mbar_arrive(bar_acc_free + 8 * (i & 1));
        else mbar_arrive_cluster_relaxed(free0 + 8u * (uint32_t)(i & 1));
      }
    }
  }

  // ------------------------------------------------------------ teardown
  // neither CTA leaves, or frees tensor memory the pair's MMAs write, while its peer may use it
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// Sum of the K ranges' partials of the split tiles (integers: any order gives the same bits),
// scales, output.  One block per 8 rows of a split tile.
constexpr int kI8ReduceRows = 8;
constexpr int kI8ReduceLoads = 4;  // partials loaded together
__global__ void __launch_bounds__(256) qgemm_i8_reduce_kernel(const I8Params p) {
  griddep_launch_dependents();
  griddep_wait();
  const int width = p.pair ? 2 * kTileRows : kTileRows;
  const int u = p.full + blockIdx.x;  // the tile
  // its partials: S in a row, or (runs) one of each CTA whose run reaches into it
  int first = blockIdx.x * p.S, count = p.S;
  if (p.runs) {
    const int a = u * p.chunks, b = a + p.chunks;
    first = (int)((unsigned)(a * p.runs) / (unsigned)(p.tiles * p.b_tiles * p.chunks));
    while (i8_run_start(p, first + 1) <= a) ++first;
    for (count = 1; first + count < p.runs && i8_run_start(p, first + count) < b;) ++count;
  }
  const int row0 = u % p.b_tiles * p.NB, rows = min(p.NB, p.M - row0);
  const int64_t n0 = (int64_t)(u / p.b_tiles) * width;
  const int quads = width / 4;  // threads along a row
  const int64_t n = n0 + threadIdx.x % quads * 4;
  for (int r = blockIdx.y * kI8ReduceRows + threadIdx.x / quads; r < min(rows, (int)(blockIdx.y + 1) * kI8ReduceRows);
       r += 256 / quads) {
    const int* src = p.ws + (size_t)r * width + threadIdx.x % quads * 4;
    int4 a = make_int4(0, 0, 0, 0);
    for (int s0 = 0; s0 < count; s0 += kI8ReduceLoads) {
      int4 v[kI8ReduceLoads];
#pragma unroll
      for (int j = 0; j < kI8ReduceLoads; ++j) {
        const int i = first + s0 + j;
        // a run that began in the tile before has this one as its second part
        const int part = !p.runs ? i : 2 * i + (i8_run_start(p, i) < u * p.chunks ? 1 : 0);
        const bool none = s0 + j >= count || (p.runs && i8_run_start(p, i) == i8_run_start(p, i + 1));  // (an empty run)
        v[j] = none ? make_int4(0, 0, 0, 0) : __ldcs(reinterpret_cast<const int4*>(src + (size_t)part * p.NB * width));
      }
#pragma unroll
      for (int j = 0; j < kI8ReduceLoads; ++j) a.x += v[j].x, a.y += v[j].y, a.z += v[j].z, a.w += v[j].w;
    }
    const int acc[4] = {a.x, a.y, a.z, a.w};
    const float sx = p.xscales[row0 + r];
    const size_t at = (size_t)(row0 + r) * p.N + n;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (n + e >= p.N) break;
      const float y = __int2float_rn(acc[e]) * p.scales[0][n + e] * sx;
      if (p.out_bf16)
        reinterpret_cast<__nv_bfloat16*>(p.out)[at + e] = __float2bfloat16_rn(y);
      else
        reinterpret_cast<float*>(p.out)[at + e] = y;
    }
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

cudaError_t launch_i8_quant(const uint16_t* x, int64_t M, int64_t K, int8_t* codes, float* scales, bool early,
                            cudaStream_t stream) {
  const I8QuantParams p{x, M, (int)K, codes, scales, early ? 1 : 0};
  const int64_t words = K / 8;
  const auto warps = [&](auto kern) {
    return launch_dep(kern, dim3((unsigned)((M + 7) / 8)), dim3(256), 0, stream, p);
  };
  const auto block = [&](auto kern, int per) {
    const int threads = (int)std::min<int64_t>(kI8QuantThreads, ((words + per - 1) / per + 31) / 32 * 32);
    return launch_dep(kern, dim3((unsigned)M), dim3(threads), 0, stream, p);
  };
  // few rows: a thread per word, for the shortest way through a row.  Many: four words per thread (2048 x
  // 5120: 14.4, 9.6, 7.6, 10.3 us with 1, 2, 4, 8), and of rows that one warp holds in
  // eight words a lane, eight to a block (81920 x 512: 86 us by blocks, 24 by warps; 16 or 20 words a lane
  // ran 20 % slower than blocks)
  if (M <= 2 * kI8SMs) return block(qgemm_i8_quant_kernel<4, false>, 1);
  if (words <= 32) return warps(qgemm_i8_quant_kernel<1, true>);
  if (words <= 64) return warps(qgemm_i8_quant_kernel<2, true>);
  if (words <= 128) return warps(qgemm_i8_quant_kernel<4, true>);
  if (words <= 256) return warps(qgemm_i8_quant_kernel<8, true>);
  return block(qgemm_i8_quant_kernel<4, false>, 4);
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

// A plain call's tiles go out in full rounds over the SMs (or pairs), each tile over all of K; the tiles
// of the last round, if they leave SMs idle, are split over K so that their ranges fill it.  A split
// costs the partials' way through L2 and the reduction's launch, about the time of kI8SplitChunks
// chunks, so it has to save more than those.
//
// Where all units fit on the device as clusters of several CTAs, a cluster splits each unit over K and sums
// in distributed shared memory instead, without a second kernel, at the price of two cluster barriers.
constexpr int kI8SplitChunks = 8, kI8ClusterChunks = 8;
// Above this many rows the pairs' smaller loads per MMA win (but see i8_plan for calls of few tiles): 4096 x 4096 takes
// 17.2, 19.2 us (257, 384 rows) by pairs, 14.5, 16.8 by lone CTAs; 17408 x 5120 37.5, 38.5 (450, 512) against 41.2, 45.4.
constexpr int kI8PairRows = 384;
// Clusters of 0 .. 8 CTAs, one per SM, that start together on a B200.  Its occupancy calculator says 45, 26 and 22 of
// 3, 5 and 6, but the last ones of these wait for others to end: 64 rows, K = 8080, 14.9, 17.4, 18.6, 23.0 us with 42
// to 45 clusters of 3 (46 of 2: 18.1); 251 rows 22.2, 24.0, 30.5 with 24 to 26 of 5, 18.6, 26.6 with 21, 22 of 6.
constexpr int kI8Clusters[9] = {0, 148, 74, 42, 33, 24, 21, 15, 15};

// Tiles of NB rows: how many, and how K is shared.  Returns what `units` of them (expected of a routed call), that
// run at once, take beyond a launch, in us.
static double i8_tile(int64_t M, int64_t rows, int nmat, int E, int NB, int64_t units, I8Params* p) {
  const bool routed = E > 0;
  p->NB = NB;
  p->b_tiles = (int)((rows + NB - 1) / NB);
  p->S = p->cs = 1;
  p->full = p->units = p->runs = 0;
  const int64_t all = (int64_t)p->tiles * p->b_tiles;
  // A chunk takes an SM 0.31 us to stream, or its bytes at 85 GB per ms where the rows of x make up the most of
  // them (a pair's CTA: at 76).
  const double us = std::max(0.31 * nmat, p->pair ? (kWCodeBytes + NB * 64) / 76e3 : (nmat * kWCodeBytes + NB * 128) / 85e3);
  if (!p->pair) {
    const int64_t most = routed ? all * std::min<int64_t>(E, M) : all;
    for (int cs = 2; cs <= 8 && cs <= p->chunks; ++cs)
      if (most <= kI8Clusters[cs] && p->chunks - (p->chunks + cs - 1) / cs > kI8ClusterChunks) p->cs = cs;
  }
  if (!routed) {
    const int64_t slots = p->pair ? kI8SMs / 2 : kI8SMs;
    const int64_t rest = all % slots;
    // as many ranges as balance their own time and the partials' way through L2
    const double way = rest * NB * kTileRows * (p->pair ? 16.0 : 8.0) / 3.5e6;
    int64_t S = rest ? std::min<int64_t>({slots / rest, p->chunks, 1 + (int64_t)std::sqrt(p->chunks * us / way)}) : 1;
    S = (p->chunks + (p->chunks + S - 1) / S - 1) / ((p->chunks + S - 1) / S);  // (no shorter ranges than needed)
    if (S > 1 && p->cs == 1 && p->chunks - (p->chunks + S - 1) / S > kI8SplitChunks) p->S = (int)S;
    if (all <= kI8MaxUnits) {
      p->full = (int)(p->S > 1 ? all - rest : all);
      p->units = (int)(p->S > 1 ? p->full + rest * p->S : all);
    }
  }
  // Tiles that fill neither the SMs nor clusters: all chunks dealt out evenly, where that saves more than the
  // second part of a run, the reduction (6.5 us in all) and the partials' way through L2 (8 bytes per
  // element at 3.5 TB/s) cost.  10240 x 20480 with 1, 64, 256 rows: 52, 53, 69 us in whole tiles on 80
  // SMs, 38, 46, 63 in runs on all; 12288 x 8192 stays with its 96 (23.4 against 23.0, 64 rows 24.3 against 28.9).
  if (!routed && !p->pair && all <= kI8SMs) {
    const int64_t now = p->cs > 1 ? (p->chunks + p->cs - 1) / p->cs + 3 : p->chunks;
    const int64_t then = (all * p->chunks + kI8SMs - 1) / kI8SMs;
    const double cost = 6.5 + 2.0 * kI8SMs * NB * kTileRows * 8 / 3.5e6;
    if ((now - then) * us > cost) {
      p->runs = kI8SMs;
      p->cs = 1;
      p->full = 0;
      p->units = 2 * kI8SMs;
      return then * us + cost;
    }
  }
  const int share = p->cs * p->S;
  double t = (p->chunks + share - 1) / share * us + (nmat == 2 ? 0.0175 : 0.006) * NB;
  if (p->cs > 1) t += 2.85 + 0.016 * NB;
  if (p->S > 1) t += 6.5 + (double)(p->units - p->full) * NB * kTileRows * (p->pair ? 16 : 8) / 3.5e6;
  // beyond 64 SMs, the kernels before and after find fewer that are free: 2048 rows by 64 x 512 6.4 us in 32 pairs
  // (tiles of 64 rows), 7.4 in 64 (32); 16 experts of 100 rows, 320 x 640 7.4 us on 96 SMs (64), 8.7 on 144 (48)
  const int64_t sms = units * share * (p->pair ? 2 : 1);
  return t + 0.014 * (double)std::max<int64_t>(0, sms - 64);
}

// Tiling of a call: rows is M, or (E experts) the most rows an expert has.
void i8_plan(int64_t M, int64_t N, int64_t K, int64_t rows, int nmat, int E, I8Params* p) {
  const bool routed = E > 0;
  p->chunks = (int)k_chunks(FMT_FP8, K);
  const int cap = nmat == 2 ? 128 : 256;
  // Tiles of fewer rows where that puts more SMs to work: as long as all units run at once, what counts is a
  // unit's time (its bytes, its read-out).  256 rows by 512 x 1024: 8.7 us in tiles of 256, 6.5 of 32; 200 by
  // 2048 x 2048 12.7 (208, clusters of 6) and 9.6 (64); 700 by 300 x 2960 21.0 (pairs of 256, K split) and 13.7
  // (32); 8 experts of 256 rows, 1024 x 1024 11.1 (256) and 10.3 (144).  An expert is expected to have an
  // eighth more rows than the mean (which counts rows behind the last expert too), and one at least where rows are
  // fewer than experts: a mean of none took calls of hundreds of units for such as run at once (512 experts of
  // 2 x 512 x 2048, 128 rows, max_rows 128: gate+up 48.8 us in tiles of 32, 44.6 of 128).
  const int64_t mean = routed ? std::max<int64_t>(1, M / E) : 0;
  const int64_t experts = std::min<int64_t>(E, M);
  // (returns whether all units run at once)
  auto tile = [&](bool pair) {
    p->pair = pair;
    p->tiles = (int)(pair ? (row_tiles(N) + 1) / 2 : row_tiles(N));
    const int64_t slots = pair ? kI8SMs / 2 : kI8SMs;
    // tiles of like size: every unit of a round then takes as long (300 rows: two tiles of 160, not 256 and 44)
    const int64_t step = pair ? 32 : 16, b = (rows + cap - 1) / cap;
    auto like = [&](int64_t b) { return (int)((rows + b * step - 1) / (b * step) * step); };
    auto count = [&](int nb) {
      return p->tiles * (routed ? experts * ((mean + mean / 8 + nb - 1) / nb) : (rows + nb - 1) / nb);
    };
    int NB = routed ? (int)std::min<int64_t>(cap, (rows + 15) / 16 * 16) : like(b);
    double best = i8_tile(M, rows, nmat, E, NB, count(NB), p);
    if (count(NB) > slots) {
      // Two matrices: one set of accumulators in place of two holds tiles of up to 256 rows.  With nothing to
      // overlap a read-out this costs more per round (64 experts of 128 rows, 1024 x 1024: 44.5 us in tiles of 128,
      // 49.6 of 160), but pays where it makes one round of two (8 of 256 18.5 in tiles of 128, 15.9 of 144).
      for (int nb = cap + 16; nmat == 2 && nb <= 256; nb += 16)
        if (count(nb) <= slots) {
          i8_tile(M, rows, nmat, E, nb, count(nb), p);
          p->cs = 1;
          return true;
        }
      return false;
    }
    for (int nb = like(b); !pair && NB > 32 && nb >= 32 && count(nb) <= slots;
         nb = like((rows + nb - std::max(16, nb / 4) - 1) / (nb - std::max(16, nb / 4)))) {
      const double t = i8_tile(M, rows, nmat, E, nb, count(nb), p);
      if (t < best) best = t, NB = nb;
      if (nb == 32) break;
    }
    i8_tile(M, rows, nmat, E, NB, count(NB), p);
    return true;
  };
  // Wide calls run on pairs, but where lone CTAs hold all tiles at once (700 by 300 x 2960 13.8 us on pairs, 11.3
  // on lone CTAs; 2048 by 128 x 2048 12.6, 11.8; 700 by 6000 x 5120 23.5, 22.0; 1000 by 4700 x 5120, 76 tiles for
  // 74 pairs, 43, 28.7); of tiles as large as theirs pairs still read less (500 by 9400 x 8192 32.6, 35.7).
  const bool lone = tile(false);
  if (!routed && rows > kI8PairRows) {
    const bool large = p->NB > 192;
    if (!lone || large) {
      if (!tile(true) && lone) tile(false);
    }
  }
  // routed: boxes of about the mean expert's rows, so that its rows bring few of its neighbours' with them; but a
  // box has a cost of its own.  8 experts of 1800 rows, 4096 x 5120 down: boxes of 32, 64, 128, 256 rows 391, 297,
  // 260, 259 us; 8 of 256 rows, 1024 x 1024: 12.5, 11.3, 10.9 (32, 64, 128); 512 of 40 rows, 2048 x 512: 116.8,
  // 117.6, 123.5
  const int most = mean >= 128 ? 128 : mean >= 64 ? 64 : 32, boxes = routed ? (p->NB + most - 1) / most : 1;
  p->box = p->pair ? p->NB / 2 : (p->NB + boxes * 16 - 1) / (boxes * 16) * 16;
  p->w_again = p->b_tiles > 1;
  // Small plain calls quantise x in the product's own kernel, each CTA for itself: one launch in place of two,
  // and no workspace.  As long as a warp has one row, or two short ones: 512 x 1024 takes 6.1 us where two
  // kernels take 7.1 (1 row) and 7.3 where they take 6.9 (16 rows, but 8.4 against 13 us of host time);
  // 16 rows of 2048 take 9.3 against 8.0, so they keep two kernels.
  const int64_t x_bytes = (p->chunks + p->cs - 1) / p->cs * (int64_t)p->NB * 128;
  const bool few = rows <= kI8FusedRows / 2 || (rows <= kI8FusedRows && K <= kI8FusedK / 2);
  p->fused = !routed && p->S == 1 && p->runs == 0 && K <= kI8FusedK && few;
  p->x_bytes = p->fused ? (int)x_bytes : 0;
  p->stage_bytes = nmat * kWCodeBytes + (p->fused ? 0 : (p->NB + p->box - 1) / p->box * p->box * 128);
  int cols = 32;
  p->one_set = 2 * nmat * p->NB > 512;
  while (cols < (p->one_set ? 1 : 2) * nmat * p->NB) cols <<= 1;
  p->tmem_cols = cols;
}

size_t i8_partial_bytes(const I8Params& p) {
  return (size_t)(p.units - p.full) * (size_t)p.NB * (p.pair ? 2 : 1) * kTileRows * 4;
}

// Partials of at most M rows.  A split takes more than kI8SplitChunks chunks off a tile's time (runs, which cost 6.5 us,
// more than 11), its units fit on the SMs at once, with 256 rows of 128 channels each or M in whole sixteens (a
// pair's unit counts as two); runs have two for each SM, where the tiles are no more than the SMs.
size_t i8_partial_bound(int64_t M, int64_t N, int64_t K) {
  if (k_chunks(FMT_FP8, K) <= kI8SplitChunks + 1) return 0;
  const size_t units = row_tiles(N) <= kI8SMs ? 2 * kI8SMs : kI8SMs;
  return units * (size_t)std::min<int64_t>(256, (M + 15) / 16 * 16) * kTileRows * 4;
}

// Raises a kernel's dynamic shared-memory limit once per device (devices beyond 64: every time).
static cudaError_t raise_smem(const void* kern, std::atomic<uint64_t>& set_mask, int dev) {
  const uint64_t bit = (dev >= 0 && dev < 64) ? (1ull << dev) : 0ull;
  if (bit != 0 && (set_mask.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit - 64);
  if (e == cudaSuccess) set_mask.fetch_or(bit, std::memory_order_release);
  return e;
}

template <typename... P, typename... A>
static cudaError_t launch_gemm(void (*kern)(P...), size_t smem, int grid, int cluster, cudaStream_t stream,
                               const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3(kI8Threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;  // (the pair kernel has its cluster size from its declaration)
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int NMAT, int MODE, bool CL>
static cudaError_t launch_i8_kernel(I8Params& p, const CUtensorMap& map, int dev, cudaStream_t stream) {
  static std::atomic<uint64_t> set_mask{0};
  const auto kern = qgemm_i8_kernel<NMAT, MODE, CL>;
  const cudaError_t e = raise_smem((const void*)kern, set_mask, dev);
  if (e != cudaSuccess) return e;
  const size_t own = MODE == kI8Routed  ? kI8List * sizeof(I8Unit<NMAT>) + 4 * (size_t)p.E
                     : MODE == kI8Fused ? 4 * (size_t)kI8FusedRows + (size_t)p.x_bytes
                                        : 0;
  const size_t misc = 1024 + 8 * (2 * kI8MaxStages + 6) + 16 + own;
  // (a ring of half the shared memory, which lets the next product's CTAs in beside these, measured 3 to
  // 15 % slower: with memory busy, a chunk takes microseconds to arrive)
  p.stages = (int)std::min<size_t>(kI8MaxStages, (kSmemLimit - 64 - misc) / (size_t)p.stage_bytes);
  if (p.stages < 2) return cudaErrorInvalidValue;
  // routed: an upper bound, the kernel counts the units that have rows
  const int64_t most = MODE == kI8Routed ? (int64_t)p.tiles * p.b_tiles * std::min(p.E, p.M)
                       : MODE == kI8Runs ? p.runs
                                         : p.units;
  const int grid = CL               ? (int)most * p.cs
                   : MODE == kI8Runs ? p.runs
                                     : (int)std::min<int64_t>(most, sm_count(dev));
  return launch_gemm(kern, misc + (size_t)p.stages * p.stage_bytes, grid, p.cs, stream, p, map);
}

template <int NMAT, int MODE>
static cudaError_t launch_i8_impl(I8Params& p, const CUtensorMap& map, int dev, cudaStream_t stream) {
  return p.cs > 1 ? launch_i8_kernel<NMAT, MODE, true>(p, map, dev, stream)
                  : launch_i8_kernel<NMAT, MODE, false>(p, map, dev, stream);
}

// p: planned (i8_plan), operands filled in; map_x: x's codes in boxes of 128 x p.box; map_w (pair):
// the packed codes in boxes of 128 x 128.
cudaError_t launch_i8_gemm(I8Params p, const CUtensorMap& map_x, const CUtensorMap& map_w, cudaStream_t stream) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (p.pair) {
    static std::atomic<uint64_t> set_mask{0};
    e = raise_smem((const void*)qgemm_i8_pair_kernel, set_mask, dev);
    if (e != cudaSuccess) return e;
    const size_t smem = 1024 + kI8PairStages * kI8PairStage + 8 * (2 * kI8PairStages + 6) + 16;
    const int grid = 2 * std::min(p.units, sm_count(dev) / 2);
    e = launch_gemm(qgemm_i8_pair_kernel, smem, grid, 1, stream, p, map_x, map_w);
  } else {
    e = p.nmat == 2 ? launch_i8_impl<2, kI8Routed>(p, map_x, dev, stream)
        : p.off     ? launch_i8_impl<1, kI8Routed>(p, map_x, dev, stream)
        : p.fused   ? launch_i8_impl<1, kI8Fused>(p, map_x, dev, stream)
        : p.runs    ? launch_i8_kernel<1, kI8Runs, false>(p, map_x, dev, stream)
                    : launch_i8_impl<1, kI8Plain>(p, map_x, dev, stream);
  }
  if (e != cudaSuccess || (p.S == 1 && !p.runs)) return e;
  const int split = p.runs ? p.tiles * p.b_tiles : (p.units - p.full) / p.S;  // tiles with partials
  return launch_dep(qgemm_i8_reduce_kernel,
                    dim3((unsigned)split, (unsigned)((p.NB + kI8ReduceRows - 1) / kI8ReduceRows)),
                    dim3(256), 0, stream, p);
}

}  // namespace qg
