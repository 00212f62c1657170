// rs_ops.h -- declarations of the layer norm and 8-bit operators' translation units (kernel
// parameter blocks and host-side launchers). Not part of the C ABI.
#pragma once

#include <atomic>

#include "rs_internal.h"

namespace rs {

// The current device's SM count (cached; allocates nothing) and status flag (allocated on a
// device's first use): RS_OK or an error. Defined beside the library's device state.
int device_sms(int* num_sms);
int device_flag(int* num_sms, int** err);
// Allows `kern` `bytes` of dynamic shared memory on the current device, once per device (`done`
// is the kernel's own, one bit per device) instead of once per launch.
template <typename... A>
inline cudaError_t allow_smem(void (*kern)(A...), int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// Layer norm forward (rs_norm.cu): y (or q and scales, by launcher) and optional row stats.
struct LnForward {
  const void* x;
  int64_t ldx;         // elements between rows
  int M, C;
  const void* gamma;   // [C] or null (ones)
  const void* beta;    // [C] or null (zeros)
  bool p32;            // gamma and beta are fp32 (else x's type)
  float eps;
  void* y;
  int64_t ldy;
  float2* stats;       // [M] (mean, rstd) or null
  uint8_t* q;          // quantised output: e4m3 rows, ldq bytes apart
  int64_t ldq;
  uint8_t* scales;     // scale tiles (rs_fp8.cuh)
  int kq;              // scale tiles along C
};
struct LnBackward {
  const void* dy;
  int64_t lddy;
  const void* x;
  int64_t ldx;
  const void* dres;    // added to dx, or null
  int64_t lddres;
  const float2* stats;
  const void* gamma;
  bool p32;
  int M, C;
  void* dx;            // or null
  int64_t lddx;
  float* dgamma;       // [C] or null
  float* dbeta;        // [C] or null
  bool sums;           // either of them wanted
  float* partials;     // [blocks][2][C] scratch, unused for a few rows
  int cluster;         // set by the launcher: blocks of the one cluster, 0 = a grid
};
// `vec`: every row of every tensor starts on 16 bytes and is a whole number of 16-byte vectors.
cudaError_t launch_ln_forward(const LnForward& p, int dtype, bool vec, int num_sms,
                              cudaStream_t s);
cudaError_t launch_ln_quantize(const LnForward& p, int dtype, int num_sms, cudaStream_t s);
// Backward, then (past a few rows) the sum of the blocks' partials, at most num_sms of them.
cudaError_t launch_ln_backward(const LnBackward& p, int dtype, bool vec, int num_sms,
                               cudaStream_t s);
bool ln_backward_few(int M, int C);  // no scratch for these sizes, whatever the type
// out[c] = sum_p partials[p][c], in 16 chains (p = i, i + 16, ..) whose sums are added in order,
// for n columns: the first `split` of them to out0, the others to out1 (either may be null).
cudaError_t launch_col_reduce(const float* partials, int P, int n, int split, float* out0,
                              float* out1, cudaStream_t stream, bool pdl);

// Quantisation (rs_quant.cu): rows in blocks along K, and/or the transposed tensor in blocks
// along the rows, and/or the column sums' partials.
struct Quant {
  const void* x;
  int64_t ldx;
  int rows, K;
  uint8_t* q;          // [rows][ldq] or null
  int64_t ldq;
  uint8_t* scales;
  uint8_t* qt;         // [K][ldqt] or null
  int64_t ldqt;
  uint8_t* scales_t;
  float* partials;     // [chunks][K] column sums, or null
  int chunks;          // blocks that share out the rows (quant_chunks, or 1)
};
// Blocks that share out the row tiles of 128 of one column tile. 296 blocks are resident (two on
// each of 148 SMs); of one to four such waves, the number that leaves the longest chain of tiles
// shortest, a wave's start (its first loads cover nothing) counted as half a tile: 12288 x 4096
// 608 blocks 46.8 us, 288 blocks 40.5.
inline int quant_chunks(int rows, int K) {
  const int tiles = (rows + 127) / 128, cols = (K + 127) / 128;
  int best = 1;
  int64_t cost = INT64_MAX;
  for (int waves = 1; waves <= 4; ++waves) {
    const int most = 296 * waves / cols;
    if (most < 1) continue;
    const int per = (tiles + most - 1) / most, chunks = (tiles + per - 1) / per;
    const int64_t real = (static_cast<int64_t>(chunks) * cols + 295) / 296;
    if (real * (2 * per + 1) < cost) {
      cost = real * (2 * per + 1);
      best = chunks;
    }
  }
  return best;
}
// With column sums, up to this many row tiles go through one block per column tile, which then
// writes the sums themselves: a launch less (2.3 us of host time) for up to three more tiles in
// a block (4 us on the device).
constexpr int kQuantDirectTiles = 4;
inline bool quant_direct(int rows) { return rows <= 128 * kQuantDirectTiles; }
cudaError_t launch_quantize(const Quant& p, int dtype, bool vec, cudaStream_t s, bool pdl = false);

// The product of two quantised operands (rs_fp8_gemm.cu): out = act(A B^T + bias) + resid.
constexpr int kOutBf16 = 0;
constexpr int kOutFp32 = 1;
constexpr int kOutQ8 = 2;
struct Fp8Gemm {
  const void* a;         // [M][lda] e4m3
  int64_t lda;
  const void* sa;        // scale tiles of a
  const void* b;         // [N][ldb] e4m3
  int64_t ldb;
  const void* sb;
  int M, N, K;
  const __nv_bfloat16* bias;  // [N] or null
  int gelu;              // 1: exact GELU after the bias
  const void* resid;     // [M][ldr] of the output's type, or null (not with kOutQ8)
  int64_t ldr;
  int rvec;              // resid's rows start on 16 bytes
  void* out;             // [M][ldo] bf16, fp32 or e4m3
  int64_t ldo;
  int direct;            // out's rows do not start on 16 bytes: plain stores, not TMA
  uint8_t* out_scales;   // kOutQ8: scale tiles of out
  int kqo;               // kOutQ8: scale tiles along N
  int* err;
  unsigned long long timeout_ns;
  int debug_skip_kb;     // test hook: CTA 0 skips this K block's loads of its first tile (-1: off)
  int n_blocks, num_tiles;  // set by the launcher
};
// RS_OK or an error status.
int launch_fp8_gemm(const Fp8Gemm& p, int out, int num_sms, cudaStream_t s, bool pdl = false);

// Tensor maps of a quantised operand [rows][ld] (128-byte swizzled boxes of 128 K x box_rows)
// and of its scale tiles as [row tiles][tiles along K][128 words] in boxes of `tiles` row tiles.
int tmap_operand(CUtensorMap* m, const void* base, int K, int rows, int64_t ld, int box_rows);
int tmap_scales(CUtensorMap* m, const void* base, int rows, int K, uint32_t tiles);

// A linear layer on a few rows (rs_fp8_few.cu): quantisation and product in one launch.
struct Fp8Few {
  const __nv_bfloat16* x;     // [M][ldx]
  int64_t ldx;
  int xvec;                   // x's rows start on 16 bytes
  int M, N, K;
  const void* w;              // [N][ldw] e4m3
  int64_t ldw;
  const void* sw;
  const __nv_bfloat16* bias;  // [N] or null
  int gelu;
  const __nv_bfloat16* resid; // [M][ldr] or null
  int64_t ldr;
  __nv_bfloat16* out;         // [M][ldo]
  int64_t ldo;
  int* err;
  unsigned long long timeout_ns;
  bool debug_skip;            // test hook: CTA 0 leaves its first weight tile unloaded
  int split, blocks;          // set by the launcher: CTAs per reduction, K blocks of each
};
bool fp8_few_rows(int M, int N, int K);  // does rs_fp8_linear take this path?
int launch_fp8_few(Fp8Few p, int num_sms, cudaStream_t s);

}  // namespace rs
