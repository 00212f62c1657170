// rs_quant.cu -- a matrix to 8-bit blocks (rs_fp8.cuh) along its rows, along its columns
// (written transposed, for a product that reduces over the rows), or both from one read,
// with its column sums (a bias gradient) on the way.
//
// Bound by memory: per value e bytes read (e = 2 or 4) and 1 written per direction. A block
// of 256 threads takes tiles of 128 x 128; a thread holds 8 rows x 8 columns in registers, so
// a block of 128 values is 16 neighbouring lanes (rows: four shuffles) or 16 threads of one
// column group (columns: shared memory), and nothing is read twice. The transposed bytes turn
// in shared memory, 8 rows of a column at a time, at 8-byte places XORed with the column group
// so that neither the writes nor the 16-byte reads meet in a bank.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "rs_fp8.cuh"
#include "rs_internal.h"
#include "rs_ptx.cuh"

namespace rs {

constexpr int kQTile = 128;

template <typename T>
__device__ __forceinline__ float elem_to_float(T v) { return static_cast<float>(v); }

// 8 neighbouring columns of a row, zero past K.
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* row, int c, int K, float (&f)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = 0.f;
  if constexpr (VEC) {
    if (c < K) {  // K is a multiple of 8
      if constexpr (Elem<T>::E == 8) {
        Elem<T>::unpack(*reinterpret_cast<const uint4*>(row + c), f);
      } else {
        float a[4], b[4];
        Elem<T>::unpack(*reinterpret_cast<const uint4*>(row + c), a);
        Elem<T>::unpack(*reinterpret_cast<const uint4*>(row + c + 4), b);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          f[e] = a[e];
          f[4 + e] = b[e];
        }
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < K) f[e] = static_cast<float>(row[c + e]);
  }
}

template <typename T, bool VEC, bool ROWS, bool COLS>
__global__ void __launch_bounds__(256, sizeof(T) == 4 ? 2 : 3) quantize_kernel(const Quant p) {
  __shared__ __align__(16) uint8_t s_t[COLS ? kQTile * kQTile : 16];
  __shared__ uint32_t s_max[COLS ? 8 : 1][kQTile];
  __shared__ float s_sum[8][COLS ? kQTile : 1];
  pdl_trigger();
  pdl_wait();
  const int t = threadIdx.x, warp = t >> 5;
  const int tx = t & 15, ty = t >> 4;  // columns 8 tx .., rows 8 ty ..
  const int c0 = static_cast<int>(blockIdx.x) * kQTile, c = c0 + 8 * tx;
  const int row_tiles = (p.rows + kQTile - 1) / kQTile;
  const int kq = (p.K + 511) / 512, kqt = (p.rows + 511) / 512;
  const T* x = static_cast<const T*>(p.x);
  float sum[8] = {};
  for (int rt = blockIdx.y; rt < row_tiles; rt += gridDim.y) {
    const int r0 = rt * kQTile + 8 * ty;
    float f[8][8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (r0 + j < p.rows) {
        load8<T, VEC>(x + static_cast<int64_t>(r0 + j) * p.ldx, c, p.K, f[j]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[j][e] = 0.f;
      }
    }
    uint32_t bad = 0;  // any infinity or NaN of this thread
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        bad |= abs_bits(f[j][e]) >= kInfBits ? 1u : 0u;
        if constexpr (COLS) sum[e] += f[j][e];
      }
    if constexpr (ROWS) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t a = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          a = max(a, bad ? finite_abs_bits(f[j][e]) : abs_bits(f[j][e]));
#pragma unroll
        for (int o = 8; o; o >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
        const uint32_t byte = e8m0_byte(a);
        const float inv = e8m0_inverse(byte);
        const int r = r0 + j;
        if (r < p.rows && c < p.K) {
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = (bad ? inf_to_nan(f[j][e]) : f[j][e]) * inv;
          uint2 o;
          o.x = e4m3x4(v[0], v[1], v[2], v[3]);
          o.y = e4m3x4(v[4], v[5], v[6], v[7]);
          *reinterpret_cast<uint2*>(p.q + static_cast<int64_t>(r) * p.ldq + c) = o;
          if (tx == 0) p.scales[scale_offset(r, c0 >> 7, kq)] = static_cast<uint8_t>(byte);
        }
      }
    }
    if constexpr (COLS) {
      uint32_t a[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        a[e] = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          a[e] = max(a[e], bad ? finite_abs_bits(f[j][e]) : abs_bits(f[j][e]));
        a[e] = max(a[e], __shfl_xor_sync(0xffffffffu, a[e], 16));
      }
      if ((t & 16) == 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) s_max[warp][8 * tx + e] = a[e];
      }
      __syncthreads();
      if (t < kQTile) {
        uint32_t m = s_max[0][t];
#pragma unroll
        for (int w = 1; w < 8; ++w) m = max(m, s_max[w][t]);
        const uint32_t byte = e8m0_byte(m);
        s_max[0][t] = byte;  // only this thread reads or writes column t here
        if (c0 + t < p.K) p.scales_t[scale_offset(c0 + t, rt, kqt)] = static_cast<uint8_t>(byte);
      }
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float inv = e8m0_inverse(s_max[0][8 * tx + e]);
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = (bad ? inf_to_nan(f[j][e]) : f[j][e]) * inv;
        uint2 o;
        o.x = e4m3x4(v[0], v[1], v[2], v[3]);
        o.y = e4m3x4(v[4], v[5], v[6], v[7]);
        *reinterpret_cast<uint2*>(s_t + (8 * tx + e) * kQTile + ((ty ^ tx) << 3)) = o;
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int col = i * 32 + (t >> 3), ch = t & 7;  // 16 rows 16 ch .. of column col
        const int g = (2 * ch) ^ (col >> 3);
        const uint4 v = *reinterpret_cast<const uint4*>(s_t + col * kQTile + ((g >> 1) << 4));
        const uint4 o = (g & 1) ? make_uint4(v.z, v.w, v.x, v.y) : v;
        const int r = rt * kQTile + 16 * ch;
        if (c0 + col < p.K && r < p.rows)
          *reinterpret_cast<uint4*>(p.qt + static_cast<int64_t>(c0 + col) * p.ldqt + r) = o;
      }
      // the next tile's s_max and s_t are written only after every thread passes its first
      // barrier, which no thread reaches before it has read s_t here; s_max[0] is rewritten
      // before that barrier, and was last read before the one above
    }
  }
  if constexpr (COLS) {
    if (p.partials != nullptr) {
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 16);
      if ((t & 16) == 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) s_sum[warp][8 * tx + e] = sum[e];
      }
      __syncthreads();
      if (t < kQTile && c0 + t < p.K) {
        float v = s_sum[0][t];
#pragma unroll
        for (int w = 1; w < 8; ++w) v += s_sum[w][t];
        p.partials[static_cast<int64_t>(blockIdx.y) * p.K + c0 + t] = v;
      }
    }
  }
}

template <typename T, bool VEC>
static cudaError_t pick(const Quant& p, cudaStream_t s, bool pdl) {
  const dim3 block(256);
  const int ct = (p.K + kQTile - 1) / kQTile;
  if (p.qt != nullptr) {
    const dim3 grid(ct, quant_chunks(p.rows));
    if (p.q != nullptr) return launch(quantize_kernel<T, VEC, true, true>, grid, block, 0, s, pdl, p);
    return launch(quantize_kernel<T, VEC, false, true>, grid, block, 0, s, pdl, p);
  }
  // rows only: nothing is carried from tile to tile, so each tile has a block of its own
  const int tiles = (p.rows + kQTile - 1) / kQTile;
  return launch(quantize_kernel<T, VEC, true, false>, dim3(ct, tiles < 65535 ? tiles : 65535), block,
                0, s, pdl, p);
}

cudaError_t launch_quantize(const Quant& p, int dtype, bool vec, cudaStream_t s, bool pdl) {
  if (dtype == RS_BF16) return vec ? pick<__nv_bfloat16, true>(p, s, pdl) : pick<__nv_bfloat16, false>(p, s, pdl);
  if (dtype == RS_FP16) return vec ? pick<__half, true>(p, s, pdl) : pick<__half, false>(p, s, pdl);
  return vec ? pick<float, true>(p, s, pdl) : pick<float, false>(p, s, pdl);
}

}  // namespace rs
