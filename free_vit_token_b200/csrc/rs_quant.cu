// rs_quant.cu -- a matrix to 8-bit blocks (rs_fp8.cuh) along its rows, along its columns
// (written transposed, for a product that reduces over the rows), or both from one read,
// with its column sums (a bias gradient) on the way.
//
// Bound by memory: per value e bytes read (e = 2 or 4) and 1 written per direction. A block
// of 256 threads takes tiles of 128 x 128; a thread holds 8 rows x 8 columns in registers, so
// a block of 128 values is 16 neighbouring lanes (rows: four shuffles) or 16 threads of one
// column group (columns: shared memory), and nothing is read twice. The transposed bytes turn
// in shared memory, 8 rows of a column at a time, at 8-byte places XORed with the column group
// so that neither the writes nor the 16-byte reads meet in a bank. Values stay 16-bit words until
// they are scaled, and the next tile's loads are under way: 128 registers, two blocks per SM.
// Measured 12288 x 4096 bf16: rows 25.8 us (5.9 TB/s), both ways with sums 40.5 us (5.0 TB/s;
// issue-bound: 47% of slots in a cold run, the transposition's shared-memory turns beside it).
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "rs_fp8.cuh"
#include "rs_ops.h"
#include "rs_ptx.cuh"

namespace rs {

constexpr int kQTile = 128;

// 8 neighbouring columns of a row as they lie in memory (16-bit types: 4 words of two, fp32:
// 8 words) and what the kernel asks of them. Magnitudes order like their bits without the
// sign, infinity above every finite value and NaN above infinity.
template <typename T>
struct Cols8 {  // bf16, fp16
  static constexpr int W = 4;
  static constexpr uint32_t kInf = sizeof(T) == 2 && Elem<T>::kBf16 ? 0x7F80u : 0x7C00u;
  uint32_t w[W];
  static __device__ __forceinline__ uint32_t vmax(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }
  __device__ __forceinline__ uint32_t mag(int i) const { return w[i] & 0x7FFF7FFFu; }
  static __device__ __forceinline__ bool nonfinite(uint32_t m) {
    return (m & 0xFFFFu) >= kInf || (m >> 16) >= kInf;
  }
  static __device__ __forceinline__ uint32_t finite_part(uint32_t m) {
    return ((m & 0xFFFFu) >= kInf ? 0u : m & 0xFFFFu) | ((m >> 16) >= kInf ? 0u : m & 0xFFFF0000u);
  }
  __device__ __forceinline__ void inf_to_nan_all() {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if ((w[i] & 0x7FFFu) == kInf) w[i] |= 0x7FFFu;
      if (((w[i] >> 16) & 0x7FFFu) == kInf) w[i] |= 0x7FFF0000u;
    }
  }
  // a 16-bit magnitude as fp32 bits; the one of a word's column e
  static __device__ __forceinline__ uint32_t wide(uint32_t h) {
    if constexpr (Elem<T>::kBf16) return h << 16;
    return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(h))));
  }
  static __device__ __forceinline__ uint32_t col(uint32_t m, int e) { return wide(e ? m >> 16 : m & 0xFFFFu); }
  __device__ __forceinline__ void pairs(uint64_t (&f)[4]) const {
    Elem<T>::pairs(make_uint4(w[0], w[1], w[2], w[3]), f);
  }
  // the larger magnitudes of two rows, reduced over the 16 threads of a block: fp32 bits
  static __device__ __forceinline__ void rows_top(uint32_t m0, uint32_t m1, uint32_t& t0, uint32_t& t1) {
    uint32_t m = __vmaxu2(__byte_perm(m0, m1, 0x5410), __byte_perm(m0, m1, 0x7632));
#pragma unroll
    for (int o = 8; o; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    t0 = wide(m & 0xFFFFu);
    t1 = wide(m >> 16);
  }
};
template <>
struct Cols8<float> {
  static constexpr int W = 8;
  uint32_t w[W];
  static __device__ __forceinline__ uint32_t vmax(uint32_t a, uint32_t b) { return max(a, b); }
  __device__ __forceinline__ uint32_t mag(int i) const { return w[i] & 0x7FFFFFFFu; }
  static __device__ __forceinline__ bool nonfinite(uint32_t m) { return m >= kInfBits; }
  static __device__ __forceinline__ uint32_t finite_part(uint32_t m) { return m >= kInfBits ? 0u : m; }
  __device__ __forceinline__ void inf_to_nan_all() {
#pragma unroll
    for (int i = 0; i < W; ++i)
      if ((w[i] & 0x7FFFFFFFu) == kInfBits) w[i] = 0x7FFFFFFFu;
  }
  static __device__ __forceinline__ uint32_t col(uint32_t m, int) { return m; }
  __device__ __forceinline__ void pairs(uint64_t (&f)[4]) const {
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = (static_cast<uint64_t>(w[2 * e + 1]) << 32) | w[2 * e];
  }
  static __device__ __forceinline__ void rows_top(uint32_t m0, uint32_t m1, uint32_t& t0, uint32_t& t1) {
    t0 = m0;
    t1 = m1;
#pragma unroll
    for (int o = 8; o; o >>= 1) {
      t0 = max(t0, __shfl_xor_sync(0xffffffffu, t0, o));
      t1 = max(t1, __shfl_xor_sync(0xffffffffu, t1, o));
    }
  }
};

// Zero past K (and for rows that do not exist).
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* row, int c, int K, bool live, Cols8<T>& v) {
#pragma unroll
  for (int i = 0; i < Cols8<T>::W; ++i) v.w[i] = 0;
  if constexpr (VEC) {
    if (live && c < K) {  // K is a multiple of 8
#pragma unroll
      for (int i = 0; i < Cols8<T>::W; i += 4) {
        const uint4 u = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint32_t*>(row + c) + i);
        v.w[i] = u.x;
        v.w[i + 1] = u.y;
        v.w[i + 2] = u.z;
        v.w[i + 3] = u.w;
      }
    }
  } else if (live) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (c + e < K) {
        if constexpr (sizeof(T) == 2)
          v.w[e >> 1] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(row)[c + e]) << (16 * (e & 1));
        else
          v.w[e] = reinterpret_cast<const uint32_t*>(row)[c + e];
      }
    }
  }
}

template <typename T, bool VEC, bool ROWS, bool COLS>
__global__ void __launch_bounds__(256, sizeof(T) == 4 ? 1 : 2) quantize_kernel(const Quant p) {
  using V = Cols8<T>;
  constexpr int CW = 8 / V::W;  // columns of a word
  __shared__ __align__(16) uint8_t s_t[COLS ? kQTile * kQTile : 16];
  __shared__ uint32_t s_max[COLS ? 8 : 1][COLS ? kQTile / CW : 1];
  __shared__ __align__(8) float s_inv[COLS ? kQTile : 1];
  __shared__ float s_sum[COLS ? 8 : 1][COLS ? kQTile : 1];
  pdl_trigger();
  pdl_wait();
  const int t = threadIdx.x, warp = t >> 5;
  const int tx = t & 15, ty = t >> 4;  // columns 8 tx .., rows 8 ty ..
  const int c0 = static_cast<int>(blockIdx.x) * kQTile, c = c0 + 8 * tx;
  const int row_tiles = (p.rows + kQTile - 1) / kQTile;
  const int kq = (p.K + 511) / 512, kqt = (p.rows + 511) / 512;
  const T* x = static_cast<const T*>(p.x);
  uint64_t sum[4] = {};  // pairs of column sums
  V v[8], nx[8];
  auto load = [&](int rt, V (&d)[8]) {
    const int r0 = rt * kQTile + 8 * ty;
    const T* row = x + static_cast<int64_t>(r0) * p.ldx;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      load8<T, VEC>(row, c, p.K, r0 + j < p.rows, d[j]);
      row += p.ldx;
    }
  };
  int rt = blockIdx.y;
  if (rt < row_tiles) load(rt, v);
  for (; rt < row_tiles; rt += gridDim.y) {
    if (rt + static_cast<int>(gridDim.y) < row_tiles) load(rt + gridDim.y, nx);
    const int r0 = rt * kQTile + 8 * ty;
    // the largest magnitude of each row (rm) and column (cm) of this thread's 8 x 8
    uint32_t rm[8], cm[V::W], all = 0;
#pragma unroll
    for (int i = 0; i < V::W; ++i) cm[i] = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      rm[j] = 0;
#pragma unroll
      for (int i = 0; i < V::W; ++i) {
        const uint32_t m = v[j].mag(i);
        rm[j] = V::vmax(rm[j], m);
        if constexpr (COLS) cm[i] = V::vmax(cm[i], m);
      }
      all = V::vmax(all, rm[j]);
    }
    if constexpr (COLS) {
      if (p.partials != nullptr) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint64_t f[4];
          v[j].pairs(f);
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[e] = fadd2(sum[e], f[e]);
        }
      }
    }
    if (V::nonfinite(all)) {  // rare: infinities become NaN, and neither counts
#pragma unroll
      for (int i = 0; i < V::W; ++i) cm[i] = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j].inf_to_nan_all();
        rm[j] = 0;
#pragma unroll
        for (int i = 0; i < V::W; ++i) {
          const uint32_t m = V::finite_part(v[j].mag(i));
          rm[j] = V::vmax(rm[j], m);
          cm[i] = V::vmax(cm[i], m);
        }
      }
    }
    if constexpr (COLS) {
#pragma unroll
      for (int i = 0; i < V::W; ++i) cm[i] = V::vmax(cm[i], __shfl_xor_sync(0xffffffffu, cm[i], 16));
      if ((t & 16) == 0) {
#pragma unroll
        for (int i = 0; i < V::W; ++i) s_max[warp][V::W * tx + i] = cm[i];
      }
      __syncthreads();
      if (t < kQTile) {
        uint32_t m = s_max[0][t / CW];
#pragma unroll
        for (int w = 1; w < 8; ++w) m = V::vmax(m, s_max[w][t / CW]);
        const uint32_t byte = e8m0_byte(V::col(m, t % CW));
        s_inv[t] = e8m0_inverse(byte);
        if (c0 + t < p.K) p.scales_t[scale_offset(c0 + t, rt, kqt)] = static_cast<uint8_t>(byte);
      }
    }
    uint32_t byte[8];
    if constexpr (ROWS) {
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        uint32_t a, b;
        V::rows_top(rm[j], rm[j + 1], a, b);
        byte[j] = e8m0_byte(a);
        byte[j + 1] = e8m0_byte(b);
      }
      if (tx == 0) {  // 8 rows of one group of 32: their bytes are 16 apart
        uint8_t* sc = p.scales + scale_offset(r0, c0 >> 7, kq);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (r0 + j < p.rows) sc[16 * j] = static_cast<uint8_t>(byte[j]);
      }
    }
    uint64_t inv[4] = {};  // pairs of column factors
    if constexpr (COLS) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 4; ++e)
        inv[e] = *reinterpret_cast<const uint64_t*>(s_inv + 8 * tx + 2 * e);
    }
    uint8_t* q = p.q + static_cast<int64_t>(r0) * p.ldq + c;
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // four rows at a time
      uint64_t f[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 * h + j].pairs(f[j]);
      if constexpr (ROWS) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float ri = e8m0_inverse(byte[4 * h + j]);
          const uint64_t r2 = f2pack(ri, ri);
          float2 g[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) g[e] = f2unpack(mul2(f[j][e], r2));
          if (r0 + 4 * h + j < p.rows && c < p.K)
            *reinterpret_cast<uint2*>(q) = make_uint2(e4m3x4(g[0].x, g[0].y, g[1].x, g[1].y),
                                                      e4m3x4(g[2].x, g[2].y, g[3].x, g[3].y));
          q += p.ldq;
        }
      }
      if constexpr (COLS) {
        uint8_t* d = s_t + 8 * tx * kQTile + ((ty ^ tx) << 3) + 4 * h;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float2 g[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) g[j] = f2unpack(mul2(f[j][e], inv[e]));
          *reinterpret_cast<uint32_t*>(d + 2 * e * kQTile) = e4m3x4(g[0].x, g[1].x, g[2].x, g[3].x);
          *reinterpret_cast<uint32_t*>(d + (2 * e + 1) * kQTile) = e4m3x4(g[0].y, g[1].y, g[2].y, g[3].y);
        }
      }
    }
    if constexpr (COLS) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int col = i * 32 + (t >> 3), ch = t & 7;  // rows 16 ch .. of column col
        const int g = (2 * ch) ^ (col >> 3);
        const uint4 u = *reinterpret_cast<const uint4*>(s_t + col * kQTile + ((g >> 1) << 4));
        const uint4 o = (g & 1) ? make_uint4(u.z, u.w, u.x, u.y) : u;
        const int r = rt * kQTile + 16 * ch;
        if (c0 + col < p.K && r < p.rows)
          *reinterpret_cast<uint4*>(p.qt + static_cast<int64_t>(c0 + col) * p.ldqt + r) = o;
      }
      // Three barriers a tile order the shared arrays: s_max is written before the first and
      // read before the second, s_inv written before the second and read before the third,
      // s_t written before the third and read before the next tile's first.
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = nx[j];
  }
  if constexpr (COLS) {
    if (p.partials != nullptr) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float2 a = f2unpack(sum[e]);
        a.x += __shfl_xor_sync(0xffffffffu, a.x, 16);
        a.y += __shfl_xor_sync(0xffffffffu, a.y, 16);
        if ((t & 16) == 0) {
          s_sum[warp][8 * tx + 2 * e] = a.x;
          s_sum[warp][8 * tx + 2 * e + 1] = a.y;
        }
      }
      __syncthreads();
      if (t < kQTile && c0 + t < p.K) {
        float a = s_sum[0][t];
#pragma unroll
        for (int w = 1; w < 8; ++w) a += s_sum[w][t];
        p.partials[static_cast<int64_t>(blockIdx.y) * p.K + c0 + t] = a;
      }
    }
  }
}

template <typename T, bool VEC>
static cudaError_t pick(const Quant& p, cudaStream_t s, bool pdl) {
  const dim3 block(256);
  const dim3 grid((p.K + kQTile - 1) / kQTile, p.chunks);
  if (p.qt == nullptr) return launch(quantize_kernel<T, VEC, true, false>, grid, block, 0, s, pdl, p);
  if (p.q == nullptr) return launch(quantize_kernel<T, VEC, false, true>, grid, block, 0, s, pdl, p);
  return launch(quantize_kernel<T, VEC, true, true>, grid, block, 0, s, pdl, p);
}

cudaError_t launch_quantize(const Quant& p, int dtype, bool vec, cudaStream_t s, bool pdl) {
  if (dtype == RS_BF16) return vec ? pick<__nv_bfloat16, true>(p, s, pdl) : pick<__nv_bfloat16, false>(p, s, pdl);
  if (dtype == RS_FP16) return vec ? pick<__half, true>(p, s, pdl) : pick<__half, false>(p, s, pdl);
  return vec ? pick<float, true>(p, s, pdl) : pick<float, false>(p, s, pdl);
}

}  // namespace rs
