// rs_norm.cu -- the layer norm written out, and its gradients.
//
//   forward:  mean = sum x / C, var = sum (x - mean)^2 / C, rstd = 1/sqrt(var + eps),
//             xh = (x - mean) rstd, y = xh gamma + beta. The variance is a second pass over
//             the row held in registers, not E[x^2] - mean^2, which cancels when the mean
//             is far from zero.
//   quantise: the same y as 8-bit blocks (rs_fp8.cuh), for a product that reads LN(x).
//   backward: w = dy gamma, dx = rstd (w - mean(w) - xh mean(w xh)) + dres,
//             dgamma = sum_rows dy xh, dbeta = sum_rows dy.
//
// All three are bound by memory. TPR threads own a row and hold it in registers (VPL 16-byte
// vectors each), the next row's loads are issued before the current row is reduced, and every
// value is read once. Backward: a thread keeps its columns' dgamma and dbeta sums in fp32
// registers over all the rows of its block, the blocks' sums go to the workspace once each
// and a second kernel adds them in a fixed order: no atomics, the same bits every run.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "rs_fp8.cuh"
#include "rs_internal.h"
#include "rs_ptx.cuh"

namespace rs {

// Where element e of vector i of thread l sits in a row. VEC: 16-byte vectors, vector
// l + TPR i. Otherwise (a width, stride or address that is no multiple of 16 bytes)
// neighbouring threads take neighbouring elements, so that narrow accesses still coalesce.
template <typename T, int TPR, bool VEC>
__device__ __forceinline__ int col_of(int l, int i, int e) {
  constexpr int E = Elem<T>::E;
  return VEC ? (l + TPR * i) * E + e : l + TPR * (i * E + e);
}

template <typename T, int TPR, int VPL, bool VEC>
__device__ __forceinline__ void load_row(const T* row, int C, int l, uint4 (&v)[VPL]) {
  constexpr int E = Elem<T>::E;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    v[i] = make_uint4(0, 0, 0, 0);
    if constexpr (VEC) {
      const int c = col_of<T, TPR, VEC>(l, i, 0);
      if (c < C) v[i] = *reinterpret_cast<const uint4*>(row + c);
    } else {
      uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int c = col_of<T, TPR, VEC>(l, i, e);
        if (c < C) {
          if constexpr (E == 8)
            w[e / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(row)[c])
                        << (16 * (e & 1));
          else
            w[e] = reinterpret_cast<const uint32_t*>(row)[c];
        }
      }
      v[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

template <typename T, int TPR, bool VEC>
__device__ __forceinline__ void store_vec(T* row, int C, int l, int i,
                                          const float (&f)[Elem<T>::E]) {
  constexpr int E = Elem<T>::E;
  const uint4 v = Elem<T>::pack(f);
  if constexpr (VEC) {
    const int c = col_of<T, TPR, VEC>(l, i, 0);
    if (c < C) *reinterpret_cast<uint4*>(row + c) = v;
  } else {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = col_of<T, TPR, VEC>(l, i, e);
      if (c < C) {
        if constexpr (E == 8)
          reinterpret_cast<uint16_t*>(row)[c] = static_cast<uint16_t>(w[e / 2] >> (16 * (e & 1)));
        else
          reinterpret_cast<uint32_t*>(row)[c] = w[e];
      }
    }
  }
}

// gamma or beta for vector i: T or fp32 in memory (p32), `def` where there is none.
template <typename T, int TPR, bool VEC>
__device__ __forceinline__ void load_param(const void* p, bool p32, float def, int C, int l, int i,
                                           float (&f)[Elem<T>::E]) {
  constexpr int E = Elem<T>::E;
#pragma unroll
  for (int e = 0; e < E; ++e) f[e] = def;
  if (p == nullptr) return;
  if constexpr (VEC) {
    const int c = col_of<T, TPR, VEC>(l, i, 0);
    if (c >= C) return;
    if (p32 || sizeof(T) == 4) {
#pragma unroll
      for (int e = 0; e < E; e += 4) {
        const float4 g = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + c + e));
        f[e] = g.x;
        f[e + 1] = g.y;
        f[e + 2] = g.z;
        f[e + 3] = g.w;
      }
    } else {
      Elem<T>::unpack(__ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p) + c)), f);
    }
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = col_of<T, TPR, VEC>(l, i, e);
      if (c < C)
        f[e] = p32 ? __ldg(static_cast<const float*>(p) + c)
                   : static_cast<float>(static_cast<const T*>(p)[c]);
    }
  }
}

// Sum of v over the TPR threads that share a row, given to all of them. Rows wider than a
// warp meet in shared memory at a barrier of their own; `par` alternates between two slots,
// so one barrier per sum is enough.
template <int TPR>
__device__ __forceinline__ float2 group_sum(float2 v, float2* red, int group, int& par) {
#pragma unroll
  for (int o = (TPR < 32 ? TPR : 32) / 2; o; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  if constexpr (TPR > 32) {
    constexpr int W = TPR / 32;
    float2* slot = red + (group * 2 + par) * W;
    const int w = (threadIdx.x % TPR) >> 5;
    if ((threadIdx.x & 31) == 0) slot[w] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(TPR) : "memory");
    v = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < W; ++i) {
      v.x += slot[i].x;
      v.y += slot[i].y;
    }
    par ^= 1;
  }
  return v;
}

__host__ __device__ constexpr int ln_threads(int tpr) { return tpr > 256 ? tpr : 256; }

// ---------------------------------------------------------------- forward
template <typename T, int TPR, int VPL, bool VEC, bool QUANT>
__global__ void __launch_bounds__(ln_threads(TPR))
    ln_fwd_kernel(const LnForward p) {
  constexpr int E = Elem<T>::E;
  constexpr int GROUPS = ln_threads(TPR) / TPR;
  static_assert(!QUANT || (VEC && E == 8 && TPR >= 16), "16 threads hold a block of 128");
  __shared__ float2 red[TPR > 32 ? GROUPS * 2 * (TPR / 32) : 1];
  pdl_trigger();
  pdl_wait();
  const int group = threadIdx.x / TPR, l = threadIdx.x % TPR;
  const int C = p.C;
  const float inv_c = 1.0f / static_cast<float>(C);
  // rows that share a warp advance together (TPR < 32), so that its shuffles stay whole
  const int sub = TPR < 32 ? group % (32 / TPR) : 0;
  const T* x = static_cast<const T*>(p.x);
  int par = 0;
  uint4 cur[VPL], nxt[VPL];
  const int step = static_cast<int>(gridDim.x) * GROUPS;
  int base = static_cast<int>(blockIdx.x) * GROUPS + group - sub;
  auto load = [&](int r, uint4 (&v)[VPL]) {
    if (r < p.M) {
      load_row<T, TPR, VPL, VEC>(x + static_cast<int64_t>(r) * p.ldx, C, l, v);
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) v[i] = make_uint4(0, 0, 0, 0);
    }
  };
  if (base < p.M) load(base + sub, cur);
  for (; base < p.M; base += step) {
    const int row = base + sub;
    if (base + step < p.M) load(row + step, nxt);
    float2 s = make_float2(0.f, 0.f);  // two running sums; padding adds zero
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      float f[E];
      Elem<T>::unpack(cur[i], f);
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        s.x += f[e];
        s.y += f[e + 1];
      }
    }
    s = group_sum<TPR>(make_float2(s.x + s.y, 0.f), red, group, par);
    const float mean = s.x * inv_c;
    float2 q = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      float f[E];
      Elem<T>::unpack(cur[i], f);
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        if (col_of<T, TPR, VEC>(l, i, e) < C) {
          const float d = f[e] - mean;
          q.x = fmaf(d, d, q.x);
        }
        if (col_of<T, TPR, VEC>(l, i, e + 1) < C) {
          const float d = f[e + 1] - mean;
          q.y = fmaf(d, d, q.y);
        }
      }
    }
    q = group_sum<TPR>(make_float2(q.x + q.y, 0.f), red, group, par);
    const float rstd = rsqrtf(q.x * inv_c + p.eps);
    const bool live = row < p.M;
    if (live && l == 0 && p.stats != nullptr) p.stats[row] = make_float2(mean, rstd);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      float f[E], g[E], b[E];
      Elem<T>::unpack(cur[i], f);
      load_param<T, TPR, VEC>(p.gamma, p.p32, 1.f, C, l, i, g);
      load_param<T, TPR, VEC>(p.beta, p.p32, 0.f, C, l, i, b);
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = fmaf((f[e] - mean) * rstd, g[e], b[e]);
      if constexpr (!QUANT) {
        if (live) store_vec<T, TPR, VEC>(static_cast<T*>(p.y) + row * p.ldy, C, l, i, f);
      } else {
        // 16 neighbouring threads hold 128 columns: one block
        const int c = col_of<T, TPR, VEC>(l, i, 0);
        uint32_t a = 0;
        if (c < C) {
#pragma unroll
          for (int e = 0; e < E; ++e) a = max(a, abs_bits(f[e]));
        }
#pragma unroll
        for (int o = 8; o; o >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
        if (__any_sync(0xffffffffu, a >= kInfBits)) {
          a = 0;
          if (c < C) {
#pragma unroll
            for (int e = 0; e < E; ++e) a = max(a, finite_abs_bits(f[e]));
          }
#pragma unroll
          for (int o = 8; o; o >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
#pragma unroll
          for (int e = 0; e < E; ++e) f[e] = inf_to_nan(f[e]);
        }
        const uint32_t byte = e8m0_byte(a);
        const float inv = e8m0_inverse(byte);
        if (live && c < C) {
          uint2 o;
          o.x = e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
          o.y = e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv);
          *reinterpret_cast<uint2*>(p.q + row * p.ldq + c) = o;
          if ((l & 15) == 0) p.scales[scale_offset(row, c >> 7, p.kq)] = static_cast<uint8_t>(byte);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) cur[i] = nxt[i];
  }
}

// ---------------------------------------------------------------- backward
// Threads of a block: as many whole rows as fit in 384 threads at 168 registers each (one
// block per SM; a row's x, dy and dres and the next row's are in registers at once).
__host__ __device__ constexpr int bwd_threads(int tpr) { return tpr >= 256 ? tpr : 384 / tpr * tpr; }

template <typename T, int TPR, int VPL, bool VEC>
__global__ void __launch_bounds__(bwd_threads(TPR), 1)
    ln_bwd_kernel(const LnBackward p) {
  constexpr int E = Elem<T>::E;
  constexpr int GROUPS = bwd_threads(TPR) / TPR;
  constexpr int NA = VPL * E;  // columns of a thread
  static_assert(TPR >= 32, "a warp shares a row");
  __shared__ float2 red[TPR > 32 ? GROUPS * 2 * (TPR / 32) : 1];
  extern __shared__ float s_acc[];  // [GROUPS / 2 rounded up][2][NA][TPR]
  pdl_trigger();
  pdl_wait();
  const int group = threadIdx.x / TPR, l = threadIdx.x % TPR;
  const int C = p.C;
  const float inv_c = 1.0f / static_cast<float>(C);
  const T* x = static_cast<const T*>(p.x);
  const T* dy = static_cast<const T*>(p.dy);
  const T* dres = static_cast<const T*>(p.dres);
  T* dx = static_cast<T*>(p.dx);
  float dg[NA], db[NA];
#pragma unroll
  for (int k = 0; k < NA; ++k) dg[k] = db[k] = 0.f;
  int par = 0;
  uint4 xc[VPL], yc[VPL], rc[VPL], xn[VPL], yn[VPL], rn[VPL];
  float2 st = make_float2(0.f, 0.f), st_n = st;
  const int step = static_cast<int>(gridDim.x) * GROUPS;
  int row = static_cast<int>(blockIdx.x) * GROUPS + group;
  auto load = [&](int r, uint4 (&a)[VPL], uint4 (&b)[VPL], uint4 (&d)[VPL], float2& s) {
    s = __ldg(p.stats + r);
    load_row<T, TPR, VPL, VEC>(x + static_cast<int64_t>(r) * p.ldx, C, l, a);
    load_row<T, TPR, VPL, VEC>(dy + static_cast<int64_t>(r) * p.lddy, C, l, b);
    if (dres != nullptr)
      load_row<T, TPR, VPL, VEC>(dres + static_cast<int64_t>(r) * p.lddres, C, l, d);
  };
#pragma unroll
  for (int i = 0; i < VPL; ++i) rc[i] = rn[i] = make_uint4(0, 0, 0, 0);
  if (row < p.M) load(row, xc, yc, rc, st);
  for (; row < p.M; row += step) {
    if (row + step < p.M) load(row + step, xn, yn, rn, st_n);
    float2 s = make_float2(0.f, 0.f);  // sum w, sum w xh; padding has dy = 0
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      float fx[E], fy[E], g[E];
      Elem<T>::unpack(xc[i], fx);
      Elem<T>::unpack(yc[i], fy);
      load_param<T, TPR, VEC>(p.gamma, p.p32, 1.f, C, l, i, g);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float xh = (fx[e] - st.x) * st.y;
        const float w = fy[e] * g[e];
        s.x += w;
        s.y = fmaf(w, xh, s.y);
        dg[i * E + e] = fmaf(fy[e], xh, dg[i * E + e]);
        db[i * E + e] += fy[e];
      }
    }
    if (dx != nullptr) {
      s = group_sum<TPR>(s, red, group, par);
      const float m1 = s.x * inv_c, m2 = s.y * inv_c;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        float fx[E], fy[E], g[E], fr[E];
        Elem<T>::unpack(xc[i], fx);
        Elem<T>::unpack(yc[i], fy);
        Elem<T>::unpack(rc[i], fr);
        load_param<T, TPR, VEC>(p.gamma, p.p32, 1.f, C, l, i, g);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float xh = (fx[e] - st.x) * st.y;
          fr[e] = fmaf(st.y, fmaf(-xh, m2, fmaf(fy[e], g[e], -m1)), fr[e]);
        }
        store_vec<T, TPR, VEC>(dx + static_cast<int64_t>(row) * p.lddx, C, l, i, fr);
      }
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      xc[i] = xn[i];
      yc[i] = yn[i];
      rc[i] = rn[i];
    }
    st = st_n;
  }
  if (p.partials == nullptr) return;
  // the block's groups added pairwise in shared memory, the upper half into the lower
#pragma unroll
  for (int n = GROUPS; n > 1;) {
    const int h = (n + 1) / 2;
    if (group >= h && group < n) {
      float* a = s_acc + static_cast<size_t>(group - h) * 2 * NA * TPR + l;
#pragma unroll
      for (int k = 0; k < NA; ++k) {
        a[k * TPR] = dg[k];
        a[(NA + k) * TPR] = db[k];
      }
    }
    __syncthreads();
    if (group + h < n) {
      const float* a = s_acc + static_cast<size_t>(group) * 2 * NA * TPR + l;
#pragma unroll
      for (int k = 0; k < NA; ++k) {
        dg[k] += a[k * TPR];
        db[k] += a[(NA + k) * TPR];
      }
    }
    __syncthreads();
    n = h;
  }
  if (group == 0) {
    float* out = p.partials + static_cast<int64_t>(blockIdx.x) * 2 * C;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int c = col_of<T, TPR, VEC>(l, i, e);
        if (c < C) {
          out[c] = dg[i * E + e];
          out[C + c] = db[i * E + e];
        }
      }
    }
  }
}

// out[c] = sum of partials[p][c], p = 0 .. P-1, for n columns; columns below `split` go to
// out0, the others to out1 (either may be null). 32 columns per block, 8 threads per column
// taking every eighth partial, their sums added in order.
__global__ void __launch_bounds__(256)
    col_reduce_kernel(const float* partials, int P, int n, int split, float* out0, float* out1) {
  __shared__ float s[8][32];
  pdl_trigger();
  pdl_wait();
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int c = static_cast<int>(blockIdx.x) * 32 + tx;
  float v = 0.f;
  if (c < n) {
#pragma unroll 8
    for (int r = ty; r < P; r += 8) v += partials[static_cast<int64_t>(r) * n + c];
  }
  s[ty][tx] = v;
  __syncthreads();
  if (ty == 0 && c < n) {
#pragma unroll
    for (int i = 1; i < 8; ++i) v += s[i][tx];
    float* out = c < split ? out0 : out1;
    if (out != nullptr) out[c < split ? c : c - split] = v;
  }
}

cudaError_t launch_col_reduce(const float* partials, int P, int n, int split, float* out0,
                              float* out1, cudaStream_t stream, bool pdl) {
  return launch(col_reduce_kernel, dim3((n + 31) / 32), dim3(256), 0, stream, pdl, partials, P, n,
                split, out0, out1);
}

// ---------------------------------------------------------------- host launchers
template <typename T, int TPR, int VPL, bool VEC, bool QUANT>
static cudaError_t go_fwd(const LnForward& p, int num_sms, cudaStream_t s) {
  constexpr int groups = ln_threads(TPR) / TPR;
  const int64_t blocks = (static_cast<int64_t>(p.M) + groups - 1) / groups;
  const int64_t most = static_cast<int64_t>(num_sms) * (2048 / ln_threads(TPR));
  return launch(ln_fwd_kernel<T, TPR, VPL, VEC, QUANT>, dim3(blocks < most ? blocks : most),
                dim3(ln_threads(TPR)), 0, s, false, p);
}

// Threads per row by width, in 16-byte vectors of the row: narrow rows share a warp, so that
// its lanes are busy; wide ones take as many threads as keep a row within 4 vectors a thread.
// Both forward kernels divide a row the same way, so their statistics agree to the bit.
template <typename T, bool VEC>
static cudaError_t pick_fwd(const LnForward& p, int num_sms, cudaStream_t s) {
  const int n = (p.C + Elem<T>::E - 1) / Elem<T>::E;
  if (n <= 32) return go_fwd<T, 16, 2, VEC, false>(p, num_sms, s);
  if (n <= 64) return go_fwd<T, 16, 4, VEC, false>(p, num_sms, s);
  if (n <= 128) return go_fwd<T, 32, 4, VEC, false>(p, num_sms, s);
  if (n <= 256) return go_fwd<T, 64, 4, VEC, false>(p, num_sms, s);
  if (n <= 512) return go_fwd<T, 128, 4, VEC, false>(p, num_sms, s);
  if (n <= 1024) return go_fwd<T, 256, 4, VEC, false>(p, num_sms, s);
  if constexpr (sizeof(T) == 4) return go_fwd<T, 512, 4, VEC, false>(p, num_sms, s);
  return cudaErrorInvalidValue;
}

cudaError_t launch_ln_forward(const LnForward& p, int dtype, bool vec, int num_sms,
                              cudaStream_t s) {
  if (dtype == RS_BF16)
    return vec ? pick_fwd<__nv_bfloat16, true>(p, num_sms, s)
               : pick_fwd<__nv_bfloat16, false>(p, num_sms, s);
  if (dtype == RS_FP16)
    return vec ? pick_fwd<__half, true>(p, num_sms, s) : pick_fwd<__half, false>(p, num_sms, s);
  return vec ? pick_fwd<float, true>(p, num_sms, s) : pick_fwd<float, false>(p, num_sms, s);
}

template <typename T>
static cudaError_t pick_quant(const LnForward& p, int num_sms, cudaStream_t s) {
  const int n = p.C / 8;
  if (n <= 32) return go_fwd<T, 16, 2, true, true>(p, num_sms, s);
  if (n <= 64) return go_fwd<T, 16, 4, true, true>(p, num_sms, s);
  if (n <= 128) return go_fwd<T, 32, 4, true, true>(p, num_sms, s);
  if (n <= 256) return go_fwd<T, 64, 4, true, true>(p, num_sms, s);
  if (n <= 512) return go_fwd<T, 128, 4, true, true>(p, num_sms, s);
  return go_fwd<T, 256, 4, true, true>(p, num_sms, s);
}

cudaError_t launch_ln_quantize(const LnForward& p, int dtype, int num_sms, cudaStream_t s) {
  return dtype == RS_BF16 ? pick_quant<__nv_bfloat16>(p, num_sms, s)
                          : pick_quant<__half>(p, num_sms, s);
}

template <typename T, int TPR, int VPL, bool VEC>
static cudaError_t go_bwd(const LnBackward& p, int blocks, cudaStream_t s) {
  constexpr int groups = bwd_threads(TPR) / TPR;
  constexpr size_t smem = static_cast<size_t>(groups / 2) * 2 * VPL * Elem<T>::E * TPR * 4;
  auto kern = ln_bwd_kernel<T, TPR, VPL, VEC>;
  if constexpr (smem > 40 * 1024) {  // with the static part past the default 48 KB
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  return launch(kern, dim3(blocks), dim3(bwd_threads(TPR)), smem, s, false, p);
}

// Threads per row and vectors per thread, by the row's 16-byte vectors: at most 4 vectors a
// thread, so that its columns' sums and two rows of three tensors stay in registers.
template <typename T, bool VEC>
static cudaError_t pick_bwd(const LnBackward& p, int blocks, cudaStream_t s) {
  const int n = (p.C + Elem<T>::E - 1) / Elem<T>::E;
  if (n <= 32) return go_bwd<T, 32, 1, VEC>(p, blocks, s);
  if (n <= 64) return go_bwd<T, 32, 2, VEC>(p, blocks, s);
  if (n <= 96) return go_bwd<T, 32, 3, VEC>(p, blocks, s);
  if (n <= 128) return go_bwd<T, 32, 4, VEC>(p, blocks, s);
  if (n <= 256) return go_bwd<T, 64, 4, VEC>(p, blocks, s);
  if (n <= 512) return go_bwd<T, 128, 4, VEC>(p, blocks, s);
  if (n <= 1024) return go_bwd<T, 256, 4, VEC>(p, blocks, s);
  if constexpr (sizeof(T) == 4) return go_bwd<T, 512, 4, VEC>(p, blocks, s);
  return cudaErrorInvalidValue;
}

// Blocks of the backward kernel: one per SM, or fewer when the rows run out.
static int bwd_blocks(int M, int C, int elem, int num_sms) {
  const int n = (C + elem - 1) / elem;
  const int rows = n <= 128 ? 12 : n <= 256 ? 6 : n <= 512 ? 3 : 1;  // per block and step
  const int64_t blocks = (static_cast<int64_t>(M) + rows - 1) / rows;
  return static_cast<int>(blocks < num_sms ? blocks : num_sms);
}

cudaError_t launch_ln_backward(const LnBackward& p, int dtype, bool vec, int num_sms, float* dgamma,
                               float* dbeta, cudaStream_t s) {
  const int blocks = bwd_blocks(p.M, p.C, dtype == RS_FP32 ? 4 : 8, num_sms);
  cudaError_t e;
  if (dtype == RS_BF16)
    e = vec ? pick_bwd<__nv_bfloat16, true>(p, blocks, s) : pick_bwd<__nv_bfloat16, false>(p, blocks, s);
  else if (dtype == RS_FP16)
    e = vec ? pick_bwd<__half, true>(p, blocks, s) : pick_bwd<__half, false>(p, blocks, s);
  else
    e = vec ? pick_bwd<float, true>(p, blocks, s) : pick_bwd<float, false>(p, blocks, s);
  if (e != cudaSuccess || p.partials == nullptr) return e;
  return launch_col_reduce(p.partials, blocks, 2 * p.C, p.C, dgamma, dbeta, s, true);
}

}  // namespace rs
