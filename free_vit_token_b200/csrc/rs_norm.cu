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
// vectors each); blocks stay resident and walk the rows, and each row of threads keeps the
// next rows on their way into a ring in shared memory (cp.async), so that the bytes in flight
// do not depend on registers. Every value is read once, gamma and beta once per block.
// Arithmetic runs on pairs of fp32 lanes. Backward: a thread keeps its columns' dgamma and
// dbeta sums in fp32 registers over all the rows of its block, the blocks' sums go to the
// workspace once each and a second kernel adds them in a fixed order: no atomics, the same bits
// every run.
//
// Rows that do not start on 16 bytes (VEC = false) are copied as the aligned 16-byte units
// that cover them and shifted into place between shared memory and registers, both ways, so
// that global memory sees the same wide accesses.
//
// Measured (bf16): forward 25104 x 1024 18.5 us (5.6 TB/s), with 8-bit output 23.1 us (77 MB, 3.3
// TB/s: a row per warp through three chains of shuffles); gradients 50432 x 768 57 us (5.4 TB/s over
// x, dy, dres and dx). Rows off 16 bytes: 8577 x 1001 fp16 forward 14.3 us against 7.7 of 1000
// columns, gradients 29.6 against 18.2.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "rs_fp8.cuh"
#include "rs_ops.h"
#include "rs_ptx.cuh"

namespace rs {

// ---------------------------------------------------------------- rows
// Element e of vector i of thread l is column (l + TPR i) E + e.
template <typename T, int TPR>
__device__ __forceinline__ int col_of(int l, int i) {
  return (l + TPR * i) * Elem<T>::E;
}

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The threads of a row meet.
template <int TPR>
__device__ __forceinline__ void group_barrier(int group) {
  if constexpr (TPR <= 32)
    __syncwarp();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(TPR) : "memory");
}

// A strided matrix of T, and how its rows lie against 16-byte boundaries.
template <typename T, bool VEC>
struct Rows {
  const T* p;
  int64_t ld;
  int M, C;
  __device__ __forceinline__ const T* row(int r) const { return p + static_cast<int64_t>(r) * ld; }
  __device__ __forceinline__ int off(int r) const {
    return VEC ? 0 : static_cast<int>(reinterpret_cast<uintptr_t>(row(r)) & 15);
  }
  // Row r to `buf` (TPR * VPL + 1 units of 16 bytes) asynchronously. With VEC thread l copies
  // exactly what it reads; else the units at a row's ends come with the neighbouring rows'
  // bytes, which nothing uses, and only a unit that would pass an end of the tensor moves by
  // elements.
  template <int TPR, int VPL>
  __device__ __forceinline__ void fetch(uint8_t* buf, int r, int l) const {
    const int len = C * static_cast<int>(sizeof(T));
    if constexpr (VEC) {
      const uint8_t* src = reinterpret_cast<const uint8_t*>(row(r));
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int o = (l + TPR * i) * 16;
        if (o < len) cp_async16(buf + o, src + o);
      }
    } else {
      const int of = off(r);
      const uint8_t* base = reinterpret_cast<const uint8_t*>(row(r)) - of;
      const uint8_t* lo = reinterpret_cast<const uint8_t*>(p);
      const uint8_t* hi = reinterpret_cast<const uint8_t*>(row(M - 1) + C);
#pragma unroll
      for (int i = 0; i <= VPL; ++i) {
        const int o = (l + TPR * i) * 16;
        if (o >= of + len) break;
        if (base + o >= lo && base + o + 16 <= hi) {
          cp_async16(buf + o, base + o);
        } else {
#pragma unroll 1
          for (int b = o > of ? o : of; b < o + 16 && b < of + len; b += static_cast<int>(sizeof(T)))
            *reinterpret_cast<T*>(buf + b) = *reinterpret_cast<const T*>(base + b);
        }
      }
    }
  }
};

// Vector i of thread l of a row at byte `of` of `buf`; zero past C.
template <typename T, int TPR, bool VEC>
__device__ __forceinline__ uint4 read_vec(const uint8_t* buf, int of, int C, int l, int i) {
  constexpr int E = Elem<T>::E;
  const int c = col_of<T, TPR>(l, i);
  if (c >= C) return make_uint4(0, 0, 0, 0);
  const uint4* unit = reinterpret_cast<const uint4*>(buf) + l + TPR * i;
  const uint4 a = unit[0];
  if constexpr (VEC) {
    return a;
  } else {
    uint32_t w[8] = {a.x, a.y, a.z, a.w, 0, 0, 0, 0};
    if (of != 0) {  // the same for all threads of the row
      const uint4 b = unit[1];
      w[4] = b.x;
      w[5] = b.y;
      w[6] = b.z;
      w[7] = b.w;
      if (of & 8) {
#pragma unroll
        for (int j = 0; j < 6; ++j) w[j] = w[j + 2];
      }
      if (of & 4) {
#pragma unroll
        for (int j = 0; j < 5; ++j) w[j] = w[j + 1];
      }
      if (of & 2) {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = __funnelshift_r(w[j], w[j + 1], 16);
      }
    }
    if (c + E > C) {  // the row ends inside the vector
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (E == 8) {
          if (c + 2 * j >= C) w[j] = 0;
          else if (c + 2 * j + 1 >= C) w[j] &= 0xFFFFu;
        } else {
          if (c + j >= C) w[j] = 0;
        }
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// An output row: VEC, straight to global memory; else to byte `of` of `buf` (the offset of the
// row in global memory), from where flush_row writes whole 16-byte units.
template <typename T, int TPR, bool VEC>
__device__ __forceinline__ void write_vec(T* row, uint8_t* buf, int of, int C, int l, int i,
                                          const float (&f)[Elem<T>::E]) {
  const int c = col_of<T, TPR>(l, i);
  if (c >= C) return;
  const uint4 v = Elem<T>::pack(f);
  if constexpr (VEC) {
    *reinterpret_cast<uint4*>(row + c) = v;
  } else {
    uint8_t* d = buf + of + (l + TPR * i) * 16;
    if (of & 2) {  // 16-bit elements between words
      *reinterpret_cast<uint16_t*>(d) = static_cast<uint16_t>(v.x);
      *reinterpret_cast<uint32_t*>(d + 2) = __funnelshift_r(v.x, v.y, 16);
      *reinterpret_cast<uint32_t*>(d + 6) = __funnelshift_r(v.y, v.z, 16);
      *reinterpret_cast<uint32_t*>(d + 10) = __funnelshift_r(v.z, v.w, 16);
      *reinterpret_cast<uint16_t*>(d + 14) = static_cast<uint16_t>(v.w >> 16);
    } else {
      uint32_t* w = reinterpret_cast<uint32_t*>(d);
      w[0] = v.x;
      w[1] = v.y;
      w[2] = v.z;
      w[3] = v.w;
    }
  }
}
template <typename T, int TPR, int VPL>
__device__ __forceinline__ void flush_row(T* row, const uint8_t* buf, int of, int C, int l) {
  const int end = of + C * static_cast<int>(sizeof(T));
  uint8_t* base = reinterpret_cast<uint8_t*>(row) - of;
#pragma unroll
  for (int i = 0; i <= VPL; ++i) {
    const int o = (l + TPR * i) * 16;
    if (o >= end) break;
    if (o >= of && o + 16 <= end)
      *reinterpret_cast<uint4*>(base + o) = *reinterpret_cast<const uint4*>(buf + o);
  }
  // the elements of the two units at the ends that belong to this row, one per thread
  constexpr int S = static_cast<int>(sizeof(T)), N = 16 / S;
  static_assert(TPR >= 2 * N, "threads for both ends");
  const int head = of == 0 ? 0 : 16, tail = end & ~15;
  const int b = l < N ? of + l * S : tail + (l - N) * S;
  const bool mine = l < N ? b < head && b < end : l < 2 * N && b < end && tail >= head;
  if (mine && (l < N || b >= of)) *reinterpret_cast<T*>(base + b) = *reinterpret_cast<const T*>(buf + b);
}

// gamma or beta in pairs of fp32; 1 or 0 where there is none.
template <typename T, bool VEC, bool P32>
__device__ __forceinline__ void param_pairs(const void* p, float def, int c, int C,
                                            uint64_t (&f)[Elem<T>::E / 2]) {
  constexpr int E = Elem<T>::E;
  if (p == nullptr) {
#pragma unroll
    for (int e = 0; e < E / 2; ++e) f[e] = f2pack(def, def);
    return;
  }
#pragma unroll
  for (int e = 0; e < E / 2; ++e) {
    float v[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (c + 2 * e + k < C)
        v[k] = P32 ? __ldg(static_cast<const float*>(p) + c + 2 * e + k)
                   : static_cast<float>(static_cast<const T*>(p)[c + 2 * e + k]);
    f[e] = f2pack(v[0], v[1]);
  }
}

// A block's copy of gamma or beta: 16-bit ones of aligned rows stay in registers as they are
// (REGS), others are pairs of fp32 in shared memory, [VPL * E / 2][TPR].
template <typename T, int TPR, int VPL, bool VEC, bool P32, bool REGS>
struct Params {
  static constexpr int E = Elem<T>::E;
  const void* p;
  float def;
  const uint64_t* s;
  uint4 raw[REGS ? VPL : 1];
  // `s_` [VPL * E / 2][TPR] is filled by the block's first row of threads; the caller puts a
  // __syncthreads between this and get().
  __device__ __forceinline__ Params(const void* p_, float def_, int C, int group, int l, uint64_t* s_)
      : p(p_), def(def_), s(s_ + l) {
    if constexpr (REGS) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int c = col_of<T, TPR>(l, i);
        raw[i] = make_uint4(0, 0, 0, 0);
        if (p != nullptr && c < C) raw[i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p) + c));
      }
    } else if (group == 0) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        uint64_t f[E / 2];
        param_pairs<T, VEC, P32>(p, def, col_of<T, TPR>(l, i), C, f);
#pragma unroll
        for (int e = 0; e < E / 2; ++e) s_[(i * E / 2 + e) * TPR + l] = f[e];
      }
    }
  }
  __device__ __forceinline__ void get(int i, uint64_t (&f)[E / 2]) const {
    if constexpr (REGS) {
      if (p == nullptr) {
#pragma unroll
        for (int e = 0; e < E / 2; ++e) f[e] = f2pack(def, def);
      } else {
        Elem<T>::pairs(raw[i], f);
      }
    } else {
#pragma unroll
      for (int e = 0; e < E / 2; ++e) f[e] = s[(i * E / 2 + e) * TPR];
    }
  }
};

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
    group_barrier<TPR>(group);
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
template <int TPR>
__device__ __forceinline__ float group_sum(float v, float2* red, int group, int& par) {
  if constexpr (TPR > 32) return group_sum<TPR>(make_float2(v, 0.f), red, group, par).x;
#pragma unroll
  for (int o = (TPR < 32 ? TPR : 32) / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__host__ __device__ constexpr int ring_row_bytes(int tpr, int vpl) { return (tpr * vpl + 1) * 16; }

// ---------------------------------------------------------------- forward
// Two blocks of 256 threads per SM (wide rows: one of 512), 3 rows on their way per row of
// threads beside the one in use: 96 KB in flight per SM at 1024 bf16 columns.
__host__ __device__ constexpr int fwd_threads(int tpr) { return tpr > 256 ? tpr : 256; }
constexpr int kFwdStages = 4;
template <typename T, bool VEC, bool P32>
__host__ __device__ constexpr bool fwd_param_regs() {
  return VEC && (sizeof(T) == 4 || !P32);
}
template <typename T, int TPR, int VPL, bool VEC, bool P32>
__host__ __device__ constexpr int fwd_smem() {
  return fwd_threads(TPR) / TPR * kFwdStages * ring_row_bytes(TPR, VPL) +
         (fwd_param_regs<T, VEC, P32>() ? 0 : 2 * VPL * Elem<T>::E * TPR * 4);
}

template <typename T, int TPR, int VPL, bool VEC, bool P32, bool QUANT>
__global__ void __launch_bounds__(fwd_threads(TPR), TPR <= 256 ? 2 : 1)
    ln_fwd_kernel(const LnForward p) {
  constexpr int E = Elem<T>::E;
  constexpr int GROUPS = fwd_threads(TPR) / TPR;
  constexpr int RB = ring_row_bytes(TPR, VPL);
  constexpr bool REGS = fwd_param_regs<T, VEC, P32>();
  static_assert(!QUANT || (VEC && E == 8 && TPR >= 16), "16 threads hold a block of 128");
  __shared__ float2 red[TPR > 32 ? GROUPS * 2 * (TPR / 32) : 1];
  extern __shared__ __align__(16) uint8_t s_dyn[];
  uint64_t* s_par = reinterpret_cast<uint64_t*>(s_dyn + GROUPS * kFwdStages * RB);
  pdl_trigger();
  pdl_wait();
  const int group = threadIdx.x / TPR, l = threadIdx.x % TPR;
  const int C = p.C;
  const float inv_c = 1.0f / static_cast<float>(C);
  const Rows<T, VEC> x{static_cast<const T*>(p.x), p.ldx, p.M, C};
  uint8_t* ring = s_dyn + group * kFwdStages * RB;
  const int step = static_cast<int>(gridDim.x) * GROUPS;
  int row = static_cast<int>(blockIdx.x) * GROUPS + group;
  auto fetch = [&](int r, int slot) {
    if (r < p.M) x.template fetch<TPR, VPL>(ring + slot * RB, r, l);
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kFwdStages - 1; ++i) fetch(row + i * step, i);
  const Params<T, TPR, VPL, VEC, P32, REGS> gamma(p.gamma, 1.f, C, group, l, s_par);
  const Params<T, TPR, VPL, VEC, P32, REGS> beta(p.beta, 0.f, C, group, l, s_par + VPL * E / 2 * TPR);
  if constexpr (!REGS) __syncthreads();
  int par = 0, slot = 0;
  // rows that share a warp (TPR < 32) go through the same steps, past the end too
  const int sub = TPR < 32 ? group % (32 / TPR) : 0;
  for (; row - sub < p.M; row += step) {
    const bool live = row < p.M;
    cp_async_wait<kFwdStages - 2>();
    // not VEC: other threads copied parts of the row; and all of them are done with the slot
    // that is refilled next
    if constexpr (!VEC) group_barrier<TPR>(group);
    fetch(row + (kFwdStages - 1) * step, slot == 0 ? kFwdStages - 1 : slot - 1);
    uint8_t* buf = ring + slot * RB;
    slot = slot + 1 == kFwdStages ? 0 : slot + 1;
    uint4 cur[VPL];
    const int xof = x.off(row);
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      cur[i] = live ? read_vec<T, TPR, VEC>(buf, xof, C, l, i) : make_uint4(0, 0, 0, 0);
    uint64_t xs[VPL][E / 2];  // the row's values as pairs of fp32
    uint64_t s2 = 0;          // pairs of running sums; padding adds zero
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      Elem<T>::pairs(cur[i], xs[i]);
#pragma unroll
      for (int e = 0; e < E / 2; ++e) s2 = fadd2(s2, xs[i][e]);
    }
    float2 t = f2unpack(s2);
    const float mean = group_sum<TPR>(t.x + t.y, red, group, par) * inv_c;
    const uint64_t nmean = f2pack(-mean, -mean);
    uint64_t q2 = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int c = col_of<T, TPR>(l, i);
#pragma unroll
      for (int e = 0; e < E / 2; ++e) {
        xs[i][e] = fadd2(xs[i][e], nmean);
        uint64_t d = xs[i][e];
        if constexpr (!VEC) {
          if (c + 2 * e + 1 >= C) d = c + 2 * e >= C ? 0 : static_cast<uint32_t>(d);
        }
        if (!VEC || c < C) q2 = ffma2(d, d, q2);
      }
    }
    t = f2unpack(q2);
    const float var = group_sum<TPR>(t.x + t.y, red, group, par) * inv_c;
    const float rstd = rsqrtf(var + p.eps);
    const uint64_t rstd2 = f2pack(rstd, rstd);
    if (live && l == 0 && p.stats != nullptr) p.stats[row] = make_float2(mean, rstd);
    T* y = static_cast<T*>(p.y) + static_cast<int64_t>(row) * p.ldy;
    const int yof = VEC ? 0 : static_cast<int>(reinterpret_cast<uintptr_t>(y) & 15);
    auto affine = [&](int i, float (&f)[E]) {
      uint64_t g[E / 2], b[E / 2];
      gamma.get(i, g);
      beta.get(i, b);
#pragma unroll
      for (int e = 0; e < E / 2; ++e) {
        const float2 v = f2unpack(ffma2(mul2(xs[i][e], rstd2), g[e], b[e]));
        f[2 * e] = v.x;
        f[2 * e + 1] = v.y;
      }
    };
    if constexpr (!QUANT) {
      if constexpr (!VEC) group_barrier<TPR>(group);  // the slot is read: y takes its place
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        float f[E];
        affine(i, f);
        if (live) write_vec<T, TPR, VEC>(y, buf, yof, C, l, i, f);
      }
    } else {
      // 16 neighbouring threads hold 128 columns: one block per vector. The blocks' maxima go
      // through their shuffles together, so that the chains overlap.
      float f[VPL][E], a[VPL], all = 0.f;  // maxima of magnitudes, which NaN does not enter
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        affine(i, f[i]);
        a[i] = 0.f;
        if (col_of<T, TPR>(l, i) < C) {
#pragma unroll
          for (int e = 0; e < E; ++e) a[i] = fmaxf(a[i], fabsf(f[i][e]));
        }
        all = fmaxf(all, a[i]);
      }
      if (__any_sync(0xffffffffu, abs_bits(all) >= kInfBits)) {  // rare: infinities
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          a[i] = 0.f;
#pragma unroll
          for (int e = 0; e < E; ++e) {
            f[i][e] = inf_to_nan(f[i][e]);
            if (col_of<T, TPR>(l, i) < C) a[i] = fmaxf(a[i], fabsf(f[i][e]));
          }
        }
      }
#pragma unroll
      for (int o = 8; o; o >>= 1)
#pragma unroll
        for (int i = 0; i < VPL; ++i) a[i] = fmaxf(a[i], __shfl_xor_sync(0xffffffffu, a[i], o));
      uint8_t* q = p.q + static_cast<int64_t>(row) * p.ldq;
      uint8_t* sc = p.scales + scale_offset(row, 0, p.kq);
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int c = col_of<T, TPR>(l, i);
        const uint32_t byte = e8m0_byte(__float_as_uint(a[i]));
        const float inv = e8m0_inverse(byte);
        const uint64_t inv2 = f2pack(inv, inv);
        if (live && c < C) {
          float2 g[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) g[e] = f2unpack(mul2(f2pack(f[i][2 * e], f[i][2 * e + 1]), inv2));
          *reinterpret_cast<uint2*>(q + c) = make_uint2(e4m3x4(g[0].x, g[0].y, g[1].x, g[1].y),
                                                        e4m3x4(g[2].x, g[2].y, g[3].x, g[3].y));
          if ((l & 15) == 0) sc[((c >> 9) << 9) + ((c >> 7) & 3)] = static_cast<uint8_t>(byte);
        }
      }
    }
    if constexpr (!VEC && !QUANT) {
      group_barrier<TPR>(group);
      if (live) flush_row<T, TPR, VPL>(y, buf, yof, C, l);
    }
  }
  cp_async_wait<0>();
}

// ---------------------------------------------------------------- backward
// Up to this many rows per row of threads of a block, a cluster of 8 blocks takes them all (4
// each) and the call is one launch without scratch: 394 x 192 fp32 16 us of host time a call
// against 20 (on the device, back to back, 7.0 us against 4.4).
constexpr int kLnFewRows = 32;

// Threads of a block (one per SM): 512 at 128 registers each where a thread's columns' sums (16
// bytes each) leave room, else 384 at 168. Each row of threads keeps a ring of 3 rows (2 where
// those are too large) of x, dy and dres, all but the one in use on their way: up to 112 KB per SM.
__host__ __device__ constexpr int bwd_threads(int tpr, int na) {
  return na <= 16 || tpr == 512 ? 512 : 384 / tpr * tpr;
}
__host__ __device__ constexpr int bwd_stages(int tpr, int vpl, int na) {
  return bwd_threads(tpr, na) / tpr * 9 * ring_row_bytes(tpr, vpl) + na * tpr * 4 + 1024 <= 232448 ? 3 : 2;
}
__host__ __device__ constexpr int bwd_ring_bytes(int tpr, int vpl, int na) {
  return bwd_threads(tpr, na) / tpr * bwd_stages(tpr, vpl, na) * 3 * ring_row_bytes(tpr, vpl);
}
template <typename T, int VPL, bool VEC, bool P32>
__host__ __device__ constexpr bool bwd_param_regs() {
  return VEC && (sizeof(T) == 4 || (!P32 && VPL <= 3));
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

template <typename T, int TPR, int VPL, bool VEC, bool P32>
__global__ void __launch_bounds__(bwd_threads(TPR, VPL * Elem<T>::E), 1)
    ln_bwd_kernel(const LnBackward p) {
  constexpr int E = Elem<T>::E;
  constexpr int NA = VPL * E;  // columns of a thread
  constexpr int THREADS = bwd_threads(TPR, NA), GROUPS = THREADS / TPR;
  constexpr int RB = ring_row_bytes(TPR, VPL);
  constexpr int STAGES = bwd_stages(TPR, VPL, NA);
  constexpr bool REGS = bwd_param_regs<T, VPL, VEC, P32>();
  static_assert(TPR >= 32, "a warp shares a row");
  __shared__ float2 red[TPR > 32 ? GROUPS * 2 * (TPR / 32) : 1];
  extern __shared__ __align__(16) uint8_t s_dyn[];
  pdl_trigger();
  pdl_wait();
  const int group = threadIdx.x / TPR, l = threadIdx.x % TPR;
  const int C = p.C;
  const float inv_c = 1.0f / static_cast<float>(C);
  const Rows<T, VEC> x{static_cast<const T*>(p.x), p.ldx, p.M, C};
  const Rows<T, VEC> dy{static_cast<const T*>(p.dy), p.lddy, p.M, C};
  const Rows<T, VEC> dres{static_cast<const T*>(p.dres), p.lddres, p.M, C};
  uint8_t* ring = s_dyn + group * STAGES * 3 * RB;
  const int step = static_cast<int>(gridDim.x) * GROUPS;
  int row = static_cast<int>(blockIdx.x) * GROUPS + group;
  auto fetch = [&](int r, int slot) {
    if (r < p.M) {
      uint8_t* b = ring + slot * 3 * RB;
      x.template fetch<TPR, VPL>(b, r, l);
      dy.template fetch<TPR, VPL>(b + RB, r, l);
      if (dres.p != nullptr) dres.template fetch<TPR, VPL>(b + 2 * RB, r, l);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) fetch(row + i * step, i);
  const Params<T, TPR, VPL, VEC, P32, REGS> gamma(
      p.gamma, 1.f, C, group, l, reinterpret_cast<uint64_t*>(s_dyn + bwd_ring_bytes(TPR, VPL, NA)));
  if constexpr (!REGS) __syncthreads();
  uint64_t dg2[NA / 2], db2[NA / 2];  // pairs of columns
#pragma unroll
  for (int k = 0; k < NA / 2; ++k) dg2[k] = db2[k] = 0;
  int par = 0, slot = 0;
  for (; row < p.M; row += step) {
    const float2 st = __ldg(p.stats + row);
    cp_async_wait<STAGES - 2>();
    // not VEC: other threads copied parts of the row; and all of them are done with the slot
    // that is refilled next
    if constexpr (!VEC) group_barrier<TPR>(group);
    fetch(row + (STAGES - 1) * step, slot == 0 ? STAGES - 1 : slot - 1);
    uint8_t* b = ring + slot * 3 * RB;
    slot = slot + 1 == STAGES ? 0 : slot + 1;
    uint4 xc[VPL], yc[VPL];
    const int xof = x.off(row), yof = dy.off(row);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      xc[i] = read_vec<T, TPR, VEC>(b, xof, C, l, i);
      yc[i] = read_vec<T, TPR, VEC>(b + RB, yof, C, l, i);
    }
    const uint64_t nmean = f2pack(-st.x, -st.x), rstd = f2pack(st.y, st.y);
    uint64_t w2 = 0, wx2 = 0;  // sum w, sum w xh; padding has dy = 0
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      uint64_t fx[E / 2], fy[E / 2], g[E / 2];
      Elem<T>::pairs(xc[i], fx);
      Elem<T>::pairs(yc[i], fy);
      gamma.get(i, g);
#pragma unroll
      for (int e = 0; e < E / 2; ++e) {
        const uint64_t xh = mul2(fadd2(fx[e], nmean), rstd);
        const uint64_t w = mul2(fy[e], g[e]);
        w2 = fadd2(w2, w);
        wx2 = ffma2(w, xh, wx2);
        dg2[i * E / 2 + e] = ffma2(fy[e], xh, dg2[i * E / 2 + e]);
        db2[i * E / 2 + e] = fadd2(db2[i * E / 2 + e], fy[e]);
      }
    }
    if (p.dx == nullptr) continue;
    const float2 wf = f2unpack(w2), wxf = f2unpack(wx2);
    const float2 s = group_sum<TPR>(make_float2(wf.x + wf.y, wxf.x + wxf.y), red, group, par);
    const float m1 = s.x * inv_c, m2 = s.y * inv_c;
    const uint64_t nm1 = f2pack(-m1, -m1), nm2 = f2pack(-m2, -m2);
    uint4 rc[VPL];
    const int rof = dres.p != nullptr ? dres.off(row) : 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      rc[i] = dres.p != nullptr ? read_vec<T, TPR, VEC>(b + 2 * RB, rof, C, l, i)
                                : make_uint4(0, 0, 0, 0);
    T* dx = static_cast<T*>(p.dx) + static_cast<int64_t>(row) * p.lddx;
    const int dof = VEC ? 0 : static_cast<int>(reinterpret_cast<uintptr_t>(dx) & 15);
    if constexpr (!VEC) group_barrier<TPR>(group);  // dres is read: dx takes its place
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      uint64_t fx[E / 2], fy[E / 2], g[E / 2], fr[E / 2];
      float o[E];
      Elem<T>::pairs(xc[i], fx);
      Elem<T>::pairs(yc[i], fy);
      Elem<T>::pairs(rc[i], fr);
      gamma.get(i, g);
#pragma unroll
      for (int e = 0; e < E / 2; ++e) {
        const uint64_t xh = mul2(fadd2(fx[e], nmean), rstd);
        const float2 v = f2unpack(ffma2(rstd, ffma2(xh, nm2, ffma2(fy[e], g[e], nm1)), fr[e]));
        o[2 * e] = v.x;
        o[2 * e + 1] = v.y;
      }
      write_vec<T, TPR, VEC>(dx, b + 2 * RB, dof, C, l, i, o);
    }
    if constexpr (!VEC) {
      group_barrier<TPR>(group);
      flush_row<T, TPR, VPL>(dx, b + 2 * RB, dof, C, l);
    }
  }
  cp_async_wait<0>();
  __syncthreads();  // the ring's memory now adds up the sums
  if (!p.sums) return;
  // every group's sums to [group][dgamma, dbeta][column], then one thread per column adds the
  // groups in order
  constexpr int W = TPR * NA;  // columns with padding
  float* acc = reinterpret_cast<float*>(s_dyn);
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    float4* a = reinterpret_cast<float4*>(acc + group * 2 * W + col_of<T, TPR>(l, i));
#pragma unroll
    for (int e = 0; e < E / 4; ++e) {
      const float2 u = f2unpack(dg2[i * E / 2 + 2 * e]), v = f2unpack(dg2[i * E / 2 + 2 * e + 1]);
      a[e] = make_float4(u.x, u.y, v.x, v.y);
      const float2 q = f2unpack(db2[i * E / 2 + 2 * e]), r = f2unpack(db2[i * E / 2 + 2 * e + 1]);
      a[W / 4 + e] = make_float4(q.x, q.y, r.x, r.y);
    }
  }
  __syncthreads();
  float* out = p.partials + static_cast<int64_t>(blockIdx.x) * 2 * C;
  for (int k = threadIdx.x; k < 2 * W; k += THREADS) {
    const int c = k < W ? k : k - W;
    if (c < C) {
      float v = acc[k];
#pragma unroll
      for (int g = 1; g < GROUPS; ++g) v += acc[g * 2 * W + k];
      if (p.cluster > 0)
        acc[k] = v;  // this thread's own place
      else
        out[k < W ? c : C + c] = v;
    }
  }
  if (p.cluster == 0) return;
  // few rows: the blocks are one cluster and add their sums through distributed shared memory,
  // each block a share of the columns, the blocks in rank order
  cluster_sync();
  const int rank = static_cast<int>(blockIdx.x);
  for (int k = rank * THREADS + threadIdx.x; k < 2 * W; k += p.cluster * THREADS) {
    const int c = k < W ? k : k - W;
    float* dst = k < W ? p.dgamma : p.dbeta;
    if (c < C && dst != nullptr) {
      float v = 0.f;
      for (int r = 0; r < p.cluster; ++r) v += ld_cluster_f32(mapa_shared(smem_u32(acc + k), r));
      dst[c] = v;
    }
  }
  cluster_sync();  // the others have read this block's sums
}

// out[c] = sum of partials[p][c], p = 0 .. P-1, for n columns; columns below `split` go to
// out0, the others to out1 (either may be null). 32 columns per block, 16 threads per column
// taking every sixteenth partial, their sums added in order.
__global__ void __launch_bounds__(512)
    col_reduce_kernel(const float* partials, int P, int n, int split, float* out0, float* out1) {
  __shared__ float s[16][32];
  pdl_trigger();
  pdl_wait();
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int c = static_cast<int>(blockIdx.x) * 32 + tx;
  float v = 0.f;
  if (c < n) {
#pragma unroll 10
    for (int r = ty; r < P; r += 16) v += partials[static_cast<int64_t>(r) * n + c];
  }
  s[ty][tx] = v;
  __syncthreads();
  if (ty == 0 && c < n) {
#pragma unroll
    for (int i = 1; i < 16; ++i) v += s[i][tx];
    float* out = c < split ? out0 : out1;
    if (out != nullptr) out[c < split ? c : c - split] = v;
  }
}

cudaError_t launch_col_reduce(const float* partials, int P, int n, int split, float* out0,
                              float* out1, cudaStream_t stream, bool pdl) {
  return launch(col_reduce_kernel, dim3((n + 31) / 32), dim3(512), 0, stream, pdl, partials, P, n,
                split, out0, out1);
}

// ---------------------------------------------------------------- host launchers
template <typename T, int TPR, int VPL, bool VEC, bool QUANT, bool P32>
static cudaError_t go_fwd_p(const LnForward& p, int num_sms, cudaStream_t s) {
  constexpr int groups = fwd_threads(TPR) / TPR;
  constexpr int smem = fwd_smem<T, TPR, VPL, VEC, P32>();
  static_assert(smem + 1024 <= 232448, "shared memory");
  constexpr int per_sm = TPR <= 256 && 2 * (smem + 2048) <= 232448 ? 2 : 1;
  auto kern = ln_fwd_kernel<T, TPR, VPL, VEC, P32, QUANT>;
  if constexpr (smem > 40 * 1024) {  // with the static part past the default 48 KB
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_smem(kern, smem, allowed);
    if (e != cudaSuccess) return e;
  }
  const int blocks = (p.M + groups - 1) / groups, most = per_sm * num_sms;
  return launch(kern, dim3(blocks < most ? blocks : most), dim3(fwd_threads(TPR)), smem, s, false, p);
}
template <typename T, int TPR, int VPL, bool VEC, bool QUANT>
static cudaError_t go_fwd(const LnForward& p, int num_sms, cudaStream_t s) {
  if constexpr (sizeof(T) == 4) return go_fwd_p<T, TPR, VPL, VEC, QUANT, true>(p, num_sms, s);
  return p.p32 ? go_fwd_p<T, TPR, VPL, VEC, QUANT, true>(p, num_sms, s)
               : go_fwd_p<T, TPR, VPL, VEC, QUANT, false>(p, num_sms, s);
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

template <typename T, int TPR, int VPL, bool VEC, bool P32>
static cudaError_t go_bwd_p(const LnBackward& p, int num_sms, int* P, cudaStream_t s) {
  constexpr int NA = VPL * Elem<T>::E, threads = bwd_threads(TPR, NA);
  static_assert(threads * NA * 8 <= bwd_ring_bytes(TPR, VPL, NA), "the sums fit the ring");
  constexpr size_t smem =
      bwd_ring_bytes(TPR, VPL, NA) + (bwd_param_regs<T, VPL, VEC, P32>() ? 0 : NA * TPR * 4);
  static_assert(smem + 1024 <= 232448, "shared memory");
  auto kern = ln_bwd_kernel<T, TPR, VPL, VEC, P32>;
  if constexpr (smem > 40 * 1024) {  // with the static part past the default 48 KB
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_smem(kern, static_cast<int>(smem), allowed);
    if (e != cudaSuccess) return e;
  }
  constexpr int groups = threads / TPR;
  const int64_t blocks = (static_cast<int64_t>(p.M) + groups - 1) / groups;
  if (p.M <= kLnFewRows * groups) {  // one launch: a cluster of up to 8 blocks adds the sums itself
    LnBackward f = p;
    f.cluster = static_cast<int>(blocks < 8 ? blocks : 8);
    *P = 0;
    return launch_cluster(kern, dim3(f.cluster), dim3(threads), smem, s, false, f.cluster, f);
  }
  *P = static_cast<int>(blocks < num_sms ? blocks : num_sms);
  return launch(kern, dim3(*P), dim3(threads), smem, s, false, p);
}
template <typename T, int TPR, int VPL, bool VEC>
static cudaError_t go_bwd(const LnBackward& p, int num_sms, int* P, cudaStream_t s) {
  if constexpr (sizeof(T) == 4) return go_bwd_p<T, TPR, VPL, VEC, true>(p, num_sms, P, s);
  return p.p32 ? go_bwd_p<T, TPR, VPL, VEC, true>(p, num_sms, P, s)
               : go_bwd_p<T, TPR, VPL, VEC, false>(p, num_sms, P, s);
}

// Threads per row and vectors per thread, by the row's 16-byte vectors: at most 24 columns of
// 16-bit values a thread (at 32, its sums and rows spill: 50000 x 1024 bf16 97 us against 75
// with 64 threads of 16 columns), 16 of fp32. *P is the number of blocks, each with a partial.
template <typename T, bool VEC>
static cudaError_t pick_bwd(const LnBackward& p, int num_sms, int* P, cudaStream_t s) {
  const int n = (p.C + Elem<T>::E - 1) / Elem<T>::E;
  if (n <= 32) return go_bwd<T, 32, 1, VEC>(p, num_sms, P, s);
  if (n <= 64) return go_bwd<T, 32, 2, VEC>(p, num_sms, P, s);
  if (n <= 96) return go_bwd<T, 32, 3, VEC>(p, num_sms, P, s);
  if (n <= 128) return go_bwd<T, 64, 2, VEC>(p, num_sms, P, s);
  if (n <= 192) return go_bwd<T, 64, 3, VEC>(p, num_sms, P, s);
  if (n <= 256) return go_bwd<T, 128, 2, VEC>(p, num_sms, P, s);
  if (n <= 512) return go_bwd<T, 256, 2, VEC>(p, num_sms, P, s);
  if (n <= 1024) return go_bwd<T, 512, 2, VEC>(p, num_sms, P, s);
  if constexpr (sizeof(T) == 4) return go_bwd<T, 512, 4, VEC>(p, num_sms, P, s);
  return cudaErrorInvalidValue;
}

// Does no type need scratch for these sizes? (Rows of threads per block as pick_bwd has them.)
bool ln_backward_few(int M, int C) {
  auto groups = [](int n, int e) {
    const int tpr = n <= 96 ? 32 : n <= 192 ? 64 : n <= 256 ? 128 : n <= 512 ? 256 : 512;
    const int v = n <= 32 ? 1 : n <= 64 ? 2 : n <= 96 ? 3 : n <= 128 ? 2 : n <= 192 ? 3 : n <= 1024 ? 2 : 4;
    return bwd_threads(tpr, v * e) / tpr;
  };
  const int a = groups((C + 7) / 8, 8), b = groups((C + 3) / 4, 4);
  return M <= kLnFewRows * (a < b ? a : b);
}

cudaError_t launch_ln_backward(const LnBackward& p, int dtype, bool vec, int num_sms,
                               cudaStream_t s) {
  int blocks = 0;
  cudaError_t e;
  if (dtype == RS_BF16)
    e = vec ? pick_bwd<__nv_bfloat16, true>(p, num_sms, &blocks, s) : pick_bwd<__nv_bfloat16, false>(p, num_sms, &blocks, s);
  else if (dtype == RS_FP16)
    e = vec ? pick_bwd<__half, true>(p, num_sms, &blocks, s) : pick_bwd<__half, false>(p, num_sms, &blocks, s);
  else
    e = vec ? pick_bwd<float, true>(p, num_sms, &blocks, s) : pick_bwd<float, false>(p, num_sms, &blocks, s);
  if (e != cudaSuccess || !p.sums || blocks == 0) return e;
  return launch_col_reduce(p.partials, blocks, 2 * p.C, p.C, p.dgamma, p.dbeta, s, true);
}

}  // namespace rs
