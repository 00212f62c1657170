// rs_fp8_few.cu -- a linear layer on a few rows (tokens served one by one) with its weight in
// 8-bit blocks (rs_fp8.cuh): out = act(Q(x) W^T + bias) + resid for up to 32 rows of x, in one
// launch without scratch.
//
// What bounds it is reading the weight once, and below a few MB the latency of one pass over
// the chip. So the operands change places: 128 rows of W are the matrix instruction's M side
// and the tokens its N side (16 or 32 columns), no lane works on padding rows of a 128-row
// token tile, and the reduction is split over a cluster of up to 8 CTAs, so that about as many
// CTAs as SMs each have all their weight tiles on the way at once. Every CTA quantises its own
// part of x (a few KB, from L2) into the swizzled operand layout while its weights arrive. The
// cluster adds its partial sums through distributed shared memory in rank order: the same bits
// every run.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "rs_fp8.cuh"
#include "rs_gelu8.cuh"
#include "rs_ops.h"
#include "rs_ptx_mx.cuh"

namespace rs {

namespace {

constexpr int kFThreads = 256;
constexpr int kFMaxBlocks = 8;                  // K blocks of 128 per CTA, all in flight
constexpr int kFMaxTiles = 3;                   // scale tiles those can touch
constexpr int kFABytes = 128 * 128;             // weight tile of one K block
constexpr uint32_t kFTmemCols = 64;             // 32 accumulator + 2 x 3 x 4 scale columns

__host__ __device__ constexpr int f_smem(int tokens, int blocks) {
  return 1024 + blocks * (kFABytes + tokens * 128) + 2 * kFMaxTiles * kScaleTile + tokens * 128 * 4 +
         256;
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

}  // namespace

template <int T>
__global__ void __launch_bounds__(kFThreads)
    fp8_few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmSW,
                   const Fp8Few p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sA = smem;                                   // [blocks][128 rows][128 B], swizzled
  uint8_t* sB = sA + p.blocks * kFABytes;               // [blocks][T rows][128 B], swizzled
  uint8_t* sSA = sB + p.blocks * T * 128;               // weight scale tiles
  uint8_t* sSB = sSA + kFMaxTiles * kScaleTile;         // token scale tiles
  float* sD = reinterpret_cast<float*>(sSB + kFMaxTiles * kScaleTile);  // [T][128]
  uint64_t* full = reinterpret_cast<uint64_t*>(sD + T * 128);
  uint64_t* done = full + kFMaxBlocks;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = p.split > 1 ? cluster_ctarank() : 0u;
  const int n0 = static_cast<int>(blockIdx.x) / p.split * 128;
  const int KB = (p.K + 127) / 128;
  const int kb0 = static_cast<int>(rank) * p.blocks;    // this CTA's K blocks
  const int nb = KB - kb0 < p.blocks ? (KB - kb0 > 0 ? KB - kb0 : 0) : p.blocks;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kFMaxBlocks; ++i) mbar_init(&full[i], 1);
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, kFTmemCols);
    tmem_relinquish();
  }
  pdl_trigger();
  pdl_wait();
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const WaitCtl wc{abort_flag, p.err, p.timeout_ns};

  if (warp == 0 && elect_one()) {
    for (int i = p.debug_skip && blockIdx.x == 0 ? 1 : 0; i < nb; ++i) {
      const int kb = kb0 + i;
      const bool scales = i == 0 || (kb & 3) == 0;
      mbar_arrive_expect_tx(&full[i], kFABytes + (scales ? kScaleTile : 0));
      tma_load_2d(sA + i * kFABytes, &tmW, &full[i], kb * 128, n0);
      if (scales)
        tma_load_3d(sSA + ((kb >> 2) - (kb0 >> 2)) * kScaleTile, &tmSW, &full[i], 0, kb >> 2, n0 >> 7);
    }
  }
  __syncwarp();

  // Q(x) for this CTA's blocks: 16 lanes take one row's block of 128. Row r of a block lies at
  // r * 128 with its 16-byte unit u at u ^ (r % 8); tokens past M are zero.
  // Four passes' loads are under way together.
  constexpr int kAhead = 4, kStep = kFThreads / 16;
  const int l = threadIdx.x & 15;
  for (int u0 = static_cast<int>(threadIdx.x) >> 4; u0 < nb * T; u0 += kAhead * kStep) {
    uint4 raw[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int u = u0 + j * kStep, i = u / T, r = u % T;
      const int c = (kb0 + i) * 128 + 8 * l;
      raw[j] = make_uint4(0, 0, 0, 0);
      if (i < nb && r < p.M) {
        const __nv_bfloat16* src = p.x + static_cast<int64_t>(r) * p.ldx + c;
        if (p.xvec && c + 8 <= p.K) {
          raw[j] = *reinterpret_cast<const uint4*>(src);
        } else {
          uint32_t w[4] = {};
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (c + e < p.K)
              w[e / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(src)[e]) << (16 * (e & 1));
          raw[j] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int u = u0 + j * kStep, i = u / T, r = u % T, kb = kb0 + i;
      if (i >= nb) break;  // the same for all lanes: a pass covers whole multiples of 16 rows
      float f[8];
      Elem<__nv_bfloat16>::unpack(raw[j], f);
      uint32_t a = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        a = max(a, finite_abs_bits(f[e]));
        f[e] = inf_to_nan(f[e]);
      }
#pragma unroll
      for (int o = 8; o; o >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
      const uint32_t byte = e8m0_byte(a);
      const float inv = e8m0_inverse(byte);
      uint2 q;
      q.x = e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
      q.y = e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv);
      *reinterpret_cast<uint2*>(sB + (i * T + r) * 128 + (((l >> 1) ^ (r & 7)) << 4) + (l & 1) * 8) = q;
      if (l == 0)
        sSB[((kb >> 2) - (kb0 >> 2)) * kScaleTile + (r & 31) * 16 + (kb & 3)] = static_cast<uint8_t>(byte);
    }
  }
  fence_proxy_async_smem();
  __syncthreads();

  if (warp == 0) {
    const uint32_t ts = tmem + 32u;  // A's scale columns, then B's
    for (int i = 0; i < nb; ++i) {
      if (!warp_wait(&full[i], 0u, wc, false)) continue;  // every copy is waited for, abort or not
      tc_fence_after_sync();
      if (elect_one()) {
        const int kb = kb0 + i, tile = (kb >> 2) - (kb0 >> 2);
        const uint32_t sa = ts + 4u * tile, sb = ts + 4u * kFMaxTiles + 4u * tile;
        if (i == 0 || (kb & 3) == 0) {
          tmem_cp_scales(sa, scale_tile_desc(smem_u32(sSA + tile * kScaleTile)));
          tmem_cp_scales(sb, scale_tile_desc(smem_u32(sSB + tile * kScaleTile)));
        }
        const uint64_t ad = sw128_kmajor_desc(smem_u32(sA + i * kFABytes));
        const uint64_t bd = sw128_kmajor_desc(smem_u32(sB + i * T * 128));
        const uint32_t id = idesc_mx_byte(idesc_mx_e4m3(128, T), static_cast<uint32_t>(kb & 3));
#pragma unroll
        for (int k = 0; k < 4; ++k)
          umma_mx(tmem, ad + 2u * k, bd + 2u * k, id, sa, sb, (i | k) != 0 ? 1u : 0u);
      }
      __syncwarp();
    }
    if (elect_one()) umma_commit(done);
    __syncwarp();
  }
  if (warp < 4) {  // accumulators: lane = weight row, columns = tokens
    warp_wait(done, 0u, wc, false);
    tc_fence_after_sync();
    uint32_t r[32];
    tmem_ld32_async(tmem + (static_cast<uint32_t>(warp * 32) << 16), r);
    tmem_wait_ld();
    reg_fence(r);
#pragma unroll
    for (int t = 0; t < T; ++t)
      sD[t * 128 + warp * 32 + lane] = nb > 0 ? __uint_as_float(r[t]) : 0.f;
    // Tensor memory goes back before this CTA waits for its cluster. A CTA pair of another stream
    // may hold all of it on one SM and wait for these columns on another (the bf16 product's
    // 64-column tiles leave room beside them), while this CTA's partner waits for it there:
    // what is held may not wait.
    tc_fence_before_sync();
    asm volatile("bar.sync 1, 128;" ::: "memory");
    if (warp == 0) {
      tc_fence_after_sync();
      tmem_dealloc(tmem, kFTmemCols);
    }
  }
  if (p.split > 1)
    cluster_sync();
  else
    __syncthreads();

  // each CTA of the cluster finishes its share of the outputs
  const int total = p.M * 128;
  for (int i = static_cast<int>(rank) * kFThreads + threadIdx.x; i < total; i += p.split * kFThreads) {
    const int t = i >> 7, n = n0 + (i & 127);
    float v = 0.f;
    if (p.split > 1) {
      const uint32_t mine = smem_u32(sD + i);
      for (int s = 0; s < p.split; ++s) v += ld_cluster_f32(mapa_shared(mine, s));
    } else {
      v = sD[i];
    }
    if (n < p.N) {
      if (p.bias != nullptr) v += __bfloat162float(p.bias[n]);
      if (p.gelu) v = f2unpack(gelu2_logit(f2pack(v, v))).x;
      if (p.resid != nullptr) v += __bfloat162float(p.resid[static_cast<int64_t>(t) * p.ldr + n]);
      p.out[static_cast<int64_t>(t) * p.ldo + n] = __float2bfloat16_rn(v);
    }
  }
  if (p.split > 1) cluster_sync();  // the others have read this CTA's sums
}

template <int T>
static int go(const Fp8Few& p, const CUtensorMap& tW, const CUtensorMap& tS, int n_tiles, cudaStream_t s) {
  auto kern = fp8_few_kernel<T>;
  const int smem = f_smem(T, p.blocks);
  static std::atomic<uint64_t> allowed{0};
  if (allow_smem(kern, f_smem(T, kFMaxBlocks), allowed) != cudaSuccess ||
      launch_cluster(kern, dim3(n_tiles * p.split), dim3(kFThreads), smem, s, false, p.split, tW, tS,
                     p) != cudaSuccess) {
    cudaGetLastError();
    return RS_ERR_CUDA;
  }
  return RS_OK;
}

// To 16 rows always; to 32 while the weight's row tiles leave SMs to the split, since every
// CTA quantises all the rows of its part of x (32 rows, two launches against one, us: 8192 x 2048
// 10.6 / 11.0, 16384 x 2048 14.6 / 20.8, 1024 x 4096 14.7 / 7.9).
bool fp8_few_rows(int M, int N, int K) {
  return (M <= 16 || (M <= 32 && N <= 8192)) && K <= 8 * kFMaxBlocks * 128;
}

int launch_fp8_few(Fp8Few p, int num_sms, cudaStream_t s) {
  const int KB = (p.K + 127) / 128, n_tiles = (p.N + 127) / 128;
  // CTAs per reduction: enough for 4 blocks each, 85 KB, of which two share an SM and one loads
  // while the other finishes (8192 x 2048 against 8 blocks each, one CTA on an SM, 8.0 -> 7.0 us),
  // doubled while all of them fit the SMs
  int split = 1;
  while (split < 8 && split * 4 < KB) split *= 2;
  while (split < 8 && 2 * split <= KB && static_cast<int64_t>(n_tiles) * 2 * split <= num_sms) split *= 2;
  p.split = split;
  p.blocks = (KB + split - 1) / split;
  CUtensorMap tW, tS;
  int st = tmap_operand(&tW, p.w, p.K, p.N, p.ldw, 128);
  if (st == RS_OK) st = tmap_scales(&tS, p.sw, p.N, p.K, 1);
  if (st != RS_OK) return st;
  return p.M <= 16 ? go<16>(p, tW, tS, n_tiles, s) : go<32>(p, tW, tS, n_tiles, s);
}

}  // namespace rs
