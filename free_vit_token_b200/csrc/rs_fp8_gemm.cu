// rs_fp8_gemm.cu -- the product of two operands held in 8-bit blocks (rs_fp8.cuh),
//
//   D[m, n] = sum_j 2^(ea[m, j] + eb[n, j]) sum_{k in block j} qa[m, k] qb[n, k],
//
// then out = act(D + bias) + resid, stored as bf16, fp32 or again as 8-bit blocks along n.
//
// tcgen05 kind::mxf8f6f4: the E8M0 scales multiply inside the matrix instruction, so the fp32
// accumulator stays in TMEM over the whole reduction. The instruction takes a scale per 32 K
// elements; a block of 128 names the same byte four times. Scale tiles (128 rows x 4 blocks,
// 512 bytes) come with every fourth K block by TMA and go to TMEM by tcgen05.cp, ordered
// before the MMAs that read them; two sets of TMEM columns take turns.
//
// One persistent CTA per SM (or a CTA pair with 256-row tiles) loops over 128 x BN tiles:
//   warps 0-15 epilogue: a tile's accumulator goes to registers at once (up to 64 columns a
//              thread) and is handed back, then bias, activation, residual and rounding, and
//              out through per-warp TMA-store boxes
//   warp 16    TMA producer, warp 17 TMEM owner and MMA issuer
// At 8 bits a tile's products take half the time they take in bf16 while its epilogue stays the
// same: sixteen epilogue warps, not eight, keep up with reductions down to K = 384
// (50432 x 384 -> 1536 with GELU and its quantiser: 126 us with eight, 106 with sixteen, as both
// stood then).
//
// Measured, back to back: 8192^3 420 us (2.6 PFLOP/s; 300 us with the operand loads left out, and
// 511 us sustained, where the power cap holds the clock near 1.06 GHz), 25104 x 4096 -> 1024
// 88 us, 25104 x 1024 -> 4096 107 us, with GELU and 8-bit output 121 us (on cool caches 116).
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "rs_fp8.cuh"
#include "rs_gelu8.cuh"
#include "rs_ops.h"
#include "rs_ptx_mx.cuh"

namespace rs {

namespace {

constexpr int kGM = 128;                       // rows of A per CTA and tile
constexpr int kGK = 128;                       // K elements (bytes) per stage
constexpr int kGABytes = kGM * kGK;            // 16 KB
constexpr int kGEpiWarps = 16;
constexpr int kGProducer = kGEpiWarps, kGIssuer = kGEpiWarps + 1;  // warps
constexpr int kGThreads = (kGEpiWarps + 2) * 32;
constexpr int kGSmemLimit = 232448;
constexpr int kGCtrl = 512;
constexpr int kGBoxBytes = 32 * 64;            // 32 rows of 64 bytes, 64-byte swizzle
constexpr int kGEpiBytes = kGEpiWarps * (kGBoxBytes + 128 + 512);  // boxes, biases, maxima

__host__ __device__ constexpr int g_scale_tiles_b(int bn) { return bn > 128 ? 2 : 1; }
__host__ __device__ constexpr int g_stage_bytes(int bn, bool pair) {
  return kGABytes + (pair ? bn / 2 : bn) * kGK + (1 + g_scale_tiles_b(bn)) * kScaleTile;
}
constexpr int kGFixed = 1024 + kGCtrl + kGEpiBytes;
__host__ __device__ constexpr int g_stages(int bn, bool pair) {
  return (kGSmemLimit - kGFixed) / g_stage_bytes(bn, pair);
}
__host__ __device__ constexpr size_t g_smem(int bn, bool pair) {
  return static_cast<size_t>(kGFixed) + g_stages(bn, pair) * g_stage_bytes(bn, pair);
}

}  // namespace

template <int BN, bool PAIR, int OUT>
__global__ void __launch_bounds__(kGThreads, 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmSA,
                    const __grid_constant__ CUtensorMap tmSB,
                    const __grid_constant__ CUtensorMap tmOut, const Fp8Gemm p) {
  constexpr int kBRows = PAIR ? BN / 2 : BN;
  constexpr int kBBytes = kBRows * kGK;
  constexpr int kSTiles = g_scale_tiles_b(BN);
  constexpr int kSBytes = (1 + kSTiles) * kScaleTile;
  constexpr int STAGES = g_stages(BN, PAIR);
  constexpr int kTileM = PAIR ? 2 * kGM : kGM;
  constexpr uint32_t kIdesc = idesc_mx_e4m3(kTileM, BN);
  constexpr uint32_t kTx = (PAIR ? 2 : 1) * (kGABytes + kBBytes);
  constexpr uint32_t kTxScales = (PAIR ? 2 : 1) * kSBytes;
  constexpr int NACC = 2 * BN + 32 <= 512 ? 2 : 1;  // accumulators that fit beside the scales
  constexpr uint32_t kScaleCol = NACC * BN;         // two sets of 4 (A) + 8 (B) columns
  constexpr int kCols = BN / 4;                     // columns of one epilogue warp
  static_assert(STAGES >= 3, "pipeline depth");
  static_assert(kCols == 32 || kCols == 64, "epilogue columns");
  static_assert(BN % kQBlock == 0, "a tile's columns start with a scale tile of B");

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sA = smem;
  uint8_t* sB = sA + STAGES * kGABytes;
  uint8_t* sBox = sB + STAGES * kBBytes;
  uint8_t* sBias = sBox + kGEpiWarps * kGBoxBytes;      // [warp][64] bf16
  volatile uint64_t* sMax =                              // [2][warp][32] (turn, magnitude)
      reinterpret_cast<volatile uint64_t*>(sBias + kGEpiWarps * 128);
  uint8_t* sS = sBox + kGEpiBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(sS + STAGES * kSBytes);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int KB = (p.K + kGK - 1) / kGK;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
  const bool leader = rank == 0;
  const int unit0 = PAIR ? static_cast<int>(blockIdx.x >> 1) : static_cast<int>(blockIdx.x);
  const int units = PAIR ? static_cast<int>(gridDim.x >> 1) : static_cast<int>(gridDim.x);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], PAIR ? 2 * kGEpiWarps : kGEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kGProducer && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmSA);
    tma_prefetch_desc(&tmSB);
    if (!p.direct) tma_prefetch_desc(&tmOut);
  }
  if (warp == kGIssuer) {
    if constexpr (PAIR) {
      tmem_alloc_pair(tmem_slot, 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, 512);
      tmem_relinquish();
    }
  }
  if (OUT == kOutQ8 && warp < kGEpiWarps) {
    sMax[warp * 32 + lane] = 0;
    sMax[(kGEpiWarps + warp) * 32 + lane] = 0;
  }
  pdl_trigger();
  pdl_wait();
  tc_fence_before_sync();
  if constexpr (PAIR) {
    cluster_sync();
  } else {
    __syncthreads();
  }
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  const WaitCtl wc{abort_flag, p.err, p.timeout_ns};

  if (warp == kGProducer) {
    // ------------------------------------------------------------ TMA producer
    int stage = 0;
    uint32_t phase = 0;
    uint32_t pend_mask = 0, pend_phase = 0;
    const uint32_t full_leader = PAIR ? mapa_shared(smem_u32(&full[0]), 0u) : 0u;
    for (int tile = unit0; tile < p.num_tiles; tile += units) {
      const int m_blk = tile / p.n_blocks, n_blk = tile % p.n_blocks;
      const int a_row = m_blk * kTileM + static_cast<int>(rank) * kGM;
      const int n0 = n_blk * BN;
      const int b_row = n0 + static_cast<int>(rank) * kBRows;
      // test hook: leave one stage unfilled so the consumer's wait runs out
      const int skip_kb = (blockIdx.x == 0 && tile == unit0) ? p.debug_skip_kb : -1;
      bool ok = true;
      for (int kb = 0; kb < KB; ++kb) {
        if (!warp_wait(&empty[stage], phase ^ 1u, wc)) { ok = false; break; }
        if (kb != skip_kb && elect_one()) {
          const bool scales = (kb & 3) == 0;
          if (leader) mbar_arrive_expect_tx(&full[stage], scales ? kTx + kTxScales : kTx);
          uint8_t* dA = sA + stage * kGABytes;
          uint8_t* dB = sB + stage * kBBytes;
          uint8_t* dS = sS + stage * kSBytes;
          // the A scales of this CTA's rows; B's of every column of the tile (both CTAs of a
          // pair need them all). Tiles past the operand's rows read as zero.
          if constexpr (PAIR) {
            const uint32_t fb = full_leader + static_cast<uint32_t>(stage) * 8u;
            tma_load_2d_pair(dA, &tmA, fb, kb * kGK, a_row);
            tma_load_2d_pair(dB, &tmB, fb, kb * kGK, b_row);
            if (scales) {
              tma_load_3d_pair(dS, &tmSA, fb, 0, kb >> 2, a_row >> 7);
              tma_load_3d_pair(dS + kScaleTile, &tmSB, fb, 0, kb >> 2, n0 >> 7);
            }
          } else {
            tma_load_2d(dA, &tmA, &full[stage], kb * kGK, a_row);
            tma_load_2d(dB, &tmB, &full[stage], kb * kGK, b_row);
            if (scales) {
              tma_load_3d(dS, &tmSA, &full[stage], 0, kb >> 2, a_row >> 7);
              tma_load_3d(dS + kScaleTile, &tmSB, &full[stage], 0, kb >> 2, n0 >> 7);
            }
          }
        }
        __syncwarp();
        if (kb != skip_kb) {
          const uint32_t bit = 1u << stage;
          pend_mask |= bit;
          pend_phase = (pend_phase & ~bit) | (phase << stage);
        }
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
      }
      if (!ok) break;
    }
    // every copy must land before the CTA may exit (a pair's land on the leader's barriers)
    if (leader) {
#pragma unroll
      for (int s = 0; s < STAGES; ++s)
        if (pend_mask & (1u << s)) warp_wait(&full[s], (pend_phase >> s) & 1u, wc, false);
    }
    if constexpr (PAIR) {
      // and the leader's releases of every stage must have arrived here
      for (int i = 0; i < STAGES; ++i) {
        if (!warp_wait(&empty[stage], phase ^ 1u, wc)) break;
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
      }
    }
  } else if (warp == kGIssuer) {
    // ------------------------------------------------------------ MMA issuer
    if (leader) {
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      uint32_t set = 0;  // scale columns in use
      uint32_t ts = 0;
      bool issued = false;
      const uint64_t ad0 = sw128_kmajor_desc(smem_u32(sA));
      const uint64_t bd0 = sw128_kmajor_desc(smem_u32(sB));
      const uint64_t sd0 = scale_tile_desc(smem_u32(sS));
      for (int tile = unit0; tile < p.num_tiles; tile += units) {
        if (!warp_wait(&tempty[acc], acc_phase ^ 1u, wc, true, PAIR)) break;
        tc_fence_after_sync();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
        bool ok = true;
        for (int kb = 0; kb < KB; ++kb) {
          if (!warp_wait(&full[stage], phase, wc)) { ok = false; break; }
          tc_fence_after_sync();
          if ((kb & 3) == 0) {
            ts = tmem_base + kScaleCol + set * 16u;
            set ^= 1u;
          }
          const uint32_t id = idesc_mx_byte(kIdesc, static_cast<uint32_t>(kb & 3));
          const uint64_t ad = ad0 + static_cast<uint64_t>(stage * (kGABytes >> 4));
          const uint64_t bd = bd0 + static_cast<uint64_t>(stage * (kBBytes >> 4));
          const int steps = (p.K - kb * kGK + 31) / 32;  // whole 32-wide steps past K hold zeros
          if (elect_one()) {
            if ((kb & 3) == 0) {
              const uint64_t sd = sd0 + static_cast<uint64_t>(stage * (kSBytes >> 4));
#pragma unroll
              for (int i = 0; i < 1 + kSTiles; ++i) {
                if constexpr (PAIR)
                  tmem_cp_scales_pair(ts + 4u * i, sd + static_cast<uint64_t>(i * (kScaleTile >> 4)));
                else
                  tmem_cp_scales(ts + 4u * i, sd + static_cast<uint64_t>(i * (kScaleTile >> 4)));
              }
            }
#pragma unroll
            for (int k = 0; k < kGK / 32; ++k) {
              if (k == 0 || k < steps) {
                if constexpr (PAIR)
                  umma_mx_pair(d_tmem, ad + 2u * k, bd + 2u * k, id, ts, ts + 4u, (kb | k) != 0 ? 1u : 0u);
                else
                  umma_mx(d_tmem, ad + 2u * k, bd + 2u * k, id, ts, ts + 4u, (kb | k) != 0 ? 1u : 0u);
              }
            }
            if constexpr (PAIR)
              umma_commit_pair_mc(&empty[stage], 0x3);
            else
              umma_commit(&empty[stage]);
          }
          __syncwarp();
          issued = true;
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        if (elect_one()) {
          if constexpr (PAIR)
            umma_commit_pair_mc(&tfull[acc], 0x3);
          else
            umma_commit(&tfull[acc]);
        }
        __syncwarp();
        if (++acc == NACC) { acc = 0; acc_phase ^= 1u; }
      }
      if (__any_sync(0xffffffffu, *abort_flag != 0) && issued) {
        if (elect_one()) {
          if constexpr (PAIR)
            umma_commit_pair(drain);
          else
            umma_commit(drain);
        }
        __syncwarp();
        warp_wait(drain, 0u, wc, false);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3, grp = warp >> 2;
    uint8_t* box = sBox + warp * kGBoxBytes;
    const uint32_t box_u32 = smem_u32(box), bias_u32 = smem_u32(sBias + warp * 128);
    constexpr int ES = OUT == kOutQ8 ? 1 : OUT == kOutBf16 ? 2 : 4;  // bytes of an output element
    constexpr int BC = 64 / ES < kCols ? 64 / ES : kCols;            // columns of a box
    constexpr int NB = kCols / BC;                                   // boxes of a tile
    int acc = 0;
    uint32_t acc_phase = 0;
    uint32_t turn = 0;  // 8-bit output: tiles whose maxima this warp has exchanged
    for (int tile = unit0; tile < p.num_tiles; tile += units) {
      const int m_blk = tile / p.n_blocks, n_blk = tile % p.n_blocks;
      const int row0 = m_blk * kTileM + static_cast<int>(rank) * kGM + q * 32;
      const int col0 = n_blk * BN + grp * kCols;
      if (p.bias != nullptr && 2 * lane < kCols) {  // this warp's biases, while the tile runs
        const int c = col0 + 2 * lane;
        uint32_t b = 0;
        if (c + 1 < p.N) b = __ldg(reinterpret_cast<const uint32_t*>(p.bias + c));
        else if (c < p.N) b = __ldg(reinterpret_cast<const uint16_t*>(p.bias + c));
        reinterpret_cast<uint32_t*>(sBias + warp * 128)[lane] = b;
      }
      int ok = 1;
      if (lane == 0) ok = wait_bounded(&tfull[acc], acc_phase, wc) ? 1 : 0;
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      mbar_try_wait(&tfull[acc], acc_phase);  // completed: acquire for every lane
      tc_fence_after_sync();
      const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                             static_cast<uint32_t>(acc * BN + grp * kCols);
      uint32_t r[kCols / 32][32];
#pragma unroll
      for (int i = 0; i < kCols / 32; ++i) tmem_ld32_async(t_row + 32u * i, r[i]);
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < kCols / 32; ++i) reg_fence(r[i]);
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        if (PAIR && !leader)
          mbar_arrive_cluster(mapa_shared(smem_u32(&tempty[acc]), 0u));
        else
          mbar_arrive(&tempty[acc]);
      }
      if (++acc == NACC) { acc = 0; acc_phase ^= 1u; }
      const int row = row0 + lane;
      // does the warp (for 8-bit blocks, any warp of its block of 128) hold part of the output?
      if (row0 >= p.M || (OUT == kOutQ8 ? col0 & ~(kQBlock - 1) : col0) >= p.N) continue;

#pragma unroll
      for (int i = 0; i < kCols / 32; ++i) {
        if (p.bias != nullptr) {
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const uint4 b4 = lds128(bias_u32 + i * 64 + v * 16);
            const uint32_t bw[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t& lo = r[i][8 * v + 2 * e];
              uint32_t& hi = r[i][8 * v + 2 * e + 1];
              const float2 z = f2unpack(
                  fadd2((static_cast<uint64_t>(hi) << 32) | lo, bf16x2_to_f2(bw[e])));
              lo = __float_as_uint(z.x);
              hi = __float_as_uint(z.y);
            }
          }
        }
        if (p.gelu) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              uint32_t& lo = r[i][16 * h + 2 * e];
              uint32_t& hi = r[i][16 * h + 2 * e + 1];
              const uint64_t g = gelu2_logit((static_cast<uint64_t>(hi) << 32) | lo);
              lo = static_cast<uint32_t>(g);
              hi = static_cast<uint32_t>(g >> 32);
            }
          }
        }
      }

      float inv = 0.f;
      if constexpr (OUT == kOutQ8) {
        // A block of a row is shared by the same lane of 128 / kCols warps, which exchange its
        // largest magnitude; columns past N hold no value.
        constexpr int S = kQBlock / kCols;
        if (col0 + kCols > p.N) {
#pragma unroll
          for (int i = 0; i < kCols / 32; ++i)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (col0 + 32 * i + e >= p.N) r[i][e] = 0;
        }
        float am[2] = {0.f, 0.f};  // two chains; NaN does not enter a maximum
#pragma unroll
        for (int i = 0; i < kCols / 32; ++i)
#pragma unroll
          for (int e = 0; e < 32; ++e) am[e & 1] = fmaxf(am[e & 1], fabsf(__uint_as_float(r[i][e])));
        uint32_t a = __float_as_uint(fmaxf(am[0], am[1]));
        if (a >= kInfBits) {
          a = 0;
#pragma unroll
          for (int i = 0; i < kCols / 32; ++i)
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float f = __uint_as_float(r[i][e]);
              a = max(a, finite_abs_bits(f));
              r[i][e] = __float_as_uint(inf_to_nan(f));
            }
        }
        // Each lane publishes its magnitude with the tile's turn and polls its partners' (as
        // bounded as every wait here, which a named barrier is not). Two slots by turns: a
        // warp writes one again only after its partners have read it, since it needs their
        // magnitudes of the turn between.
        ++turn;
        volatile uint64_t* mx = sMax + (turn & 1u) * kGEpiWarps * 32;
        mx[warp * 32 + lane] = (static_cast<uint64_t>(turn) << 32) | a;
#pragma unroll
        for (int k = 1; k < S; ++k) {
          const int other = q + 4 * (grp / S * S + (grp + k) % S);
          uint64_t v = mx[other * 32 + lane], t0 = 0;
          for (uint32_t i = 1; static_cast<uint32_t>(v >> 32) != turn; ++i) {
            if ((i & 255u) == 0) {
              if (t0 == 0) t0 = global_timer_ns();
              if (*abort_flag) break;
              if (global_timer_ns() - t0 > p.timeout_ns) {
                *abort_flag = 1;
                atomicCAS(p.err, 0, static_cast<int>(RS_ERR_DEVICE_TIMEOUT));
                break;
              }
            }
            v = mx[other * 32 + lane];
          }
          a = max(a, static_cast<uint32_t>(v));
        }
        __syncwarp();
        const uint32_t byte = e8m0_byte(a);
        inv = e8m0_inverse(byte);
        if (row < p.M && grp % S == 0)
          p.out_scales[scale_offset(row, col0 >> 7, p.kqo)] = static_cast<uint8_t>(byte);
      }

#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int c = col0 + b * BC;
        if (c >= p.N) break;
        uint32_t w[BC * ES / 4];  // this row of the box
        if constexpr (OUT == kOutQ8) {
#pragma unroll
          for (int e = 0; e < BC / 4; ++e) {
            const int k = b * BC + 4 * e;
            w[e] = e4m3x4(__uint_as_float(r[k / 32][k % 32]) * inv,
                          __uint_as_float(r[k / 32][k % 32 + 1]) * inv,
                          __uint_as_float(r[k / 32][k % 32 + 2]) * inv,
                          __uint_as_float(r[k / 32][k % 32 + 3]) * inv);
          }
        } else {
          float f[BC];
#pragma unroll
          for (int e = 0; e < BC; ++e) {
            const int k = b * BC + e;
            f[e] = __uint_as_float(r[k / 32][k % 32]);
          }
          if (p.resid != nullptr && row < p.M) {
            const uint8_t* rr = static_cast<const uint8_t*>(p.resid) +
                                (static_cast<int64_t>(row) * p.ldr + c) * ES;
            if (p.rvec && c + BC <= p.N) {
#pragma unroll
              for (int v = 0; v < 4; ++v) {
                const uint4 x4 = *(reinterpret_cast<const uint4*>(rr) + v);
                const uint32_t xw[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  if constexpr (OUT == kOutBf16) {
                    f[8 * v + 2 * e] += bf16lo(xw[e]);
                    f[8 * v + 2 * e + 1] += bf16hi(xw[e]);
                  } else {
                    f[4 * v + e] += __uint_as_float(xw[e]);
                  }
                }
              }
            } else {
#pragma unroll
              for (int e = 0; e < BC; ++e)
                if (c + e < p.N) {
                  if constexpr (OUT == kOutBf16)
                    f[e] += __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(rr)[e]);
                  else
                    f[e] += reinterpret_cast<const float*>(rr)[e];
                }
            }
          }
#pragma unroll
          for (int e = 0; e < BC * ES / 4; ++e) {
            if constexpr (OUT == kOutBf16)
              w[e] = pack_bf16x2(f[2 * e], f[2 * e + 1]);
            else
              w[e] = __float_as_uint(f[e]);
          }
        }
        // the store that last used this box has read it
        if (lane == 0) bulk_wait_group_read0();
        __syncwarp();
        // 64-byte rows in the 64-byte swizzle (32-byte rows, 8-bit blocks of narrow tiles, in
        // the 32-byte one)
        constexpr int U = BC * ES / 16;  // 16-byte units of a row
        const uint32_t sw = U == 4 ? (lane >> 1) & 3 : (lane >> 2) & 1;
#pragma unroll
        for (int u = 0; u < U; ++u)
          sts128(box_u32 + lane * (16 * U) + ((u ^ sw) << 4),
                 make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]));
        // TMA stores whole 16-byte units: where the last columns end inside one, they and rows
        // that TMA cannot address (a pitch or base off 16 bytes) go by plain stores,
        // neighbouring lanes writing neighbouring elements
        if (!p.direct && (c + BC <= p.N || OUT == kOutQ8 || p.N * ES % 16 == 0)) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&tmOut, box, c, row0);
            bulk_commit_group();
          }
        } else if constexpr (OUT != kOutQ8) {
          __syncwarp();
#pragma unroll 4
          for (int it = 0; it < BC; ++it) {
            const int idx = it * 32 + lane, rr = idx / BC, cc = idx % BC;
            const uint8_t* src = box + rr * 64 + ((((cc * ES) >> 4) ^ ((rr >> 1) & 3)) << 4) + ((cc * ES) & 15);
            if (row0 + rr < p.M && c + cc < p.N) {
              uint8_t* dst = static_cast<uint8_t*>(p.out) +
                             (static_cast<int64_t>(row0 + rr) * p.ldo + c + cc) * ES;
              if constexpr (ES == 2)
                *reinterpret_cast<uint16_t*>(dst) = *reinterpret_cast<const uint16_t*>(src);
              else
                *reinterpret_cast<uint32_t*>(dst) = *reinterpret_cast<const uint32_t*>(src);
            }
          }
          __syncwarp();
        }
      }
    }
    if (lane == 0) bulk_wait_group0();
    __syncwarp();
  }

  __syncthreads();
  if constexpr (PAIR) {
    // as in the bf16 GEMM: after an abort, time for the other CTA's loads to land; neither CTA
    // leaves or frees TMEM before the other is done
    if (threadIdx.x == 0 && (*abort_flag || *reinterpret_cast<volatile int*>(p.err) != 0))
      spin_ns(1000000);
    cluster_sync();
  }
  if (warp == kGIssuer) {
    tc_fence_after_sync();
    if constexpr (PAIR)
      tmem_dealloc_pair(tmem_base, 512);
    else
      tmem_dealloc(tmem_base, 512);
  }
}

// ------------------------------------------------------------------ host
namespace {

int tmap_2d(CUtensorMap* m, CUtensorMapDataType t, int es, const void* base, uint64_t inner,
            uint64_t rows, uint64_t pitch, uint32_t box_inner, uint32_t box_rows,
            CUtensorMapSwizzle sw) {
  auto fn = encode_fn();
  if (fn == nullptr) return RS_ERR_CUDA;
  cuuint64_t dims[2] = {inner, rows};
  cuuint64_t strides[1] = {pitch * es};
  cuuint32_t box[2] = {box_inner, box_rows};
  cuuint32_t one[2] = {1, 1};
  return fn(m, t, 2, const_cast<void*>(base), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? RS_OK
             : RS_ERR_CUDA;
}

}  // namespace

int tmap_operand(CUtensorMap* m, const void* base, int K, int rows, int64_t ld, int box_rows) {
  return tmap_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, base, K, rows, ld, kGK, box_rows,
                 CU_TENSOR_MAP_SWIZZLE_128B);
}

// Scale tiles as [row tiles][tiles along K][128 words].
int tmap_scales(CUtensorMap* m, const void* base, int rows, int K, uint32_t tiles) {
  auto fn = encode_fn();
  if (fn == nullptr) return RS_ERR_CUDA;
  const cuuint64_t kq = (K + 511) / 512, rt = (rows + 127) / 128;
  cuuint64_t dims[3] = {128, kq, rt};
  cuuint64_t strides[2] = {kScaleTile, kScaleTile * kq};
  cuuint32_t box[3] = {128, 1, tiles};
  cuuint32_t one[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<void*>(base), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? RS_OK
             : RS_ERR_CUDA;
}

namespace {

template <int BN, bool PAIR, int OUT>
int go(Fp8Gemm p, int num_sms, cudaStream_t s, bool pdl) {
  constexpr int tile_m = PAIR ? 256 : 128;
  p.n_blocks = (p.N + BN - 1) / BN;
  p.num_tiles = ((p.M + tile_m - 1) / tile_m) * p.n_blocks;
  CUtensorMap tA, tB, tSA, tSB, tO{};
  const auto u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  int st = tmap_operand(&tA, p.a, p.K, p.M, p.lda, kGM);
  if (st == RS_OK) st = tmap_operand(&tB, p.b, p.K, p.N, p.ldb, PAIR ? BN / 2 : BN);
  if (st == RS_OK) st = tmap_scales(&tSA, p.sa, p.M, p.K, 1);
  if (st == RS_OK) st = tmap_scales(&tSB, p.sb, p.N, p.K, g_scale_tiles_b(BN));
  constexpr int es = OUT == kOutQ8 ? 1 : OUT == kOutBf16 ? 2 : 4;
  constexpr int box = 64 / es < BN / 4 ? 64 / es : BN / 4;  // the epilogue's boxes
  if (st == RS_OK && !p.direct)
    st = tmap_2d(&tO, OUT == kOutQ8     ? u8
                      : OUT == kOutBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                        : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                 es, p.out, p.N, p.M, p.ldo, box, 32,
                 box * es == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B);
  if (st != RS_OK) return st;
  auto kern = fp8_gemm_kernel<BN, PAIR, OUT>;
  constexpr size_t smem = g_smem(BN, PAIR);
  static std::atomic<uint64_t> allowed{0};
  if (allow_smem(kern, static_cast<int>(smem), allowed) != cudaSuccess) {
    cudaGetLastError();
    return RS_ERR_CUDA;
  }
  cudaError_t e;
  if constexpr (PAIR) {
    static std::atomic<int> resident[64];  // pairs at once, by device
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
      cudaGetLastError();
      return RS_ERR_CUDA;
    }
    int max_pairs = resident[dev & 63].load(std::memory_order_relaxed);
    if (max_pairs == 0) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(2 * (num_sms / 2));
      cfg.blockDim = dim3(kGThreads);
      cfg.dynamicSmemBytes = smem;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = 2;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&max_pairs, kern, &cfg) != cudaSuccess || max_pairs <= 0) {
        cudaGetLastError();
        max_pairs = num_sms / 2;
      }
      max_pairs = max_pairs < num_sms / 2 ? max_pairs : num_sms / 2;
      resident[dev & 63].store(max_pairs, std::memory_order_relaxed);
    }
    const int pairs = p.num_tiles < max_pairs ? p.num_tiles : max_pairs;
    e = launch_cluster(kern, dim3(2 * pairs), dim3(kGThreads), smem, s, pdl, 2, tA, tB, tSA, tSB, tO,
                       p);
  } else {
    const int grid = p.num_tiles < num_sms ? p.num_tiles : num_sms;
    e = launch(kern, dim3(grid), dim3(kGThreads), smem, s, pdl, tA, tB, tSA, tSB, tO, p);
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return RS_ERR_CUDA;
  }
  return RS_OK;
}

// Tiles of 128 x 128 while one wave of them covers the output: more SMs share a small product
// and each epilogue is short. Else 256 columns, by single CTAs while the reduction is short (a
// pair's accumulator goes back and forth between two SMs once a tile) and by CTA pairs on 256
// rows past that (a third less operand traffic). Measured 16384 x 4096, single / pair, us: plain
// K = 512 42 / 49, K = 768 61 / 55; GELU K = 768 68 / 74, K = 1024 77 / 80, K = 1536 102 / 97.
template <int OUT>
int pick(const Fp8Gemm& p, int num_sms, cudaStream_t s, bool pdl) {
  const int64_t small = (static_cast<int64_t>(p.M) + 127) / 128 * ((static_cast<int64_t>(p.N) + 127) / 128);
  if (small <= num_sms || p.M <= 128) return go<128, false, OUT>(p, num_sms, s, pdl);
  const bool pair = p.K > (p.gelu ? 1024 : 512);
  if (p.N <= 128) return pair ? go<128, true, OUT>(p, num_sms, s, pdl) : go<128, false, OUT>(p, num_sms, s, pdl);
  return pair ? go<256, true, OUT>(p, num_sms, s, pdl) : go<256, false, OUT>(p, num_sms, s, pdl);
}

}  // namespace

int launch_fp8_gemm(const Fp8Gemm& p, int out, int num_sms, cudaStream_t s, bool pdl) {
  switch (out) {
    case kOutBf16: return pick<kOutBf16>(p, num_sms, s, pdl);
    case kOutFp32: return pick<kOutFp32>(p, num_sms, s, pdl);
    default: return pick<kOutQ8>(p, num_sms, s, pdl);
  }
}

}  // namespace rs
