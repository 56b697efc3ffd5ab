// C = A B^T for E4M3 operands with one power-of-two scale per 128 elements of K (sm_103a, tcgen05).
//
// The tensor core applies the scales itself: tcgen05.mma kind::mxf8f6f4.block_scale multiplies by one UE8M0
// byte per row and 32 elements of K, chosen by an id inside a 32-bit word of tensor memory; the four MMAs of a
// 128-wide stage take the same byte, so a word serves 512 elements of K and a 128-row operand's scales for
// them are one 512-byte atom, moved to tensor memory by tcgen05.cp right before the MMAs that read it.
// Accumulation is FP32 over the whole K and C is rounded once.
//
// A cluster of two CTAs computes a 256 x 256 tile with two-SM MMAs: CTA r stages A rows [128 r, +128) and B rows
// [128 r, +128), receives C rows [128 r, +128); per SM 32 KB of operands feed 8.4 MFLOP per stage.  Warps: TMA
// producer, MMA issuer (pair leader), eight epilogue warps.  Operands past M, N or K are zeros (TMA fill, code
// padding), stores are clipped.  Every wait is bounded (FP4_ERR_TIMEOUT in the status word).
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"

namespace nvfp4 {
namespace f8 {

constexpr int BK = 128;
constexpr int STAGES = 5;
constexpr int A_BYTES = 128 * BK, B_BYTES = 128 * BK;  // this CTA's rows of each operand
constexpr int SF_ATOM = 512;                           // 128 rows x 4 scale bytes: 512 elements of K
constexpr int SF_BYTES = 3 * SF_ATOM;                  // this CTA's A rows, all 256 B rows
constexpr int STAGE_BYTES = A_BYTES + B_BYTES + 2048;  // (a stage starts on a 1024-byte boundary)
constexpr int EPI_WARPS = 8, FIRST_EPI_WARP = 2;
constexpr int CHUNK_BYTES = 32 * 64;                   // 32 rows x 32 BF16 columns, 64-byte swizzled rows
constexpr int OUT_BYTES = EPI_WARPS * 2 * CHUNK_BYTES;
constexpr int kSfGroup = 4;                            // stages per scale word
constexpr uint32_t TM_ACC = 0, TM_SF = 256, TM_SF_SLOT = 16, TM_COLS = 512;
constexpr int NUM_THREADS = (FIRST_EPI_WARP + EPI_WARPS) * 32;
constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + OUT_BYTES + 1024 + 256;
static_assert(STAGE_BYTES % 1024 == 0 && SMEM_BYTES <= 232448, "shared memory");

struct Params {
  uint32_t M, N, num_k, tiles_m, tiles_n;
  uint32_t n_fastest;  // tile order: the larger operand is walked slowest
  void* C;
  int64_t ldc;
  int c_f32, tma_store;
  uint32_t vec;        // C rows allow 16-byte stores
};

// kind::mxf8f6f4: E4M3 x E4M3, UE8M0 scales, K-major operands; the scale byte's id is added per stage.
__host__ __device__ constexpr uint32_t idesc_mxf8(uint32_t M, uint32_t N) {
  return ((N >> 3) << 17) | (1u << 23) | ((M >> 4) << 24);
}
__device__ __forceinline__ uint32_t idesc_sf(uint32_t id) { return (id << 4) | (id << 29); }

__device__ __forceinline__ void mma_mxf8_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                              uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
      " tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
// 512 bytes (32 x 16) of each CTA's shared memory to 4 columns of its tensor memory, in every lane quadrant.
__device__ __forceinline__ void tc_cp_sf_pair(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NUM_THREADS, 1)
    gemm_pair_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
                     const __grid_constant__ CUtensorMap tmap_sa, const __grid_constant__ CUtensorMap tmap_sb,
                     const __grid_constant__ CUtensorMap tmap_c, const Params p) {
  pdl_trigger();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_out = smem + STAGES * STAGE_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(s_out + OUT_BYTES);  // leader: both CTAs' copies landed
  uint64_t* empty = full + STAGES;                                  // each CTA: the MMAs have read the stage
  uint64_t* acc_full = empty + STAGES;                              // each CTA: accumulator complete
  uint64_t* acc_empty = acc_full + 1;                               // leader: both CTAs drained it
  uint64_t* done_bar = acc_empty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, 2 * EPI_WARPS);
    mbar_init(done_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmap_a);
    prefetch_tmap(&tmap_b);
    prefetch_tmap(&tmap_sa);
    prefetch_tmap(&tmap_sb);
    if (p.tma_store) prefetch_tmap(&tmap_c);
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, TM_COLS);
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();  // (the set-up above touches no global data)

  const uint32_t cluster_id = blockIdx.x >> 1, num_clusters = gridDim.x >> 1;
  const uint32_t num_tiles = p.tiles_m * p.tiles_n, num_k = p.num_k;
  auto tile_at = [&](uint32_t t, uint32_t& mb, uint32_t& nb) {
    mb = p.n_fastest ? t / p.tiles_n : t % p.tiles_m;
    nb = p.n_fastest ? t % p.tiles_n : t / p.tiles_m;
  };

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA producer (both CTAs; completion on the leader's barrier) ----------------
      const uint32_t full0 = mapa_shared(smem_u32(&full[0]), 0);
      uint32_t stage = 0, phase = 0;
      bool ok = true;
      for (uint32_t t = cluster_id; ok && t < num_tiles; t += num_clusters) {
        uint32_t mb, nb;
        tile_at(t, mb, nb);
        for (uint32_t it = 0; it < num_k; ++it) {
          if (!mbar_wait(&empty[stage], phase ^ 1)) {
            ok = false;
            break;
          }
          uint8_t* sA = smem + stage * STAGE_BYTES;
          uint8_t* sB = sA + A_BYTES;
          uint8_t* sS = sB + B_BYTES;
          const uint32_t full_l = full0 + stage * 8;
          const bool sf = it % kSfGroup == 0;
          if (leader) mbar_arrive_expect_tx(&full[stage], 2 * (A_BYTES + B_BYTES + (sf ? SF_BYTES : 0)));
          tma_load_2d_pair(sA, &tmap_a, full_l, (int32_t)(it * BK), (int32_t)(mb * 256 + rank * 128));
          tma_load_2d_pair(sB, &tmap_b, full_l, (int32_t)(it * BK), (int32_t)(nb * 256 + rank * 128));
          if (sf) {
            const int32_t x = (int32_t)(it / kSfGroup * 64);  // 8-byte units
            tma_load_2d_pair(sS, &tmap_sa, full_l, x, (int32_t)(mb * 2 + rank));
            tma_load_2d_pair(sS + SF_ATOM, &tmap_sb, full_l, x, (int32_t)(nb * 2));
          }
          if (++stage == STAGES) stage = 0, phase ^= 1;
        }
      }
      if (!ok) *abort_flag = 1;
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      // ---------------- MMA issuer ----------------
      const uint64_t adesc0 = smem_desc(smem_u32(smem), 16, 1024, kSwizzle128B);
      const uint64_t bdesc0 = adesc0 + (A_BYTES >> 4);
      const uint64_t sdesc0 = smem_desc(smem_u32(smem) + A_BYTES + B_BYTES, 0, 128, kSwizzleNone);
      constexpr uint64_t kStageD = STAGE_BYTES >> 4;
      uint32_t stage = 0, phase = 0, slot = 0, n = 0;
      bool ok = true;
      for (uint32_t t = cluster_id; ok && t < num_tiles; t += num_clusters, ++n) {
        if (*abort_flag || !mbar_wait(acc_empty, (n & 1) ^ 1)) { ok = false; break; }
        tc_fence_after();
        for (uint32_t it = 0; it < num_k; ++it) {
          if (!mbar_wait(&full[stage], phase)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (it % kSfGroup == 0) {
            slot ^= 1;
            const uint32_t sf = tmem + TM_SF + slot * TM_SF_SLOT;
            const uint64_t sd = sdesc0 + stage * kStageD;
            tc_cp_sf_pair(sf, sd);
            tc_cp_sf_pair(sf + 8, sd + (SF_ATOM >> 4));
            tc_cp_sf_pair(sf + 12, sd + (2 * SF_ATOM >> 4));
          }
          const uint32_t sfa = tmem + TM_SF + slot * TM_SF_SLOT, sfb = sfa + 8;
          const uint32_t idesc = idesc_mxf8(256, 256) | idesc_sf(it % kSfGroup);
          const uint64_t ad = adesc0 + stage * kStageD, bd = bdesc0 + stage * kStageD;
          mma_mxf8_pair(tmem + TM_ACC, ad, bd, idesc, sfa, sfb, it != 0);
          mma_mxf8_pair(tmem + TM_ACC, ad + 2, bd + 2, idesc, sfa, sfb, 1);
          mma_mxf8_pair(tmem + TM_ACC, ad + 4, bd + 4, idesc, sfa, sfb, 1);
          mma_mxf8_pair(tmem + TM_ACC, ad + 6, bd + 6, idesc, sfa, sfb, 1);
          tc_commit_pair_mc(&empty[stage], 3);
          if (++stage == STAGES) stage = 0, phase ^= 1;
        }
        if (!ok) break;
        tc_commit_pair_mc(acc_full, 3);
      }
      if (!ok) *abort_flag = 1;
      tc_commit_pair_mc(done_bar, 1);
      mbar_wait(done_bar, 0);
    }
  } else {
    // ---------------- epilogue (both CTAs) ----------------
    // warp w reads TMEM lane quadrant w % 4 (32 of this CTA's rows) and 128 columns, in four chunks of 32
    const uint32_t quad = warp & 3, h = (uint32_t)(warp - FIRST_EPI_WARP) >> 2;
    const uint32_t lane_off = (quad * 32) << 16;
    const uint32_t acc_empty0 = mapa_shared(smem_u32(acc_empty), 0);
    uint8_t* buf0 = s_out + (warp - FIRST_EPI_WARP) * 2 * CHUNK_BYTES;
    uint8_t* buf1 = buf0 + CHUNK_BYTES;
    const uint32_t tacc = tmem + lane_off + TM_ACC + h * 128;
    auto release = [&] {  // every TMEM read of this warp is complete
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (leader) mbar_arrive(acc_empty);
        else mbar_arrive_cluster_relaxed(acc_empty0);
      }
    };
    uint32_t n = 0;
    for (uint32_t t = cluster_id; t < num_tiles; t += num_clusters, ++n) {
      uint32_t mb, nb;
      tile_at(t, mb, nb);
      if (*abort_flag || !mbar_wait_warp(acc_full, n & 1)) {
        *abort_flag = 1;
        break;
      }
      tc_fence_after();
      const uint32_t row0 = mb * 256 + rank * 128 + quad * 32, col0 = nb * 256 + h * 128;
      if (p.tma_store) {
        auto convert = [&](const uint32_t (&a)[32], uint32_t (&pk)[16]) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(a[2 * e]), __uint_as_float(a[2 * e + 1]));
            pk[e] = *reinterpret_cast<const uint32_t*>(&b);
          }
        };
        // row = lane, 64 bytes; 16-byte unit u lands at u ^ ((row >> 1) & 3) (64-byte swizzle)
        auto stage_chunk = [&](uint8_t* chunk, const uint32_t (&pk)[16]) {
#pragma unroll
          for (int u = 0; u < 4; ++u)
            *reinterpret_cast<uint4*>(chunk + lane * 64 + ((u ^ ((lane >> 1) & 3)) << 4)) =
                make_uint4(pk[4 * u], pk[4 * u + 1], pk[4 * u + 2], pk[4 * u + 3]);
        };
        auto store = [&](const uint8_t* chunk, uint32_t col) {  // (clipped at the tensor's edges)
          if (col < p.N && row0 < p.M) tma_store_2d(&tmap_c, chunk, (int32_t)col, (int32_t)row0);
        };
        uint32_t ra[32], rb[32], pk[16], pk2[16], pk3[16];
        if (lane == 0) bulk_wait_read<0>();  // the previous tile's stores have read both buffers
        __syncwarp();
        tmem_ld_32x32b_x32(tacc, ra);
        tmem_ld_wait(ra);
        tmem_ld_32x32b_x32(tacc + 32, rb);
        convert(ra, pk);
        stage_chunk(buf0, pk);
        tmem_ld_wait(rb);
        tmem_ld_32x32b_x32(tacc + 64, ra);
        convert(rb, pk);
        stage_chunk(buf1, pk);
        tmem_ld_wait(ra);
        tmem_ld_32x32b_x32(tacc + 96, rb);
        convert(ra, pk2);
        tmem_ld_wait(rb);
        release();
        convert(rb, pk3);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          store(buf0, col0);
          store(buf1, col0 + 32);
          bulk_commit_group();
          bulk_wait_read<0>();
        }
        __syncwarp();
        stage_chunk(buf0, pk2);
        stage_chunk(buf1, pk3);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          store(buf0, col0 + 64);
          store(buf1, col0 + 96);
          bulk_commit_group();
        }
      } else {
        const uint32_t row = row0 + lane;
#pragma unroll 1
        for (int j = 0; j < 4; ++j) {
          uint32_t acc[32];
          tmem_ld_32x32b_x32(tacc + j * 32, acc);
          tmem_ld_wait(acc);
          const uint32_t col = col0 + j * 32;
          if (row < p.M && col < p.N) {
            if (p.c_f32) {
              float* dst = static_cast<float*>(p.C) + (size_t)row * p.ldc + col;
              if (p.vec && col + 32 <= p.N) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  reinterpret_cast<uint4*>(dst)[i] = make_uint4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
              } else {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (col + i < p.N) dst[i] = __uint_as_float(acc[i]);
              }
            } else {
              __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.C) + (size_t)row * p.ldc + col;
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (col + i < p.N) dst[i] = __float2bfloat16_rn(__uint_as_float(acc[i]));
            }
          }
        }
        release();
      }
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }

  __syncthreads();
  if (*abort_flag) {  // a wait expired: let copies still in flight land first
    if (threadIdx.x == 0) drain_pause();
    __syncthreads();
  }
  tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, TM_COLS);
  }
  cluster_sync();
}

}  // namespace f8

cudaError_t launch_fp8_gemm(const Fp8GemmArgs& g, int num_sms, cudaStream_t s) {
  using namespace f8;
  static cudaError_t attr =
      cudaFuncSetAttribute(gemm_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
  if (attr != cudaSuccess) return attr;
  const uint64_t pitch = fp8_pitch(g.K), atoms = (g.K + 511) / 512;
  CUtensorMap ta, tb, tsa, tsb, tc;
  const auto u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8, u64 = CU_TENSOR_MAP_DATA_TYPE_UINT64;
  if (!encode_tmap_2d(&ta, u8, g.a_codes, pitch, g.M, pitch, BK, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_tmap_2d(&tb, u8, g.b_codes, pitch, g.N, pitch, BK, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_tmap_2d(&tsa, u64, g.a_scales, atoms * 64, (g.M + 127) / 128, atoms * 512, 64, 1, CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !encode_tmap_2d(&tsb, u64, g.b_scales, atoms * 64, (g.N + 127) / 128, atoms * 512, 64, 2, CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorInvalidValue;
  Params p{};
  p.M = (uint32_t)g.M;
  p.N = (uint32_t)g.N;
  p.num_k = (uint32_t)(pitch / BK);
  p.tiles_m = (p.M + 255) / 256;
  p.tiles_n = (p.N + 255) / 256;
  p.n_fastest = g.M > g.N;
  p.C = g.C;
  p.ldc = g.ldc;
  p.c_f32 = g.c_f32;
  const bool aligned = (reinterpret_cast<uintptr_t>(g.C) & 15u) == 0 && (g.ldc * (g.c_f32 ? 4 : 2)) % 16 == 0;
  p.vec = aligned;
  p.tma_store = aligned && !g.c_f32;
  if (p.tma_store) {
    if (!encode_tmap_2d(&tc, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, g.C, g.N, g.M, (uint64_t)g.ldc * 2, 32, 32,
                CU_TENSOR_MAP_SWIZZLE_64B))
      return cudaErrorInvalidValue;
  } else {
    tc = ta;
  }
  const uint32_t tiles = p.tiles_m * p.tiles_n, pairs = (uint32_t)num_sms / 2;
  const uint32_t clusters = tiles < pairs ? tiles : pairs;
  const cudaError_t e =
      launch_pdl(gemm_pair_kernel, dim3(clusters * 2), dim3(NUM_THREADS), SMEM_BYTES, s, ta, tb, tsa, tsb, tc, p);
  count_launch();
  return e;
}

cudaError_t fp8_status_read_clear(unsigned int* out, cudaStream_t s) {
  cudaError_t e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return e;
  e = cudaMemcpyFromSymbol(out, g_status, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_status, &zero, sizeof(unsigned int));
}

}  // namespace nvfp4
