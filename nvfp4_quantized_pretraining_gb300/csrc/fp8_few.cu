// Y = X W^T for a few tokens (at most 16), the FP8 linear layer of generation: every weight is read for a handful of
// rows, so the call is bound by the weights' bytes and, below some ten megabytes, by latency.  One launch: a CTA takes
// 16 R rows of W, its 8 warps a share of K each; a warp quantizes the tokens' block of 128 itself, in registers, in the
// layout of the MMA's operand (no second kernel, no shared-memory staging, no scales in memory), multiplies with
// mma.sync m16n8k32 (E4M3, FP32 accumulation; at this width the tensor pipe is idle anyway) and applies the two
// power-of-two scales per block of 128.  Shares are added in shared memory in a fixed order, and Y is rounded once.
//
// K is permuted the same way in both operands so that a lane's 16 bytes of a row are 16 consecutive codes: of 64
// elements of K, lane q of a quad holds k = 16 q .. 16 q + 15, words 0 and 1 for one MMA, 2 and 3 for the next.
#include <cuda_bf16.h>

#include "common.cuh"
#include "fp8.cuh"
#include "kernels.h"
#include "scale_layout.cuh"

namespace nvfp4 {
namespace few {

constexpr int kWarps = 8, kThreads = kWarps * 32;

struct Args {
  const __nv_bfloat16* x;
  int64_t ldx;
  const uint8_t* w;
  const uint8_t* w_scales;
  __nv_bfloat16* y;
  int64_t ldy, pitch;
  uint32_t T, N, K;
};

__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 16 BF16 values from p, zeros from element `left` on.
template <bool WIDE>
__device__ __forceinline__ void load16(uint32_t (&v)[8], const __nv_bfloat16* p, int left) {
  if (WIDE && left >= 16) {
    const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = 0;
      if (2 * i < left) v[i] = reinterpret_cast<const uint16_t*>(p)[2 * i];
      if (2 * i + 1 < left) v[i] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[2 * i + 1] << 16;
    }
  }
}
__device__ __forceinline__ uint32_t codes4(uint32_t w0, uint32_t w1, float inv) {
  const float2 f = make_float2(inv, inv);
  const float2 a = __fmul2_rn(make_float2(bf16_lo(w0), bf16_hi(w0)), f), b = __fmul2_rn(make_float2(bf16_lo(w1), bf16_hi(w1)), f);
  uint32_t r;
  asm("{\n .reg .b16 lo, hi;\n cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n"
      " mov.b32 %0, {lo, hi};\n}\n"
      : "=r"(r)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ bool odd_half(uint32_t h) { return (h & 0x7FFFu) >= 0x7F80u; }

template <int NT, int R, bool WIDE>
__global__ void __launch_bounds__(kThreads) few_kernel(const Args a) {
  __shared__ float s_sum[kWarps][NT * 8][R * 16 + 1];
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
  const uint32_t n0 = blockIdx.x * (16 * R), KB = (a.K + 127) / 128, atoms = (KB + 3) / 4;
  float sum[R][NT][4];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[r][t][i] = 0.0f;
  const uint8_t* rows[2 * R];
  uint32_t row[2 * R];
#pragma unroll
  for (int i = 0; i < 2 * R; ++i) {
    row[i] = min(n0 + i * 8 + g, a.N - 1);  // (a row past the tensor: the last one again, its results are not stored)
    rows[i] = a.w + (size_t)row[i] * a.pitch + q * 16;
  }
  pdl_wait();
  for (uint32_t kb = warp; kb < KB; kb += kWarps) {
    uint4 w[2 * R][2];
    uint32_t ws[2 * R];
#pragma unroll
    for (int i = 0; i < 2 * R; ++i) {
      w[i][0] = *reinterpret_cast<const uint4*>(rows[i] + kb * 128);
      w[i][1] = *reinterpret_cast<const uint4*>(rows[i] + kb * 128 + 64);
      ws[i] = a.w_scales[sf_offset(row[i], kb, atoms)];
    }
    // the tokens' block: lane holds token 8 t + g's elements 16 q.. and 64 + 16 q..
    uint32_t x[NT][2][8];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t k = kb * 128 + h * 64 + q * 16, token = t * 8 + g;
        load16<WIDE>(x[t][h], a.x + (int64_t)token * a.ldx + k, token < a.T ? (int)a.K - (int)k : 0);
      }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      uint32_t m = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 8; ++i) m = __vmaxu2(m, x[t][h][i] & 0x7FFF7FFFu);
      uint32_t most = max(m & 0xFFFFu, m >> 16);
      most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
      most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
      const bool odd = __any_sync(0xFFFFFFFFu, most >= 0x7F80u);
      if (odd) {  // Inf or NaN in some token's block: they take no part in the scale
        most = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t lo = x[t][h][i] & 0x7FFFu, hi = x[t][h][i] >> 16 & 0x7FFFu;
            most = max(most, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
          }
        most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
        most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
      }
      const uint32_t byte = fp8_scale_byte(most << 16, kTopE4M3);
      const float inv = fp8_scale_inverse(byte);
      uint32_t b[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t w0 = x[t][h][2 * i], w1 = x[t][h][2 * i + 1];
          b[h][i] = codes4(w0, w1, inv);
          if (odd) {
            if (odd_half(w0)) b[h][i] |= 0x0000007Fu;
            if (odd_half(w0 >> 16)) b[h][i] |= 0x00007F00u;
            if (odd_half(w1)) b[h][i] |= 0x007F0000u;
            if (odd_half(w1 >> 16)) b[h][i] |= 0x7F000000u;
          }
        }
      // the scales of the two tokens whose results this lane holds
      const float sx = fp8_scale_value(byte);
      const float s0 = __shfl_sync(0xFFFFFFFFu, sx, q * 8), s1 = __shfl_sync(0xFFFFFFFFu, sx, q * 8 + 4);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 &lo = w[2 * r][h], &hi = w[2 * r + 1][h];
          mma_e4m3(c, lo.x, hi.x, lo.y, hi.y, b[h][0], b[h][1]);
          mma_e4m3(c, lo.z, hi.z, lo.w, hi.w, b[h][2], b[h][3]);
        }
        // (each product of two scales by itself could leave FP32's range where the result does not)
        const float wl = fp8_scale_value(ws[2 * r]), wh = fp8_scale_value(ws[2 * r + 1]);
        sum[r][t][0] += c[0] * wl * s0;
        sum[r][t][1] += c[1] * wl * s1;
        sum[r][t][2] += c[2] * wh * s0;
        sum[r][t][3] += c[3] * wh * s1;
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      s_sum[warp][t * 8 + 2 * q][r * 16 + g] = sum[r][t][0];
      s_sum[warp][t * 8 + 2 * q + 1][r * 16 + g] = sum[r][t][1];
      s_sum[warp][t * 8 + 2 * q][r * 16 + 8 + g] = sum[r][t][2];
      s_sum[warp][t * 8 + 2 * q + 1][r * 16 + 8 + g] = sum[r][t][3];
    }
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < NT * 8 * R * 16; i += kThreads) {
    const uint32_t token = i / (R * 16), in = i % (R * 16);
    if (token >= a.T || n0 + in >= a.N) continue;
    float v = s_sum[0][token][in];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) v += s_sum[w][token][in];
    a.y[(int64_t)token * a.ldy + n0 + in] = __float2bfloat16_rn(v);
  }
}

template <int NT, int R>
static cudaError_t launch(const Args& a, bool wide, cudaStream_t s) {
  const dim3 grid((a.N + 16 * R - 1) / (16 * R));
  const cudaError_t e = wide ? launch_pdl(few_kernel<NT, R, true>, grid, dim3(kThreads), 0, s, a)
                             : launch_pdl(few_kernel<NT, R, false>, grid, dim3(kThreads), 0, s, a);
  count_launch();
  return e;
}
template <int NT>
static cudaError_t launch_rows(const Args& a, bool wide, int num_sms, cudaStream_t s) {
  // 32 rows a CTA halve the work on the tokens; 16 where 32 would leave SMs without a CTA
  return a.N >= 32 * (uint32_t)num_sms ? launch<NT, 2>(a, wide, s) : launch<NT, 1>(a, wide, s);
}

}  // namespace few

cudaError_t launch_fp8_few(const void* x, int64_t T, int64_t K, int64_t ldx, const void* w_codes, const void* w_scales,
                           int64_t N, void* y, int64_t ldy, int num_sms, cudaStream_t s) {
  const few::Args a{static_cast<const __nv_bfloat16*>(x), ldx, static_cast<const uint8_t*>(w_codes),
                    static_cast<const uint8_t*>(w_scales), static_cast<__nv_bfloat16*>(y), ldy, fp8_pitch(K),
                    static_cast<uint32_t>(T), static_cast<uint32_t>(N), static_cast<uint32_t>(K)};
  const bool wide = (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && (ldx % 8 == 0 || T == 1);
  return T <= 8 ? few::launch_rows<1>(a, wide, num_sms, s) : few::launch_rows<2>(a, wide, num_sms, s);
}

}  // namespace nvfp4
