// BF16 to blocks of 128 E4M3 codes with one power-of-two scale, along rows, along columns (stored
// transposed), or both from one read; or one scale per 128 x 128 block, shared by both forms (so that the
// transposed weights are exactly the weights).
//
// A CTA takes a 128 x 128 tile.  Row form: 16 lanes hold a row's 128 elements, its amax is four shuffles of
// packed BF16 magnitudes, each lane converts its 8.  Column form: the tile goes through shared memory, a thread
// takes two adjacent columns and 32 rows (so shared reads are whole words without conflicts) and writes 2 x 32
// consecutive codes.  Memory-bound: 2 bytes read, 1 written per form and element.
#include <cuda_bf16.h>

#include "common.cuh"
#include "fp8.cuh"
#include "kernels.h"
#include "scale_layout.cuh"

namespace nvfp4 {
namespace fq {

constexpr int kThreads = 256;
constexpr uint32_t kAbs = 0x7FFF7FFFu;

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }
// |BF16| patterns with those that are not finite as 0.
__device__ __forceinline__ uint32_t finite_only(uint32_t w) {
  w &= kAbs;
  if ((w & 0xFFFFu) >= 0x7F80u) w &= 0xFFFF0000u;
  if ((w >> 16) >= 0x7F80u) w &= 0x0000FFFFu;
  return w;
}
// Two BF16 values to two codes (low element in the low byte): exact product, round to nearest even.  The largest
// finite magnitude of the block lands at most on 448; what is not finite becomes NaN (0x7F).
__device__ __forceinline__ uint32_t codes2(uint32_t w, float inv) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
      : "=h"(r)
      : "f"(__fmul_rn(bf16_hi(w), inv)), "f"(__fmul_rn(bf16_lo(w), inv)));
  uint32_t c = r;
  if ((w & 0x7FFFu) >= 0x7F80u) c |= 0x007Fu;
  if ((w >> 16 & 0x7FFFu) >= 0x7F80u) c |= 0x7F00u;
  return c;
}

__device__ __forceinline__ uint32_t larger_half(uint32_t m) { return max(m & 0xFFFFu, m >> 16); }

template <bool ROW, bool COL, bool SQUARE>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const __nv_bfloat16* x, uint32_t rows, uint32_t cols,
                                                            int64_t ld, bool wide, Fp8Out r, Fp8Out c) {
  __shared__ uint4 s_tile[COL ? 128 * 16 : 1];  // [128 rows][16 x 8 elements]
  __shared__ uint32_t s_max[COL && !SQUARE ? 4 * 64 : 8];
  pdl_trigger();
  pdl_wait();
  const uint32_t kb = blockIdx.x, rb = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t col0 = kb * 128 + (lane & 15) * 8;

  // the tile: pass i has rows 16 i + 2 warp + lane / 16; elements outside the tensor are zeros
  uint4 q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t row = rb * 128 + i * 16 + warp * 2 + (lane >> 4);
    q[i] = make_uint4(0, 0, 0, 0);
    if (row < rows) {
      const __nv_bfloat16* p = x + row * ld + col0;
      if (wide && col0 + 8 <= cols) {
        q[i] = *reinterpret_cast<const uint4*>(p);
      } else {
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (col0 + j < cols) w[j >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[j] << (16 * (j & 1));
        q[i] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    if (COL) s_tile[(i * 16 + warp * 2 + (lane >> 4)) * 16 + (lane & 15)] = q[i];
  }
  auto largest = [](const uint4& v) {
    return max_u16x2(max_u16x2(v.x & kAbs, v.y & kAbs), max_u16x2(v.z & kAbs, v.w & kAbs));
  };
  auto largest_finite = [](const uint4& v) {
    return max_u16x2(max_u16x2(finite_only(v.x), finite_only(v.y)), max_u16x2(finite_only(v.z), finite_only(v.w)));
  };
  uint32_t square = 0;  // SQUARE: the tile's scale byte
  if (SQUARE) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max_u16x2(m, largest_finite(q[i]));
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) m = max_u16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    if (lane == 0) s_max[warp] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max_u16x2(m, s_max[i]);
    square = fp8_scale_byte(larger_half(m) << 16, kTopE4M3);
  }
  const uint32_t row_atoms = (r.cols + 511) / 512, col_atoms = (c.cols + 511) / 512;
  if (ROW) {
    uint8_t* codes = static_cast<uint8_t*>(r.codes);
    uint8_t* scales = static_cast<uint8_t*>(r.scales);
    const bool last = kb == gridDim.x - 1;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t row = rb * 128 + i * 16 + warp * 2 + (lane >> 4);
      uint32_t byte = square;
      if (!SQUARE) {
        uint32_t m = largest(q[i]);
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) m = max_u16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        if (__any_sync(0xFFFFFFFFu, larger_half(m) >= 0x7F80u)) {
          m = largest_finite(q[i]);
#pragma unroll
          for (int o = 1; o < 16; o <<= 1) m = max_u16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        }
        byte = fp8_scale_byte(larger_half(m) << 16, kTopE4M3);
      }
      const float inv = fp8_scale_inverse(byte);
      if (row < rows) {
        const uint2 o = make_uint2(codes2(q[i].x, inv) | codes2(q[i].y, inv) << 16,
                                   codes2(q[i].z, inv) | codes2(q[i].w, inv) << 16);
        *reinterpret_cast<uint2*>(codes + (size_t)row * r.pitch + col0) = o;
      }
      // the scale, and zeros after the last block of the row's atom; rows past the tensor have scale 0
      if ((lane & 15) == 0) scales[sf_offset(row, kb, row_atoms)] = static_cast<uint8_t>(row < rows ? byte : 0);
      else if (last && (lane & 15) < 4 && (kb & 3) + (lane & 15) < 4)
        scales[sf_offset(row, kb + (lane & 15), row_atoms)] = 0;
    }
  }
  if (COL) {
    if (!SQUARE) __syncthreads();  // (SQUARE: the tile was complete before its amax)
    const uint32_t* words = reinterpret_cast<const uint32_t*>(s_tile);  // [128][64] column pairs
    const uint32_t pair = tid & 63, group = tid >> 6;
    uint32_t w[32], b0 = square, b1 = square;
#pragma unroll
    for (int i = 0; i < 32; ++i) w[i] = words[(group * 32 + i) * 64 + pair];
    if (!SQUARE) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 32; ++i) m = max_u16x2(m, w[i] & kAbs);
      if ((m & 0xFFFFu) >= 0x7F80u || (m >> 16) >= 0x7F80u) {
        m = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) m = max_u16x2(m, finite_only(w[i]));
      }
      s_max[group * 64 + pair] = m;
      __syncthreads();
      m = max_u16x2(max_u16x2(s_max[pair], s_max[64 + pair]), max_u16x2(s_max[128 + pair], s_max[192 + pair]));
      b0 = fp8_scale_byte(m << 16, kTopE4M3);
      b1 = fp8_scale_byte(m & 0xFFFF0000u, kTopE4M3);
    }
    const float i0 = fp8_scale_inverse(b0), i1 = fp8_scale_inverse(b1);
    uint32_t o0[8], o1[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o0[i] = o1[i] = 0;
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      // rows i, i + 1 of each column as one packed pair
      const uint32_t a = __byte_perm(w[i], w[i + 1], 0x5410), b = __byte_perm(w[i], w[i + 1], 0x7632);
      o0[i >> 2] |= codes2(a, i0) << (8 * (i & 2));
      o1[i >> 2] |= codes2(b, i1) << (8 * (i & 2));
    }
    uint8_t* codes = static_cast<uint8_t*>(c.codes);
    uint8_t* scales = static_cast<uint8_t*>(c.scales);
    const uint32_t col = kb * 128 + pair * 2;
    uint8_t* p = codes + (size_t)col * c.pitch + rb * 128 + group * 32;
    if (col < cols) {
      reinterpret_cast<uint4*>(p)[0] = make_uint4(o0[0], o0[1], o0[2], o0[3]);
      reinterpret_cast<uint4*>(p)[1] = make_uint4(o0[4], o0[5], o0[6], o0[7]);
    }
    if (col + 1 < cols) {
      p += c.pitch;
      reinterpret_cast<uint4*>(p)[0] = make_uint4(o1[0], o1[1], o1[2], o1[3]);
      reinterpret_cast<uint4*>(p)[1] = make_uint4(o1[4], o1[5], o1[6], o1[7]);
    }
    const bool last = rb == gridDim.y - 1;
    if (group == 0) {
      scales[sf_offset(col, rb, col_atoms)] = static_cast<uint8_t>(col < cols ? b0 : 0);
      scales[sf_offset(col + 1, rb, col_atoms)] = static_cast<uint8_t>(col + 1 < cols ? b1 : 0);
    } else if (last && (rb & 3) + group < 4) {
      scales[sf_offset(col, rb + group, col_atoms)] = 0;
      scales[sf_offset(col + 1, rb + group, col_atoms)] = 0;
    }
  }
}

}  // namespace fq

cudaError_t launch_fp8_quantize(const void* x, int64_t rows, int64_t cols, int64_t ld, bool square, const Fp8Out* row,
                                const Fp8Out* col, cudaStream_t s) {
  const dim3 grid(static_cast<uint32_t>((cols + 127) / 128), static_cast<uint32_t>((rows + 127) / 128));
  const bool wide = (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && (ld % 8 == 0 || rows == 1);
  const Fp8Out none{};
  const Fp8Out r = row ? *row : none, c = col ? *col : none;
  const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(x);
  const uint32_t R = static_cast<uint32_t>(rows), C = static_cast<uint32_t>(cols);
  auto go = [&](auto kernel) { return launch_pdl(kernel, grid, dim3(fq::kThreads), 0, s, p, R, C, ld, wide, r, c); };
  cudaError_t e;
  if (square)
    e = row && col ? go(fq::quantize_kernel<true, true, true>)
                   : row ? go(fq::quantize_kernel<true, false, true>) : go(fq::quantize_kernel<false, true, true>);
  else
    e = row && col ? go(fq::quantize_kernel<true, true, false>)
                   : row ? go(fq::quantize_kernel<true, false, false>) : go(fq::quantize_kernel<false, true, false>);
  count_launch();
  return e;
}

}  // namespace nvfp4
