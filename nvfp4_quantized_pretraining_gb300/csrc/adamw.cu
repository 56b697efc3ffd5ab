// AdamW over many tensors in one launch, moments in FP32 or in 8 bits (E4M3 for the first, E5M2 for
// the second, one power-of-two scale per 128 elements).
//
// Per element, each line one FP32 operation per operator (no contraction), so that a step is
// reproducible to the bit:
//   g = grad * grad_scale                      (without one: grad)
//   m = b1 m + (1 - b1) g        v = b2 v + (1 - b2) (g g)
//   p = p (1 - lr wd) - size (m / (sqrt(v) root + eps)),
//   size = lr / (1 - b1^t), root = 1 / sqrt(1 - b2^t)   (computed in FP64 on the host)
// and with 8-bit states m and v are rounded after p has used them unrounded.
//
// The step is bound by memory: 30 bytes per element with FP32 states, FP32 gradients and a BF16 copy;
// 16 with 8-bit states and BF16 gradients.  A thread owns 8 consecutive elements, so a block of 128 is
// 16 lanes and its amax four shuffles; every stream moves in 8- or 16-byte accesses.
#include <cuda_bf16.h>

#include "common.cuh"
#include "fp8.cuh"
#include "kernels.h"
#include "sr.cuh"

namespace nvfp4 {
namespace aw {

constexpr int kThreads = 256;
constexpr int kChunk = kThreads * 8;  // elements of one CTA step: 16 whole blocks of 128
// Tensors of one launch: the table travels in the kernel's parameters (no device copy to keep in
// step with the caller's pointers).  Two capacities, so that a short list stays a small launch.
constexpr int kCapSmall = 48, kCapLarge = 400;

struct Scalars {
  float b1, c1, b2, c2, size, root, eps;
  uint32_t step, first_tensor, count, chunks;
  const float* grad_scale;
  PhiloxKeys keys;
};
template <int CAP>
struct Table {
  AdamWEntry t[CAP];
  uint32_t first_chunk[CAP + 1];
};

__device__ __forceinline__ void load8(float (&x)[8], const float* p) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Eight values of a block of 128 (16 lanes) to codes: amax over the finite ones, the block's scale,
// then code = top bits of the FP32 pattern of a * 2^-e * 2^(least normal exponent + 126).  That product
// lines the 8-bit format's exponent field up with FP32's, subnormals included (FP32's own subnormals
// take over there), so rounding is one integer addition below bit SHIFT: a random 16-bit fraction
// (stochastic) or the nearest-even increment.  A value that is not finite becomes NAN_CODE and takes
// no part in the scale.  FLOOR: a positive value never becomes 0 (a second moment of zero would turn
// its element's next update into m / eps).
template <int TOP, int SHIFT, uint32_t NAN_CODE, bool FLOOR, bool SR>
__device__ __forceinline__ uint2 encode8(const float (&a)[8], const uint4& rnd, uint32_t& byte) {
  uint32_t mx = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = __float_as_uint(a[i]) & 0x7FFFFFFFu;
    mx = max(mx, b < 0x7F800000u ? b : 0u);
  }
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
  byte = fp8_scale_byte(mx, TOP);
  const float inv = fp8_scale_inverse(byte);
  const float line = SHIFT == 20 ? 0x1p-120f : 0x1p-112f;
  const uint32_t w[4] = {rnd.x, rnd.y, rnd.z, rnd.w};
  uint32_t out[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t bits = __float_as_uint(__fmul_rn(__fmul_rn(a[i], inv), line));
    const uint32_t size = bits & 0x7FFFFFFFu;
    uint32_t add;
    if (SR) add = ((i & 1) ? w[i >> 1] >> 16 : w[i >> 1] & 0xFFFFu) << (SHIFT - 16);
    else add = (1u << (SHIFT - 1)) - 1u + ((size >> SHIFT) & 1u);
    uint32_t code = (size + add) >> SHIFT;
    if (FLOOR && code == 0 && a[i] > 0.0f) code = 1;
    if ((__float_as_uint(a[i]) & 0x7FFFFFFFu) >= 0x7F800000u) code = NAN_CODE;
    code |= (bits >> 24) & 0x80u;
    out[i >> 2] |= code << (8 * (i & 3));
  }
  return make_uint2(out[0], out[1]);
}

template <bool GBF16, bool BITS8, bool SR, int CAP>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ Table<CAP> tab,
                                                         const __grid_constant__ Scalars k) {
  const float gs = k.grad_scale ? *k.grad_scale : 1.0f;
  if (!(fabsf(gs) <= 3.402823466e38f)) return;  // the caller's signal that this step is not to be taken
  // this CTA's consecutive chunks, and the tensor of the first one
  const uint32_t c0 = static_cast<uint32_t>((uint64_t)k.chunks * blockIdx.x / gridDim.x);
  const uint32_t c1 = static_cast<uint32_t>((uint64_t)k.chunks * (blockIdx.x + 1) / gridDim.x);
  uint32_t lo = 0, hi = k.count;  // first_chunk[lo] <= c0 < first_chunk[hi]
  while (hi - lo > 1) {
    const uint32_t mid = (lo + hi) >> 1;
    if (tab.first_chunk[mid] <= c0) lo = mid;
    else hi = mid;
  }
  for (uint32_t c = c0; c < c1; ++c) {
    while (tab.first_chunk[lo + 1] <= c) ++lo;
    const AdamWEntry& t = tab.t[lo];
    const int64_t e0 = (int64_t)(c - tab.first_chunk[lo]) * kChunk + threadIdx.x * 8;
    const int64_t left = t.numel - e0;
    const bool whole = left >= 8 && t.vector;
    float p[8], g[8], m[8], v[8];
    uint32_t mb = 0, vb = 0;
    if (whole) {
      load8(p, t.param + e0);
      if (GBF16) {
        const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(t.grad) + e0);
        g[0] = bf16_lo(q.x), g[1] = bf16_hi(q.x), g[2] = bf16_lo(q.y), g[3] = bf16_hi(q.y);
        g[4] = bf16_lo(q.z), g[5] = bf16_hi(q.z), g[6] = bf16_lo(q.w), g[7] = bf16_hi(q.w);
      } else {
        load8(g, static_cast<const float*>(t.grad) + e0);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool in = i < left;
        p[i] = in ? t.param[e0 + i] : 0.0f;
        if (GBF16) g[i] = in ? __bfloat162float(static_cast<const __nv_bfloat16*>(t.grad)[e0 + i]) : 0.0f;
        else g[i] = in ? static_cast<const float*>(t.grad)[e0 + i] : 0.0f;
      }
    }
    if (BITS8) {
      uint2 mc = make_uint2(0, 0), vc = make_uint2(0, 0);
      const uint8_t* mp = static_cast<const uint8_t*>(t.m) + e0;
      const uint8_t* vp = static_cast<const uint8_t*>(t.v) + e0;
      if (whole) {
        mc = *reinterpret_cast<const uint2*>(mp);
        vc = *reinterpret_cast<const uint2*>(vp);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < left) {
            (i < 4 ? mc.x : mc.y) |= (uint32_t)mp[i] << (8 * (i & 3));
            (i < 4 ? vc.x : vc.y) |= (uint32_t)vp[i] << (8 * (i & 3));
          }
      }
      if (left > 0) {
        mb = t.m_scale[e0 / kFp8Block];
        vb = t.v_scale[e0 / kFp8Block];
      }
      const float ms = fp8_scale_value(mb), vs = fp8_scale_value(vb);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 a = e4m3x2_to_f32((i < 2 ? mc.x : mc.y) >> (16 * (i & 1)));
        const float2 b = e5m2x2_to_f32((i < 2 ? vc.x : vc.y) >> (16 * (i & 1)));
        m[2 * i] = __fmul_rn(a.x, ms), m[2 * i + 1] = __fmul_rn(a.y, ms);
        v[2 * i] = __fmul_rn(b.x, vs), v[2 * i + 1] = __fmul_rn(b.y, vs);
      }
    } else if (whole) {
      load8(m, static_cast<const float*>(t.m) + e0);
      load8(v, static_cast<const float*>(t.v) + e0);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool in = i < left;
        m[i] = in ? static_cast<const float*>(t.m)[e0 + i] : 0.0f;
        v[i] = in ? static_cast<const float*>(t.v)[e0 + i] : 0.0f;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (k.grad_scale) g[i] = __fmul_rn(g[i], gs);
      m[i] = __fadd_rn(__fmul_rn(k.b1, m[i]), __fmul_rn(k.c1, g[i]));
      v[i] = __fadd_rn(__fmul_rn(k.b2, v[i]), __fmul_rn(k.c2, __fmul_rn(g[i], g[i])));
      const float d = __fadd_rn(__fmul_rn(__fsqrt_rn(v[i]), k.root), k.eps);
      p[i] = __fsub_rn(__fmul_rn(p[i], t.keep), __fmul_rn(k.size, __fdiv_rn(m[i], d)));
    }
    if (whole) {
      store8(t.param + e0, p);
      if (t.model)
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(t.model) + e0) = make_uint4(
            pack_bf16(p[0], p[1]), pack_bf16(p[2], p[3]), pack_bf16(p[4], p[5]), pack_bf16(p[6], p[7]));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) {
          t.param[e0 + i] = p[i];
          if (t.model) static_cast<__nv_bfloat16*>(t.model)[e0 + i] = __float2bfloat16_rn(p[i]);
        }
    }
    if (BITS8) {
      uint4 rm = make_uint4(0, 0, 0, 0), rv = rm;
      if (SR) {
        const uint64_t j = static_cast<uint64_t>(e0) >> 3;
        const uint32_t st = 2u * (k.first_tensor + lo);
        rm = philox4x32_10(make_uint4((uint32_t)j, (uint32_t)(j >> 32), st, k.step), k.keys);
        rv = philox4x32_10(make_uint4((uint32_t)j, (uint32_t)(j >> 32), st + 1u, k.step), k.keys);
      }
      if (left < 8) {  // a block's elements beyond the tensor count as zeros
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i >= left) m[i] = 0.0f, v[i] = 0.0f;
      }
      const uint2 mc = encode8<kTopE4M3, 20, 0x7Fu, false, SR>(m, rm, mb);
      const uint2 vc = encode8<kTopE5M2, 21, 0x7Fu, true, SR>(v, rv, vb);
      uint8_t* mp = static_cast<uint8_t*>(t.m) + e0;
      uint8_t* vp = static_cast<uint8_t*>(t.v) + e0;
      if (whole) {
        *reinterpret_cast<uint2*>(mp) = mc;
        *reinterpret_cast<uint2*>(vp) = vc;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < left) {
            mp[i] = static_cast<uint8_t>((i < 4 ? mc.x : mc.y) >> (8 * (i & 3)));
            vp[i] = static_cast<uint8_t>((i < 4 ? vc.x : vc.y) >> (8 * (i & 3)));
          }
      }
      if ((threadIdx.x & 15) == 0 && left > 0) {
        t.m_scale[e0 / kFp8Block] = static_cast<uint8_t>(mb);
        t.v_scale[e0 / kFp8Block] = static_cast<uint8_t>(vb);
      }
    } else if (whole) {
      store8(static_cast<float*>(t.m) + e0, m);
      store8(static_cast<float*>(t.v) + e0, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) {
          static_cast<float*>(t.m)[e0 + i] = m[i];
          static_cast<float*>(t.v)[e0 + i] = v[i];
        }
    }
  }
}

template <bool GBF16, bool BITS8, bool SR, int CAP>
static cudaError_t launch_table(const AdamWEntry* t, int n, Scalars k, int num_sms, cudaStream_t s) {
  Table<CAP> tab;
  uint32_t chunks = 0;
  for (int i = 0; i < n; ++i) {
    tab.t[i] = t[i];
    tab.first_chunk[i] = chunks;
    chunks += static_cast<uint32_t>((t[i].numel + kChunk - 1) / kChunk);
  }
  tab.first_chunk[n] = chunks;
  k.count = static_cast<uint32_t>(n);
  k.chunks = chunks;
  const uint32_t most = static_cast<uint32_t>(num_sms) * 32u;
  const uint32_t grid = chunks < most ? chunks : most;
  adamw_kernel<GBF16, BITS8, SR, CAP><<<grid, kThreads, 0, s>>>(tab, k);
  const cudaError_t e = cudaGetLastError();
  count_launch();
  return e;
}
template <bool GBF16, bool BITS8, bool SR>
static cudaError_t launch_some(const AdamWEntry* t, int n, const Scalars& k, int num_sms, cudaStream_t s) {
  return n <= kCapSmall ? launch_table<GBF16, BITS8, SR, kCapSmall>(t, n, k, num_sms, s)
                        : launch_table<GBF16, BITS8, SR, kCapLarge>(t, n, k, num_sms, s);
}

}  // namespace aw

int adamw_capacity() { return aw::kCapLarge; }

cudaError_t launch_adamw(const AdamWEntry* t, int n, int first_tensor, bool grad_bf16, int bits, bool sr,
                         const AdamWScalars& a, int num_sms, cudaStream_t s) {
  aw::Scalars k{};
  k.b1 = a.b1, k.c1 = a.c1, k.b2 = a.b2, k.c2 = a.c2;
  k.size = a.size, k.root = a.root, k.eps = a.eps;
  k.step = a.step;
  k.first_tensor = static_cast<uint32_t>(first_tensor);
  k.grad_scale = a.grad_scale;
  k.keys = philox_keys(a.seed);
  if (bits == 32)
    return grad_bf16 ? aw::launch_some<true, false, false>(t, n, k, num_sms, s)
                     : aw::launch_some<false, false, false>(t, n, k, num_sms, s);
  if (sr)
    return grad_bf16 ? aw::launch_some<true, true, true>(t, n, k, num_sms, s)
                     : aw::launch_some<false, true, true>(t, n, k, num_sms, s);
  return grad_bf16 ? aw::launch_some<true, true, false>(t, n, k, num_sms, s)
                   : aw::launch_some<false, true, false>(t, n, k, num_sms, s);
}

}  // namespace nvfp4
