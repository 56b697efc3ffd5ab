// Log probabilities of given tokens over a vocabulary, with the distribution's entropy and its largest
// entries, and their gradient.
//
// Forward: one read of the logits.  Each thread keeps a running maximum m of its logits with
// S = sum 2^(x2) and E = sum 2^(x2) x2, x2 = (z - m) log2(e) / temperature; when the maximum grows by d,
// S <- S 2^-d and E <- (E - S d) 2^-d.  Threads, warps and the CTAs of a row's cluster are joined the same
// way in a fixed order; logprob = x_target - ln S, entropy = ln S - ln 2 E / S.
//
// Top k: a thread's maximum costs nothing extra.  The threads form 64 groups; the k-th largest group
// maximum tau is a lower bound of the k-th largest logit (k groups hold an element that large), so only
// threads whose maximum reaches tau are read again (from L2), and the elements >= tau, little more than
// k of them, are ranked by counting.  Ties that overflow the candidate list, and rows with NaN, take
// k rounds of a block-wide maximum instead.
//
// Both directions are bound by memory: 2 or 4 bytes per logit forward, twice that backward.
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"

namespace nvfp4 {
namespace lp {

constexpr int kMaxTop = 32;
constexpr int kGroups = 64;
constexpr int kCap = 1024;  // candidates ranked by counting
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// 2^x2 is 0 below this; a banned token's x2 = -inf would make 0 * inf of its entropy term
constexpr float kFloor = -16384.0f;

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// 16 bytes of logits as FP32 values; kNone fills a lane without elements.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static constexpr uint32_t kNone = 0xFF800000u;
  __device__ static __forceinline__ void unpack(const uint4& q, float (&f)[4]) {
    f[0] = __uint_as_float(q.x), f[1] = __uint_as_float(q.y), f[2] = __uint_as_float(q.z), f[3] = __uint_as_float(q.w);
  }
  __device__ static __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
  __device__ static __forceinline__ float largest(const uint4&, const float (&f)[4]) {
    return max_nan(max_nan(f[0], f[1]), max_nan(f[2], f[3]));
  }
  __device__ static __forceinline__ float load(const float* p) { return *p; }
  __device__ static __forceinline__ void store(float* p, float v) { *p = v; }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static constexpr uint32_t kNone = 0xFF80FF80u;
  __device__ static __forceinline__ void unpack(const uint4& q, float (&f)[8]) {
    f[0] = bf16_lo(q.x), f[1] = bf16_hi(q.x), f[2] = bf16_lo(q.y), f[3] = bf16_hi(q.y);
    f[4] = bf16_lo(q.z), f[5] = bf16_hi(q.z), f[6] = bf16_lo(q.w), f[7] = bf16_hi(q.w);
  }
  __device__ static __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  __device__ static __forceinline__ uint4 pack(const float (&f)[8]) {
    return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
  }
  __device__ static __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  __device__ static __forceinline__ float largest(const uint4& q, const float (&)[8]) {
    const uint32_t w = max2(max2(q.x, q.y), max2(q.z, q.w));
    return max_nan(bf16_lo(w), bf16_hi(w));
  }
  __device__ static __forceinline__ float load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  __device__ static __forceinline__ void store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
};

// The order of top k as an unsigned key: larger logits larger keys, -0 as +0, NaN above all.
__device__ __forceinline__ uint32_t order_key(float z) {
  const uint32_t b = __float_as_uint(__fadd_rn(z, 0.0f));
  if (z != z) return 0xFFFFFFFFu;
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  if (k == 0xFFFFFFFFu) return __uint_as_float(0x7FFFFFFFu);
  return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}
// key and index as one number: the larger key first, then the lower index
__device__ __forceinline__ uint64_t entry_of(uint32_t key, uint32_t idx) {
  return (static_cast<uint64_t>(key) << 32) | (0xFFFFFFFFu - idx);
}

struct Sum {
  float m, s, e;  // s = sum 2^x2, e = sum 2^x2 x2 relative to m; m = -inf: nothing yet
};
__device__ __forceinline__ Sum join(const Sum& a, const Sum& b, float k2) {
  Sum r;
  r.m = fmaxf(a.m, b.m);
  // (a side of nothing has s = e = 0; fmaxf also turns -inf - -inf into the floor)
  const float da = fmaxf((a.m - r.m) * k2, -1e30f), db = fmaxf((b.m - r.m) * k2, -1e30f);
  const float ca = ex2(da), cb = ex2(db);
  r.s = a.s * ca + b.s * cb;
  r.e = (a.e + a.s * da) * ca + (b.e + b.s * db) * cb;
  return r;
}

__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ float ld_cluster_f32(const void* p, uint32_t rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(mapa_shared(smem_u32(p), rank)) : "memory");
  return v;
}
__device__ __forceinline__ uint64_t ld_cluster_u64(const void* p, uint32_t rank) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(mapa_shared(smem_u32(p), rank)) : "memory");
  return v;
}

// A row cut at 16-byte boundaries: `head` elements, `vecs` aligned vectors, `tail` elements.
struct RowCut {
  uint32_t head, vecs, tail;
};
template <typename T>
__device__ __forceinline__ RowCut cut_row(const T* row, uint32_t V) {
  constexpr uint32_t N = Vec<T>::N;
  const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T);
  RowCut c;
  c.head = min((N - off) & (N - 1), V);
  c.vecs = (V - c.head) / N;
  c.tail = V - c.head - c.vecs * N;
  return c;
}

// One cluster of CTAs per row, each CTA a consecutive share of the row's vectors (rank 0 also the
// edge elements).
template <typename T, int THREADS, bool TOP>
__global__ void __launch_bounds__(THREADS) logprob_kernel(const LogprobArgs a) {
  using V8 = Vec<T>;
  constexpr int N = V8::N, WARPS = THREADS / 32;
  __shared__ Sum s_sum[WARPS];
  __shared__ Sum s_cta;
  __shared__ uint32_t s_group[TOP ? kGroups : 1];
  __shared__ uint64_t s_cand[TOP ? kCap : 1];
  __shared__ uint16_t s_list[TOP ? THREADS : 1];
  __shared__ uint64_t s_top[TOP ? kMaxTop : 1];
  __shared__ uint64_t s_best[TOP ? WARPS : 1];
  __shared__ uint32_t s_tau, s_count, s_listed;
  const uint32_t rank = cluster_ctarank(), C = cluster_size();
  const int64_t t = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const T* row = static_cast<const T*>(a.logits) + t * a.ld;
  const RowCut cut = cut_row(row, static_cast<uint32_t>(a.V));
  const uint4* vec = reinterpret_cast<const uint4*>(row + cut.head);
  const uint32_t v0 = static_cast<uint32_t>((uint64_t)cut.vecs * rank / C);
  const uint32_t v1 = static_cast<uint32_t>((uint64_t)cut.vecs * (rank + 1) / C);
  const float k2 = a.scale * kLog2e;
  const float neg_inf = __uint_as_float(0xFF800000u);

  float m = neg_inf;
  float2 s2 = make_float2(0.0f, 0.0f), e2 = make_float2(0.0f, 0.0f);
  auto grow = [&](float to) {  // the running maximum becomes `to`
    const float d = fmaxf((m - to) * k2, -1e30f), c = ex2(d);
    e2.x = (e2.x + s2.x * d) * c, e2.y = (e2.y + s2.y * d) * c;
    s2.x *= c, s2.y *= c;
    m = to;
  };
  auto add = [&](const uint4& q) {
    float f[N];
    V8::unpack(q, f);
    const float top = V8::largest(q, f);
    if (top == neg_inf) return;  // nothing but banned tokens (NaN goes on, and makes s NaN)
    if (top > m) grow(top);
    const float2 mm = make_float2(-m, -m), kk = make_float2(k2, k2);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      float2 x = __fmul2_rn(__fadd2_rn(make_float2(f[i], f[i + 1]), mm), kk);
      x.x = max_nan(x.x, kFloor), x.y = max_nan(x.y, kFloor);
      const float2 e = make_float2(ex2(x.x), ex2(x.y));
      s2 = __fadd2_rn(s2, e);
      e2 = __ffma2_rn(e, x, e2);
    }
  };
  constexpr int U = 4;
  for (uint32_t i = v0 + tid; i < v1; i += U * THREADS) {
    uint4 q[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      q[u] = i + u * THREADS < v1 ? vec[i + u * THREADS]
                                  : make_uint4(V8::kNone, V8::kNone, V8::kNone, V8::kNone);
#pragma unroll
    for (int u = 0; u < U; ++u) add(q[u]);
  }
  // the edge elements, one per thread of rank 0
  const uint32_t edges = rank == 0 ? cut.head + cut.tail : 0u;
  const uint32_t edge_idx = tid < cut.head ? tid : cut.head + cut.vecs * N + (tid - cut.head);
  float edge = neg_inf;
  if (tid < edges) {
    edge = V8::load(row + edge_idx);
    if (edge != neg_inf) {
      if (edge > m) grow(edge);
      const float x = (edge - m) * k2, e = ex2(x);  // (NaN stays; finite edges are at most m: no floor needed
      s2.x += e;                                    //  above 2^-16384, where e x is -0)
      e2.x += x < kFloor ? 0.0f : e * x;
    }
  }

  Sum mine{m, s2.x + s2.y, e2.x + e2.y};
  Sum w = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    Sum other;
    other.m = __shfl_xor_sync(0xFFFFFFFFu, w.m, o);
    other.s = __shfl_xor_sync(0xFFFFFFFFu, w.s, o);
    other.e = __shfl_xor_sync(0xFFFFFFFFu, w.e, o);
    w = (lane & o) ? join(other, w, k2) : join(w, other, k2);
  }
  if (lane == 0) s_sum[warp] = w;
  if (TOP) {
    // 64 groups of THREADS / 64 consecutive lanes
    uint32_t g = order_key(mine.m);
#pragma unroll
    for (int o = 1; o < THREADS / kGroups; o <<= 1) g = max(g, __shfl_xor_sync(0xFFFFFFFFu, g, o));
    if (tid % (THREADS / kGroups) == 0) s_group[tid / (THREADS / kGroups)] = g;
    if (tid == 0) s_count = 0, s_listed = 0;
    if (tid < kMaxTop) s_top[tid] = 0;
  }
  __syncthreads();
  if (tid == 0) {
    Sum r = s_sum[0];
#pragma unroll 1
    for (int i = 1; i < WARPS; ++i) r = join(r, s_sum[i], k2);
    s_cta = r;
  }

  if (TOP) {
    const uint32_t k = a.top_k;
    const uint32_t length = (v1 - v0) * N + edges;
    if (tid < kGroups) {
      const uint32_t g = s_group[tid];
      uint32_t above = 0;
#pragma unroll 8
      for (uint32_t j = 0; j < kGroups; ++j) above += s_group[j] > g || (s_group[j] == g && j < (uint32_t)tid);
      if (above == k - 1) s_tau = g;
    }
    // NaN hides in a thread's maximum: such rows take the rounds below
    const bool odd = __syncthreads_or(mine.s != mine.s);
    const uint32_t tau = s_tau;
    uint32_t found = 0;
    if (!odd) {
      if (tid < edges && order_key(edge) >= tau) {
        const uint32_t at = atomicAdd(&s_count, 1u);
        if (at < kCap) s_cand[at] = entry_of(order_key(edge), edge_idx);
      }
      if (order_key(mine.m) >= tau) s_list[atomicAdd(&s_listed, 1u)] = static_cast<uint16_t>(tid);
      __syncthreads();
      const uint32_t strips = s_listed, per = (v1 - v0 + THREADS - 1) / THREADS;
      for (uint32_t q = tid; q < strips * per; q += THREADS) {
        const uint32_t i = v0 + s_list[q / per] + (q % per) * THREADS;
        if (i >= v1) continue;
        float f[N];
        V8::unpack(vec[i], f);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const uint32_t key = order_key(f[j]);
          if (key >= tau) {
            const uint32_t at = atomicAdd(&s_count, 1u);
            if (at < kCap) s_cand[at] = entry_of(key, cut.head + i * N + j);
          }
        }
      }
      __syncthreads();
      found = s_count;
    }
    if (!odd && found <= kCap && found >= min(k, length)) {
      // (the candidates' order in the list is not fixed, their ranks are)
      for (uint32_t i = tid; i < found; i += THREADS) {
        const uint64_t c = s_cand[i];
        uint32_t above = 0;
        for (uint32_t j = 0; j < found; ++j) above += s_cand[j] > c;
        if (above < k) s_top[above] = c;
      }
    } else {
      uint64_t last = ~0ull;
      for (uint32_t r = 0; r < min(k, length); ++r) {
        uint64_t best = 0;
        auto see = [&](float z, uint32_t idx) {
          const uint64_t c = entry_of(order_key(z), idx);
          if (c < last && c > best) best = c;
        };
        for (uint32_t i = v0 + tid; i < v1; i += THREADS) {
          float f[N];
          V8::unpack(vec[i], f);
#pragma unroll
          for (int j = 0; j < N; ++j) see(f[j], cut.head + i * N + j);
        }
        if (tid < edges) see(edge, edge_idx);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint64_t other = __shfl_xor_sync(0xFFFFFFFFu, best, o);
          best = other > best ? other : best;
        }
        __syncthreads();  // (s_best of the round before has been read)
        if (lane == 0) s_best[warp] = best;
        __syncthreads();
        best = s_best[0];
#pragma unroll 1
        for (int i = 1; i < WARPS; ++i) best = s_best[i] > best ? s_best[i] : best;
        last = best;
        if (tid == 0) s_top[r] = best;
      }
    }
  }

  if (C > 1) cluster_sync();
  else __syncthreads();
  if (rank == 0) {
    Sum r = s_cta;
    for (uint32_t c = 1; c < C; ++c) {
      const Sum other{ld_cluster_f32(&s_cta.m, c), ld_cluster_f32(&s_cta.s, c), ld_cluster_f32(&s_cta.e, c)};
      r = join(r, other, k2);
    }
    const bool empty = r.m == neg_inf && r.s == 0.0f;
    const bool bad = r.s != r.s;
    const float nan = __uint_as_float(0x7FFFFFFFu);
    const float ln_s = logf(r.s);
    if (tid == 0) {
      *reinterpret_cast<float2*>(a.stats + 2 * t) = bad ? make_float2(nan, nan) : make_float2(r.m, r.s);
      if (a.entropy) a.entropy[t] = bad ? nan : empty ? 0.0f : ln_s - kLn2 * (r.e / r.s);
      if (a.targets) {
        const int64_t at = a.targets[t];
        float v = 0.0f;
        if (at >= a.V || (bad && at >= 0)) v = nan;
        else if (at >= 0) v = empty ? neg_inf : (V8::load(row + at) - r.m) * a.scale - ln_s;
        a.logprob[t] = v;
      }
    }
    if (TOP) {
      const uint32_t k = a.top_k;
      if (C > 1) {
        for (uint32_t i = tid; i < C * k; i += THREADS) s_cand[i] = ld_cluster_u64(&s_top[i % k], i / k);
        __syncthreads();
        for (uint32_t i = tid; i < C * k; i += THREADS) {
          const uint64_t c = s_cand[i];
          uint32_t above = 0;
          for (uint32_t j = 0; j < C * k; ++j) above += s_cand[j] > c;
          if (c != 0 && above < k) s_group[above] = i;  // (entries are distinct: one writer per rank)
        }
        __syncthreads();
      }
      if (tid < k) {
        const uint64_t c = C > 1 ? s_cand[s_group[tid]] : s_top[tid];
        const float z = key_value(static_cast<uint32_t>(c >> 32));
        a.top_index[t * k + tid] = static_cast<int64_t>(0xFFFFFFFFu - static_cast<uint32_t>(c));
        a.top_logprob[t * k + tid] = bad ? nan : empty ? neg_inf : (z - r.m) * a.scale - ln_s;
      }
    }
  }
  if (C > 1) cluster_sync();  // rank 0 has read this CTA's shared memory
}

// ---------------------------------------------------------------------------
// Gradient: dz = e (A + B x2) with e = 2^x2, A = (-G - g_H (H - ln S)) scale / S, B = -g_H ln 2 scale / S,
// plus the single entries' own gradients.  One CTA per chunk of a row.
// ---------------------------------------------------------------------------
constexpr int kBwdThreads = 256, kBwdVecs = 4;

template <typename T, bool TOP>
__global__ void __launch_bounds__(kBwdThreads) logprob_bwd_kernel(const LogprobBwdArgs a, uint32_t chunks) {
  using V8 = Vec<T>;
  constexpr int N = V8::N;
  const int64_t t = blockIdx.x / chunks;
  const uint32_t chunk = blockIdx.x % chunks, V = static_cast<uint32_t>(a.V);
  const int tid = threadIdx.x;
  const T* row = static_cast<const T*>(a.logits) + t * a.ld;
  T* out = static_cast<T*>(a.dlogits) + t * a.ldd;
  const float neg_inf = __uint_as_float(0xFF800000u), nan = __uint_as_float(0x7FFFFFFFu);
  // vectors where source and destination share their alignment, else single elements
  RowCut cut = cut_row(row, V);
  const bool wide = (((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(out)) & 15u) == 0);
  constexpr uint32_t kVecs = kBwdThreads * kBwdVecs;

  const float m = a.stats[2 * t], s = a.stats[2 * t + 1];
  const float gh = a.g_entropy ? a.g_entropy[t] : 0.0f;
  int64_t target = a.targets ? a.targets[t] : -1;
  const float gt = target >= 0 ? a.g_logprob[t] : 0.0f;
  bool wrong = target >= a.V;
  float g_all = gt;
  if (TOP) {
    for (int i = 0; i < a.top_k; ++i) {
      g_all += a.g_top[t * a.top_k + i];
      const int64_t at = a.top_index[t * a.top_k + i];
      wrong |= at < 0 || at >= a.V;
    }
  }
  const float inv = s == 0.0f ? 0.0f : a.scale / s;  // (a row of banned tokens: all zeros)
  float c0 = -g_all;
  if (gh != 0.0f && s != 0.0f) c0 -= gh * (a.entropy[t] - logf(s));
  const float A = wrong ? nan : s == 0.0f ? 0.0f : c0 * inv, B = -gh * kLn2 * inv;
  const float k2 = a.scale * kLog2e;
  auto base = [&](float z) {
    const float x = fmaxf((z - m) * k2, kFloor);
    return ex2(x) * __fmaf_rn(B, x, A);
  };
  const float own_t = gt * a.scale;

  // in place, the entries with gradients of their own are read before anything is written
  const uint32_t e_lo = wide ? 0 : chunk * kVecs * N;
  auto inside = [&](int64_t at) {  // whether this CTA writes element `at`
    if (at < 0 || at >= a.V) return false;
    if (!wide) return at >= e_lo && at < (int64_t)e_lo + kVecs * N;
    const int64_t v = at - cut.head;
    if (v < 0 || v >= (int64_t)cut.vecs * N) return chunk == 0;
    return v / N / kVecs == chunk;
  };
  int64_t mine = -1;
  float z_mine = 0.0f;
  if (TOP) {
    if (tid < a.top_k) mine = a.top_index[t * a.top_k + tid];
    else if (tid == a.top_k) mine = target;
    if (!inside(mine)) mine = -1;
    if (mine >= 0) z_mine = V8::load(row + mine);
    __syncthreads();
  }
  auto one = [&](uint32_t idx) {
    const float z = V8::load(row + idx);
    float d = base(z);
    if (!TOP && idx == target && z != neg_inf) d += own_t;
    V8::store(out + idx, d);
  };
  if (wide) {
    const uint4* vec = reinterpret_cast<const uint4*>(row + cut.head);
    uint4* dst = reinterpret_cast<uint4*>(out + cut.head);
    const uint32_t i0 = chunk * kVecs + tid;
    uint4 q[kBwdVecs];
#pragma unroll
    for (int u = 0; u < kBwdVecs; ++u)
      if (i0 + u * kBwdThreads < cut.vecs) q[u] = vec[i0 + u * kBwdThreads];
#pragma unroll
    for (int u = 0; u < kBwdVecs; ++u) {
      const uint32_t i = i0 + u * kBwdThreads;
      if (i >= cut.vecs) break;
      float f[N], d[N];
      V8::unpack(q[u], f);
#pragma unroll
      for (int j = 0; j < N; ++j) d[j] = base(f[j]);
      if (!TOP) {
        const int64_t at = target - cut.head - (int64_t)i * N;
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (at == j && f[j] != neg_inf) d[j] += own_t;
      }
      dst[i] = V8::pack(d);
    }
    if (chunk == 0 && tid < cut.head + cut.tail) one(tid < cut.head ? tid : cut.vecs * N + tid);
  } else {
    for (uint32_t i = tid; i < kVecs * N; i += kBwdThreads) {
      if (V - e_lo <= i || e_lo >= V) break;
      one(e_lo + i);
    }
  }
  if (TOP) {
    __syncthreads();
    if (mine >= 0 && z_mine != neg_inf) {
      float d = base(z_mine);
      bool first = true;
      if (mine == target) d += own_t;
      for (int i = 0; i < a.top_k; ++i) {
        if (a.top_index[t * a.top_k + i] != mine) continue;
        d += a.g_top[t * a.top_k + i] * a.scale;
        if (i < tid) first = false;  // one writer per entry
      }
      if (first) V8::store(out + mine, d);
    }
  }
}

template <typename T, int THREADS, bool TOP>
static cudaError_t launch_fwd(const LogprobArgs& a, uint32_t cluster, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<uint32_t>(a.T) * cluster);
  cfg.blockDim = dim3(THREADS);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, logprob_kernel<T, THREADS, TOP>, a);
  count_launch();
  return e;
}

template <typename T>
static cudaError_t launch_fwd_t(const LogprobArgs& a, int num_sms, cudaStream_t s) {
  // Few rows: a cluster of up to 8 CTAs shares a row, while the CTAs of all rows fit the SMs about
  // twice and each still has a vector or more per thread.
  uint32_t cluster = 1;
  while (cluster < 8 && a.T * cluster < num_sms && a.V / (cluster * 2) >= 256 * Vec<T>::N) cluster *= 2;
  return a.top_k ? launch_fwd<T, 256, true>(a, cluster, s) : launch_fwd<T, 256, false>(a, cluster, s);
}

}  // namespace lp

cudaError_t launch_token_logprobs(const LogprobArgs& a, int num_sms, cudaStream_t s) {
  return a.f32 ? lp::launch_fwd_t<float>(a, num_sms, s) : lp::launch_fwd_t<__nv_bfloat16>(a, num_sms, s);
}

template <typename T>
static cudaError_t launch_bwd_t(const LogprobBwdArgs& a, cudaStream_t s) {
  const int64_t per = lp::kBwdThreads * lp::kBwdVecs * lp::Vec<T>::N;
  const int64_t chunks = (a.V + per - 1) / per;
  if (a.T * chunks > INT32_MAX) return cudaErrorInvalidConfiguration;
  const dim3 grid(static_cast<uint32_t>(a.T * chunks));
  if (a.top_k) lp::logprob_bwd_kernel<T, true><<<grid, lp::kBwdThreads, 0, s>>>(a, (uint32_t)chunks);
  else lp::logprob_bwd_kernel<T, false><<<grid, lp::kBwdThreads, 0, s>>>(a, (uint32_t)chunks);
  const cudaError_t e = cudaGetLastError();
  count_launch();
  return e;
}
cudaError_t launch_token_logprobs_bwd(const LogprobBwdArgs& a, int num_sms, cudaStream_t s) {
  (void)num_sms;
  return a.f32 ? launch_bwd_t<float>(a, s) : launch_bwd_t<__nv_bfloat16>(a, s);
}

}  // namespace nvfp4
