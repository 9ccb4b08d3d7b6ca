// Device helpers that the operators share: bf16 and fp32 elements through vector accesses, rows
// of logits spread over the lanes of a warp, warp-wide sums and maxima, softmax and Philox.
#pragma once
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "mok.h"

namespace mok {
namespace {

constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ float load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float load(const float* p) { return *p; }
__device__ __forceinline__ void store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store(float* p, float v) { *p = v; }

// Eight consecutive elements through 16-byte accesses.
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* v) {
  const uint4 q = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float* v) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, const float* v) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// V elements at a time, in pairs: one instruction does two fp32 operations, each rounded as usual.
template <int V>
struct Vec {
  float v[V];
  static __device__ __forceinline__ Vec all(float x) {
    Vec o;
#pragma unroll
    for (int j = 0; j < V; ++j) o.v[j] = x;
    return o;
  }
  __device__ __forceinline__ float2 pair(int j) const { return make_float2(v[j], v[(j + 1) % V]); }
  __device__ __forceinline__ void set(int j, float2 p) { v[j] = p.x; v[(j + 1) % V] = p.y; }
  __device__ __forceinline__ float sum() const {
    if constexpr (V == 1) return v[0];
    float2 t = pair(0);
#pragma unroll
    for (int j = 2; j + 1 < V; j += 2) t = __fadd2_rn(t, pair(j));
    return t.x + t.y;
  }
};
template <int V>
__device__ __forceinline__ Vec<V> operator+(const Vec<V>& a, const Vec<V>& b) {
  Vec<V> o;
  if constexpr (V == 1) o.v[0] = a.v[0] + b.v[0];
#pragma unroll
  for (int j = 0; j + 1 < V; j += 2) o.set(j, __fadd2_rn(a.pair(j), b.pair(j)));
  return o;
}
template <int V>
__device__ __forceinline__ Vec<V> operator*(const Vec<V>& a, const Vec<V>& b) {
  Vec<V> o;
  if constexpr (V == 1) o.v[0] = a.v[0] * b.v[0];
#pragma unroll
  for (int j = 0; j + 1 < V; j += 2) o.set(j, __fmul2_rn(a.pair(j), b.pair(j)));
  return o;
}
template <int V>
__device__ __forceinline__ float dot(const Vec<V>& a, const Vec<V>& b) {
  if constexpr (V == 1) return a.v[0] * b.v[0];
  float2 t = __fmul2_rn(a.pair(0), b.pair(0));
#pragma unroll
  for (int j = 2; j + 1 < V; j += 2) t = __ffma2_rn(a.pair(j), b.pair(j), t);
  return t.x + t.y;
}
template <int V>
__device__ __forceinline__ Vec<V> fma(const Vec<V>& a, const Vec<V>& b, const Vec<V>& c) {
  Vec<V> o;
  if constexpr (V == 1) o.v[0] = fmaf(a.v[0], b.v[0], c.v[0]);
#pragma unroll
  for (int j = 0; j + 1 < V; j += 2) o.set(j, __ffma2_rn(a.pair(j), b.pair(j), c.pair(j)));
  return o;
}

// A logit as the rule reads it: NaN masks like -inf, +inf is the largest finite value.
__device__ __forceinline__ float clean(float l) { return fminf(fmaxf(l, -INFINITY), FLT_MAX); }

// Unsigned key in the order of v (equal for -0 and +0; -inf lowest, above 0 = "no candidate").
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kAll, v, off);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {   // no NaN among the values
  return key_value(__reduce_max_sync(kAll, order_key(v)));
}

// 1 - sigmoid(l) is sigmoid(-l): no cancellation near 1
__device__ __forceinline__ float sigmoid(float l) { return 1.f / (1.f + expf(-l)); }

// The NV consecutive elements from e0 of a row of E; `fill` past its end. vec: e0 NV-aligned,
// E a multiple of NV, addresses aligned for the widest access that divides NV elements.
template <int NV, typename T>
__device__ __forceinline__ void load_row(const T* row, int e0, int E, bool vec, float fill,
                                         float* v) {
  constexpr int bytes = NV * (int)sizeof(T);
  if constexpr (bytes % 4 == 0) {
    if (vec) {
      if (e0 < E) {
        uint32_t w[bytes / 4];
        if constexpr (bytes % 16 == 0) {
#pragma unroll
          for (int i = 0; i < bytes / 16; ++i) {
            const uint4 q = reinterpret_cast<const uint4*>(row + e0)[i];
            w[4 * i] = q.x; w[4 * i + 1] = q.y; w[4 * i + 2] = q.z; w[4 * i + 3] = q.w;
          }
        } else if constexpr (bytes % 8 == 0) {
#pragma unroll
          for (int i = 0; i < bytes / 8; ++i) {
            const uint2 q = reinterpret_cast<const uint2*>(row + e0)[i];
            w[2 * i] = q.x; w[2 * i + 1] = q.y;
          }
        } else {
#pragma unroll
          for (int i = 0; i < bytes / 4; ++i) w[i] = reinterpret_cast<const uint32_t*>(row + e0)[i];
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if constexpr (sizeof(T) == 4) v[i] = __uint_as_float(w[i]);
          else v[i] = __uint_as_float((i & 1) ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
        }
      } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = fill;
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = e0 + i < E ? load(row + e0 + i) : fill;
}
template <int NV, typename T>
__device__ __forceinline__ void store_row(T* row, int e0, int E, bool vec, const float* v) {
  constexpr int bytes = NV * (int)sizeof(T);
  if constexpr (bytes % 4 == 0) {
    if (vec) {
      if (e0 >= E) return;
      uint32_t w[bytes / 4];
#pragma unroll
      for (int i = 0; i < bytes / 4; ++i) {
        if constexpr (sizeof(T) == 4) {
          w[i] = __float_as_uint(v[i]);
        } else {
          const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
          w[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
      }
      if constexpr (bytes % 16 == 0) {
#pragma unroll
        for (int i = 0; i < bytes / 16; ++i)
          reinterpret_cast<uint4*>(row + e0)[i] =
              make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
      } else if constexpr (bytes % 8 == 0) {
#pragma unroll
        for (int i = 0; i < bytes / 8; ++i)
          reinterpret_cast<uint2*>(row + e0)[i] = make_uint2(w[2 * i], w[2 * i + 1]);
      } else {
#pragma unroll
        for (int i = 0; i < bytes / 4; ++i) reinterpret_cast<uint32_t*>(row + e0)[i] = w[i];
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (e0 + i < E) store(row + e0 + i, v[i]);
}

// Softmax over the warp's logits s (cleaned): s becomes the scores, m and 1 / z its
// statistics. A fully masked row has scores 0. expf, not __expf, whose error grows with the
// argument (to 1e-5 of the smallest scores, all of which the dense gradient writes).
template <int NV>
__device__ __forceinline__ void warp_softmax(float* s, float& m, float& inv_z) {
  m = s[0];
#pragma unroll
  for (int i = 1; i < NV; ++i) m = fmaxf(m, s[i]);
  m = warp_max(m);
  if (m == -INFINITY) m = 0.f;
  float z = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    s[i] = expf(s[i] - m);
    z += s[i];
  }
  z = warp_sum(z);
  inv_z = z > 0.f ? 1.f / z : 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) s[i] *= inv_z;
}

// Philox4x32 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011,
// whose multipliers and key increments appear here): four 32-bit words of a counter and a key.
template <int ROUNDS>
__device__ __forceinline__ uint4 philox(uint64_t counter, uint32_t c2, uint64_t seed) {
  uint32_t c0 = (uint32_t)counter, c1 = (uint32_t)(counter >> 32), c3 = 0;
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
  for (int i = 0; i < ROUNDS; ++i) {
    const uint64_t p0 = (uint64_t)c0 * 0xD2511F53u, p1 = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(p1 >> 32) ^ c1 ^ k0;
    c2 = (uint32_t)(p0 >> 32) ^ c3 ^ k1;
    c1 = (uint32_t)p1;
    c3 = (uint32_t)p0;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// Logits per lane: the smallest of the built widths that holds a row in 32 lanes.
inline int lane_width(int E) {
  const int nv = (E + 31) / 32;
  return nv <= 2 ? nv : nv <= 4 ? 4 : nv <= 8 ? 8 : nv <= 12 ? 12 : 16;
}
template <class F>
void by_width(int E, F f) {
  switch (lane_width(E)) {
    case 1: f(std::integral_constant<int, 1>{}); break;
    case 2: f(std::integral_constant<int, 2>{}); break;
    case 4: f(std::integral_constant<int, 4>{}); break;
    case 8: f(std::integral_constant<int, 8>{}); break;
    case 12: f(std::integral_constant<int, 12>{}); break;
    default: f(std::integral_constant<int, 16>{}); break;
  }
}

inline bool is_type(mok_out_dtype t) { return t == MOK_OUT_BF16 || t == MOK_OUT_F32; }
inline bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Vector accesses to the rows of [T][E]: whole lanes only, aligned to the widest power of
// two that divides a lane's bytes (at most 16).
inline bool rows_vectorize(int E, const void* p, mok_out_dtype type) {
  const int nv = lane_width(E), es = type == MOK_OUT_BF16 ? 2 : 4;
  const int width = std::min(16, (nv * es) & -(nv * es));
  return E % nv == 0 && (long long)E * es % width == 0 && aligned_to(p, width);
}

}  // namespace
}  // namespace mok
