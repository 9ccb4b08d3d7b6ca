// Dropout from a counter-based generator (include/mok_ops.h, mok_dropout).
//
//   y_i = add_i + (u_i >= t ? x_i * 65536 / (65536 - t) : 0),   t = round(65536 p)
//
// u_i is the i-th 16-bit word of a Philox4x32-10 stream (Salmon, Moraes, Dror, Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", SC 2011, whose multipliers and key
// increments appear below), so the mask is a function of (seed, offset, i): nothing is
// stored, and the backward draws the same bits again. Sixteen bits per element make one
// generator call serve eight elements, one 16-byte vector of bf16. The scale is the inverse
// of the kept share of the 65536 words, so E[y] = x exactly.
//
// Bound: HBM, x (and add) in, y out; ten rounds per eight elements cost about as many issue
// slots as the copy has time for. One group of eight per thread: 8192 x 7168 bf16 with add takes
// 57 us, 6.2 TB/s, 0.91 of a plain copy (two or four groups per thread, their loads first, took
// 76 and 104 us).
#include <cmath>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "mok_internal.h"
#include "mok_ops.h"

namespace mok {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint4 philox(uint64_t counter, uint64_t seed) {
  uint32_t c0 = (uint32_t)counter, c1 = (uint32_t)(counter >> 32), c2 = 0, c3 = 0;
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
  for (int i = 0; i < 10; ++i) {
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

// One thread per group of eight elements. VEC: every pointer is 16-byte aligned, full
// groups go as vectors; the last partial group, and unaligned tensors, element by element.
// y may be x or add (each thread reads its elements before it writes them), so neither is
// __restrict__.
template <typename E, bool VEC>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const E* x, const E* add, E* y,
                                                           size_t n, uint32_t t, float up,
                                                           uint64_t seed, uint64_t offset) {
  const size_t g = (size_t)blockIdx.x * kThreads + threadIdx.x;
  const size_t i0 = g * 8;
  if (i0 >= n) return;
  const bool whole = VEC && i0 + 8 <= n;
  const int cnt = n - i0 < 8 ? (int)(n - i0) : 8;
  float v[8], a[8];
  if (whole) {
    load8(x + i0, v);
    if (add) load8(add + i0, a);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = j < cnt ? load(x + i0 + j) : 0.f;
      a[j] = j < cnt && add ? load(add + i0 + j) : 0.f;
    }
  }
  const uint4 r = philox(offset + g, seed);
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t u = (j & 1) ? w[j >> 1] >> 16 : w[j >> 1] & 0xffffu;
    // a select, not a product: a dropped inf or NaN gives 0
    v[j] = u >= t ? v[j] * up : 0.f;
    if (add) v[j] += a[j];
  }
  if (whole) {
    store8(y + i0, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < cnt) store(y + i0 + j, v[j]);
  }
}

template <typename E>
cudaError_t launch(const void* x, const void* add, void* y, size_t n, uint32_t t, uint64_t seed,
                   uint64_t offset, cudaStream_t s) {
  const uintptr_t bits = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(add) |
                         reinterpret_cast<uintptr_t>(y);
  const float up = 65536.f / (float)(65536u - t);
  const size_t blocks = ((n + 7) / 8 + kThreads - 1) / kThreads;
  const E* px = static_cast<const E*>(x);
  const E* pa = static_cast<const E*>(add);
  if ((bits & 15) == 0)
    dropout_kernel<E, true><<<(unsigned)blocks, kThreads, 0, s>>>(px, pa, static_cast<E*>(y), n, t,
                                                                  up, seed, offset);
  else
    dropout_kernel<E, false><<<(unsigned)blocks, kThreads, 0, s>>>(px, pa, static_cast<E*>(y), n, t,
                                                                   up, seed, offset);
  return cudaGetLastError();
}

}  // namespace
}  // namespace mok

extern "C" mok_status mok_dropout(const void* x, const void* add, void* y, size_t n, float p,
                                  uint64_t seed, uint64_t offset, mok_out_dtype type,
                                  void* stream) {
  using namespace mok;
  if (type != MOK_OUT_BF16 && type != MOK_OUT_F32) return MOK_ERR_INVALID_ARG;
  if (!(p >= 0.f && p < 1.f)) return MOK_ERR_INVALID_ARG;
  const uint32_t t = (uint32_t)std::lrint((double)p * 65536.0);
  if (t >= 65536u) return MOK_ERR_INVALID_ARG;
  if (n == 0) return MOK_OK;
  if (!x || !y) return MOK_ERR_INVALID_ARG;
  if ((n + 7) / 8 > (size_t)0x7fffffff * kThreads) return MOK_ERR_UNSUPPORTED;   // grid size
  const uintptr_t low = type == MOK_OUT_BF16 ? 1 : 3;
  if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(add) |
       reinterpret_cast<uintptr_t>(y)) & low)
    return MOK_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = type == MOK_OUT_BF16
                            ? launch<__nv_bfloat16>(x, add, y, n, t, seed, offset, s)
                            : launch<float>(x, add, y, n, t, seed, offset, s);
  return e == cudaSuccess ? MOK_OK : MOK_ERR_CUDA;
}
