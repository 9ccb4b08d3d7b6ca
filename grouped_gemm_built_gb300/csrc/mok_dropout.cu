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
#include "mok_internal.h"
#include "mok_ops.h"
#include "mok_rows.cuh"

namespace mok {
namespace {

constexpr int kThreads = 256;

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
  const uint4 r = philox<10>(offset + g, 0, seed);
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
