// The norm of many gradients and the AdamW step over many tensors (include/mok_ops.h).
//
// The tensors' addresses and sizes travel in the kernel's parameters (up to 32 KB of them), so a
// call copies nothing to the device and a captured graph holds its own table.
#include <memory>
#include <new>

#include "mok_internal.h"
#include "mok_launch.cuh"
#include "mok_ops.h"
#include "mok_rows.cuh"

namespace mok {
namespace {

constexpr int kThreads = 256;
constexpr int kBlock = 256;           // state elements that share the scales of 8-bit moments
constexpr int kRound = kThreads * 8;  // elements of a CTA at a time: a warp has one block

// ---------------------------------------------------------------- norm of many gradients
// A CTA takes 16 KB of a tensor at a time, four 16-byte loads a thread.
constexpr int kNormBytes = kThreads * 64;
constexpr int kNormCtas = 152 * 6;

struct GradEntry {
  const void* g;
  unsigned long long n;
  bool bf16, vec;
};
template <int N>
struct GradTable {
  int count;
  unsigned chunks;
  unsigned first[N];   // an entry's first chunk: by themselves, as a search reads only these
  GradEntry e[N];
};
constexpr int kGradTable = 1100;   // 28 bytes each

// The entry that holds chunk i: the last whose first chunk is at or before it.
template <typename T>
__device__ __forceinline__ int find_entry(const T& table, unsigned i) {
  int lo = 0, hi = table.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (table.first[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Sum of the squares of four vectors' elements, in fp32.
template <typename E>
__device__ __forceinline__ float squares(const uint4 (&x)[4]) {
  constexpr int V = 16 / (int)sizeof(E);
  Vec<V> s = Vec<V>::all(0.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    Vec<V> v;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if constexpr (sizeof(E) == 4) v.v[j] = __uint_as_float(w[j]);
      else v.v[j] = __uint_as_float((j & 1) ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
    }
    s = fma(v, v, s);
  }
  return s.sum();
}
// The same in fp64, for sums that fp32 cannot hold; zeros cost little.
template <typename E>
__device__ __noinline__ double wide_squares(uint4 a, uint4 b, uint4 c, uint4 d) {
  const uint4 x[4] = {a, b, c, d};
  double s = 0.;
  for (int i = 0; i < 4; ++i) {
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    for (int j = 0; j < 4; ++j) {
      const float lo = __uint_as_float(sizeof(E) == 4 ? w[j] : w[j] << 16);
      const float hi = sizeof(E) == 4 ? 0.f : __uint_as_float(w[j] & 0xffff0000u);
      if (lo != 0.f) s += (double)lo * (double)lo;
      if (hi != 0.f) s += (double)hi * (double)hi;
    }
  }
  return s;
}

// The sum of one thread's share of a chunk that begins at element `at`.
template <typename E>
__device__ __forceinline__ double chunk_squares(const GradEntry& e, size_t at) {
  constexpr int V = 16 / (int)sizeof(E);
  const E* g = static_cast<const E*>(e.g);
  uint4 x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const size_t a = at + (size_t)(i * kThreads + threadIdx.x) * V;
    x[i] = make_uint4(0u, 0u, 0u, 0u);
    if (e.vec && a + V <= e.n) {
      x[i] = *reinterpret_cast<const uint4*>(g + a);
    } else if (a < e.n) {
      uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (a + j < e.n) {
          if constexpr (sizeof(E) == 4) w[j] = __float_as_uint(g[a + j]);
          else w[j / 2] |= (uint32_t)__bfloat16_as_ushort(g[a + j]) << (16 * (j & 1));
        }
      }
      x[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  uint32_t any = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) any |= x[i].x | x[i].y | x[i].z | x[i].w;
  if (!any) return 0.;   // zeros, or behind the tensor's end
  const float s = squares<E>(x);
  if (s > 1e-30f && s < 1e38f) return (double)s;   // what underflowed is below the sum's last bit
  return wide_squares<E>(x[0], x[1], x[2], x[3]);
}

__device__ __forceinline__ double block_sum(double v) {   // in thread 0
  __shared__ double s[kThreads / 32];
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kAll, v, off);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x >= 32) return 0.;
  v = threadIdx.x < kThreads / 32 ? s[threadIdx.x] : 0.;
#pragma unroll
  for (int off = kThreads / 64; off > 0; off >>= 1) v += __shfl_xor_sync(kAll, v, off);
  return v;
}

// Bound by memory: 352M elements 105 us in bf16 (6.7 TB/s), 198 in fp32 (7.1). The CTAs' sums go on in 64
// bits, in a fixed order.
template <int N>
__global__ void __launch_bounds__(kThreads, 6)
    grad_squares_kernel(const __grid_constant__ GradTable<N> table, double* part, bool add) {
  launch_dependents();
  double d = 0.;
  for (unsigned i = blockIdx.x; i < table.chunks; i += gridDim.x) {
    const int at = find_entry(table, i);
    const GradEntry& e = table.e[at];
    const size_t c = i - table.first[at];
    d += e.bf16 ? chunk_squares<__nv_bfloat16>(e, c * (kNormBytes / 2)) : chunk_squares<float>(e, c * (kNormBytes / 4));
  }
  d = block_sum(d);
  if (threadIdx.x == 0) part[blockIdx.x] = add ? part[blockIdx.x] + d : d;
}

__global__ void __launch_bounds__(kThreads)
    grad_norm_kernel(const double* part, int parts, float max_norm, float scale, float* norm,
                     float* coef) {
  wait_prerequisites();
  double d = 0.;
  for (int i = threadIdx.x; i < parts; i += kThreads) d += part[i];
  d = block_sum(d);
  if (threadIdx.x) return;
  d = sqrt(d) * (double)scale;
  const float n = (float)d;
  *norm = n;
  *coef = !isfinite(n) ? NAN : d > (double)max_norm ? (float)(scale * (max_norm / d)) : scale;
}

// -------------------------------------------------------------------------- AdamW
struct StepEntry {
  void* p;
  const void* g;
  unsigned long long n;
  unsigned long long base;   // its first element in the state
  float decay;
  bool p_bf16, g_bf16, p_vec, g_vec;
};
template <int N>
struct StepTable {
  int count, rounds;   // a chunk: `rounds` times kRound elements
  unsigned first[N];   // an entry's first chunk
  StepEntry e[N];
};
constexpr int kStepTable = 700;   // 44 bytes each

struct Step {
  float beta1, beta2, rest1, rest2, eps;   // rest: 1 - beta
  float lr, inv_c1, inv_sqrt_c2;           // c: 1 - beta^t
  float log_beta1, log_beta2;              // for a step number on the device
  float minus_zero;
  bool all_random;                          // every code of m is rounded at random, not the small ones alone
  int t;
  const float* lr_dev;
  const int32_t* t_dev;
  const float* coef;
  uint64_t seed;
  float* master;
  void *m, *v;
  uint8_t* scales;
};

using Eight = Vec<8>;

// Products that are rounded by themselves, as a b + (-0) with a -0 that the compiler does not know:
// it fuses a paired product with the sum that follows, also where both are written as rounded.
__device__ __forceinline__ Eight mul_rn(const Eight& a, const Eight& b, const Eight& minus_zero) {
  return fma(a, b, minus_zero);
}

// 8-bit moments of the eight elements of a lane; the warp holds one block.
__device__ __forceinline__ void decode8(const uint2 mc, const uint2 vc, int a, int b, Eight& m, Eight& v) {
  const uint32_t mw[2] = {mc.x, mc.y}, vw[2] = {vc.x, vc.y};
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const uint16_t two = (uint16_t)(mw[j / 4] >> (8 * (j & 3)));
    uint32_t h2;   // two fp16
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(two));
    asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;}"
        : "=f"(m.v[j]), "=f"(m.v[j + 1])
        : "r"(h2));
  }
  m = m * Eight::all(__int_as_float((a - 7) << 23));   // 2^(a - 134)
  const int base = (b - 30) << 23;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int up = 20 - 8 * (j & 3);   // the code's byte goes to bits 20 .. 27
    const uint32_t c = (up >= 0 ? vw[j / 4] << up : vw[j / 4] >> -up) & 0x0ff00000u;
    v.v[j] = c ? __int_as_float((int)c + base) : 0.f;
  }
}

// Codes of m rounded up or down at random, as v's are, in place of the nearest ones `mc` where |x| is
// below 2^-6, or (all) everywhere. m's noise is v's with the bits in reverse order: each decides by its
// highest ones, which are the other's lowest. Codes are 2^20 apart: at and above 2^-6 in the bits of |x|,
// below in steps of 2^-29, which are the bits of |x| + 2^-6.
__device__ __noinline__ uint2 round_at_random(const Eight x, const uint2 mc, const uint4 noise, bool all) {
  const uint32_t r[4] = {noise.x, noise.y, noise.z, noise.w};
  uint32_t w[2] = {mc.x, mc.y};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t bits = __float_as_uint(x.v[j]), size = bits & 0x7fffffffu;
    const bool low = size < 121u << 23;
    const uint32_t place = low ? __float_as_uint(__uint_as_float(size) + 0x1p-6f) - (121u << 23) : size - (120u << 23);
    // 16 bits at 4 .. 19, the highest inverted: a word of 0 rounds to nearest
    const uint32_t turned = __brev(r[j / 2]);
    const uint32_t u = (((j & 1) ? turned << 4 : turned >> 12) & 0xffff0u) ^ 0x80000u;
    const uint32_t c = ((place + u) >> 20 & 0x7fu) | (bits >> 24 & 0x80u);
    const int at = 8 * (j & 3);
    if (all || low) w[j / 4] = (w[j / 4] & ~(255u << at)) | c << at;
  }
  return make_uint2(w[0], w[1]);
}

// Codes of finite moments, or (CHECK) of any: those that are not finite count for no scale. m goes to
// nearest where a step's decay, (1 - beta1) of it, is more than half the distance to the next code: for
// beta1 <= 0.9 everywhere but below 2^-6, as codes from there on are 1/16 to 1/8 of themselves apart.
// Where it is less, a nearest rounding would keep m when the gradient fades while v, rounded at random,
// goes on falling: there m is rounded at random too. (60 steps of normal gradients, then 200 of zeros,
// beta1 = beta2 = 0.95: to nearest a weight went 157 times as far as with fp32 moments, at random 1.06
// times.) All codes at random: 705 us for 235M elements, the small ones 681, none 677.
template <bool CHECK>
__device__ __forceinline__ bool encode8(const Eight& m, const Eight& v, const uint4 noise, bool all_random, uint2* mc,
                                        uint2* vc, int* a, int* b) {
  // the largest |m| and v by their fp32 bits, whose order is the values'
  uint32_t top_m = 0, top_v = 0;
  auto bad = [&](int j) {
    return (__float_as_uint(m.v[j]) & 0x7fffffffu) >= 0x7f800000u || __float_as_uint(v.v[j]) >= 0x7f800000u;
  };
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (CHECK && bad(j)) continue;
    top_m = max(top_m, __float_as_uint(m.v[j]) & 0x7fffffffu);
    top_v = max(top_v, __float_as_uint(v.v[j]));
  }
  top_m = __reduce_max_sync(kAll, top_m);
  top_v = __reduce_max_sync(kAll, top_v);
  if (!CHECK && max(top_m, top_v) >= 0x7f800000u) return false;
  *a = max((int)(top_m >> 23), 8);
  *b = max((int)(top_v >> 23), 31);
  const Eight x = m * Eight::all(__int_as_float((261 - *a) << 23));   // 2^(134 - a)
  uint32_t mw[2], vw[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x.v[4 * i + 1]), "f"(x.v[4 * i]));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x.v[4 * i + 3]), "f"(x.v[4 * i + 2]));
    mw[i] = (uint32_t)lo | (uint32_t)hi << 16;
  }
  // a byte reaches 0x80 where the code is above 8, the nearest one of 2^-6
  const uint32_t large = ((mw[0] & 0x7f7f7f7fu) + 0x77777777u) & ((mw[1] & 0x7f7f7f7fu) + 0x77777777u);
  if (all_random || (~large & 0x80808080u)) {
    const uint2 w = round_at_random(x, make_uint2(mw[0], mw[1]), noise, all_random);
    mw[0] = w.x;
    mw[1] = w.y;
  }
  // v: the bits below the code's last, plus noise of 16 bits, carry into the code. Up to 248, as the
  // largest exponent leaves room; at least 1 above 0.
  const uint32_t r[4] = {noise.x, noise.y, noise.z, noise.w};
  const int base = (*b - 30) << 23;
  int c[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int u = (int)((j & 1) ? r[j / 2] >> 12 : r[j / 2] << 4) & 0xffff0;
    const int bits = __float_as_int(v.v[j]);
    c[j] = max((bits + u - base) >> 20, min(bits, 1));
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
    vw[i] = (uint32_t)(c[4 * i] + (c[4 * i + 1] << 8) + (c[4 * i + 2] << 16)) + ((uint32_t)c[4 * i + 3] << 24);
  if (CHECK) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t byte = 255u << (8 * j);
        if (bad(4 * i + j)) {
          mw[i] = (mw[i] & ~byte) | (0x7fu << (8 * j));
          c[4 * i + j] = 255;
        }
      }
      vw[i] = (uint32_t)c[4 * i] | (uint32_t)c[4 * i + 1] << 8 | (uint32_t)c[4 * i + 2] << 16 |
              (uint32_t)c[4 * i + 3] << 24;
    }
  }
  *mc = make_uint2(mw[0], mw[1]);
  *vc = make_uint2(vw[0], vw[1]);
  return true;
}
__device__ __noinline__ void encode8_any(const Eight m, const Eight v, const uint4 noise, bool all_random, uint2* mc,
                                         uint2* vc, int* a, int* b) {
  encode8<true>(m, v, noise, all_random, mc, vc, a, b);
}

template <typename E>
__device__ __forceinline__ void load_some(const E* p, bool vec, int cnt, float* v) {
  if (vec && cnt == 8) {
    load8(p, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < cnt ? load(p + j) : 0.f;
  }
}
template <typename E>
__device__ __forceinline__ void store_some(E* p, bool vec, int cnt, const float* v) {
  if (vec && cnt == 8) {
    store8(p, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < cnt) store(p + j, v[j]);
  }
}

__device__ __forceinline__ float root(float x) {      // to 2 ulp, of subnormal numbers too
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float inverse(float x) {   // to 1 ulp, of normal numbers
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// CTAs a SM: 8-bit moments wait for their loads at four (742 us for 235M elements, 677 at six; m's small
// codes, rounded at random, add 4); 32-bit ones keep the memory busy (971 us, 1011). With fp32 masters and bf16 gradients, 352M elements: 32 bits
// 1451 us (6.8 TB/s), bound by memory; 8 bits 1016 us (5.5 TB/s), by the waits for its loads beside 67
// instructions an element. (The next elements' loads started ahead, through shared memory: 750 against
// 677 us; the noise drawn before the loads are waited for: 720.)
template <int N, bool SMALL>
__global__ void __launch_bounds__(kThreads, SMALL ? 6 : 4)
    adamw_kernel(const __grid_constant__ StepTable<N> table, const __grid_constant__ Step q) {
  const int at = find_entry(table, blockIdx.x);
  const StepEntry& e = table.e[at];
  const int lane = threadIdx.x & 31;
  size_t i = ((size_t)(blockIdx.x - table.first[at]) * table.rounds) * kRound + threadIdx.x * 8;
  const float coef = q.coef ? *q.coef : 1.f;
  float lr = q.lr, inv_c1 = q.inv_c1, inv_sqrt_c2 = q.inv_sqrt_c2;
  int t = q.t;
  if (q.lr_dev) lr = *q.lr_dev;
  if (q.t_dev) {
    t = max(*q.t_dev, 1);
    inv_c1 = -1.f / expm1f((float)t * q.log_beta1);
    inv_sqrt_c2 = 1.f / sqrtf(-expm1f((float)t * q.log_beta2));
  }
  for (int round = 0; round < table.rounds; ++round, i += kRound) {
    // this lane's eight elements: i of the tensor, s of the state
    if (i - lane * 8 >= e.n) return;   // the warp's block lies behind the tensor
    const size_t s = e.base + i;
    const int cnt = i >= e.n ? 0 : e.n - i < 8 ? (int)(e.n - i) : 8;
    Eight p, g, m, v;
    if (e.g_bf16) load_some(static_cast<const __nv_bfloat16*>(e.g) + i, e.g_vec, cnt, g.v);
    else load_some(static_cast<const float*>(e.g) + i, e.g_vec, cnt, g.v);
    if (e.p_bf16) load8(q.master + s, p.v);
    else load_some(static_cast<const float*>(e.p) + i, e.p_vec, cnt, p.v);
    if constexpr (SMALL) {
      const uchar2 ab = reinterpret_cast<const uchar2*>(q.scales)[s / kBlock];
      decode8(*reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(q.m) + s),
              *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(q.v) + s), ab.x, ab.y, m, v);
    } else {
      load8(static_cast<const float*>(q.m) + s, m.v);
      load8(static_cast<const float*>(q.v) + s, v.v);
    }
    if (!isfinite(coef)) return;
    // Every step of the moments is rounded by itself (no fused products): 8-bit moments are a
    // function of these bits.
    const Eight z = Eight::all(q.minus_zero);
    g = mul_rn(g, Eight::all(coef), z);
    m = mul_rn(m, Eight::all(q.beta1), z) + mul_rn(g, Eight::all(q.rest1), z);
    v = mul_rn(v, Eight::all(q.beta2), z) + mul_rn(mul_rn(g, g, z), Eight::all(q.rest2), z);
    Eight d;
#pragma unroll
    for (int j = 0; j < 8; ++j) d.v[j] = inverse(fmaf(root(v.v[j]), inv_sqrt_c2, q.eps));
    p = fma(fma(p, Eight::all(e.decay), (m * Eight::all(inv_c1)) * d), Eight::all(-lr), p);
    if (e.p_bf16) {
      store_some(q.master + s, true, cnt, p.v);
      store_some(static_cast<__nv_bfloat16*>(e.p) + i, e.p_vec, cnt, p.v);
    } else {
      store_some(static_cast<float*>(e.p) + i, e.p_vec, cnt, p.v);
    }
    if constexpr (SMALL) {
      uint2 mc, vc;
      int a, b;
      const uint4 noise = philox<7>(s / 8, (uint32_t)t, q.seed);
      if (!encode8<false>(m, v, noise, q.all_random, &mc, &vc, &a, &b))
        encode8_any(m, v, noise, q.all_random, &mc, &vc, &a, &b);
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(q.m) + s) = mc;
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(q.v) + s) = vc;
      if (lane == 0) reinterpret_cast<uchar2*>(q.scales)[s / kBlock] = make_uchar2(a, b);
    } else {
      store8(static_cast<float*>(q.m) + s, m.v);
      store8(static_cast<float*>(q.v) + s, v.v);
    }
  }
}

// Bound by memory: 352M elements 305 us (6.9 TB/s).
__global__ void __launch_bounds__(kThreads)
    moments_kernel(size_t elements, const uint8_t* mc, const uint8_t* vc, const uint8_t* scales,
                   __nv_bfloat16* m_out, __nv_bfloat16* v_out) {
  const size_t s = ((size_t)blockIdx.x * kThreads + threadIdx.x) * 8;
  if (s >= elements) return;
  const uchar2 ab = reinterpret_cast<const uchar2*>(scales)[s / kBlock];
  Eight m, v;
  decode8(*reinterpret_cast<const uint2*>(mc + s), *reinterpret_cast<const uint2*>(vc + s), ab.x,
          ab.y, m, v);
  store8(m_out + s, m.v);
  store8(v_out + s, v.v);
}

constexpr size_t kMaxElements = (size_t)1 << 40;

// Bytes that a call reads or writes.
struct Range {
  uintptr_t begin, end;
};
void ascend(Range* r, size_t n) {
  const auto less = [](const Range& a, const Range& b) { return a.begin < b.begin; };
  if (!std::is_sorted(r, r + n, less)) std::sort(r, r + n, less);   // one buffer's parts come sorted
}
// Whether what is written overlaps nothing else. Both lists are sorted here.
bool disjoint(Range* written, size_t n, Range* read, size_t m) {
  ascend(written, n);
  ascend(read, m);
  for (size_t i = 1; i < n; ++i)
    if (written[i].begin < written[i - 1].end) return false;
  for (size_t i = 0, w = 0; i < m; ++i) {
    while (w < n && written[w].end <= read[i].begin) ++w;
    if (w < n && written[w].begin < read[i].end) return false;
  }
  return true;
}

}  // namespace
}  // namespace mok

extern "C" mok_status mok_grad_norm_get_sizes(size_t* workspace_bytes) {
  using namespace mok;
  if (!workspace_bytes) return MOK_ERR_INVALID_ARG;
  *workspace_bytes = align_up(kNormCtas * sizeof(double), 256);
  return MOK_OK;
}

extern "C" mok_status mok_grad_norm(int count, const mok_grad* grads, float max_norm, float scale,
                                    float* norm, float* coef, void* workspace, void* stream) {
  using namespace mok;
  if (count < 0 || (count && !grads) || !(max_norm > 0.f) || !(scale > 0.f) ||
      !std::isfinite(scale) || !norm || !coef || !aligned_to(norm, 4) || !aligned_to(coef, 4))
    return MOK_ERR_INVALID_ARG;
  if (!workspace || !aligned_to(workspace, 256)) return MOK_ERR_WORKSPACE;
  for (int i = 0; i < count; ++i) {
    const mok_grad& g = grads[i];
    if (!is_type(g.type) || !aligned_to(g.g, g.type == MOK_OUT_BF16 ? 2 : 4) || g.n > kMaxElements)
      return MOK_ERR_INVALID_ARG;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  double* part = static_cast<double*>(workspace);
  int parts = 0;
  GradTable<kGradTable> table;
  table.count = 0;
  table.chunks = 0;
  cudaError_t status = cudaSuccess;
  auto flush = [&] {
    if (!table.count || status != cudaSuccess) return;
    // a later table of a longer list adds to the first's sums, in its places
    const int ctas = parts ? parts : (int)std::min<size_t>(kNormCtas, table.chunks);
    auto go = [&](const auto& tab) {
      constexpr int N = std::extent<decltype(tab.e)>::value;
      status = launch(grad_squares_kernel<N>, dim3(ctas), dim3(kThreads), 0, 1, false, s, tab, part, parts > 0);
    };
    auto few = [&](auto size) {
      GradTable<decltype(size)::value> small;
      small.count = table.count;
      small.chunks = table.chunks;
      std::copy(table.first, table.first + table.count, small.first);
      std::copy(table.e, table.e + table.count, small.e);
      go(small);
    };
    if (table.count <= 16) few(std::integral_constant<int, 16>{});
    else if (table.count <= 128) few(std::integral_constant<int, 128>{});
    else go(table);
    parts = ctas;
    table.count = 0;
    table.chunks = 0;
  };
  for (int i = 0; i < count; ++i) {
    const mok_grad& g = grads[i];
    if (!g.g || !g.n) continue;
    const size_t per = kNormBytes / (g.type == MOK_OUT_BF16 ? 2 : 4), chunks = (g.n + per - 1) / per;
    if (table.count == kGradTable || table.chunks + chunks > 0x7fffffffu) flush();
    table.first[table.count] = table.chunks;
    table.e[table.count++] = {g.g, g.n, g.type == MOK_OUT_BF16, aligned_to(g.g, 16)};
    table.chunks += (unsigned)chunks;
  }
  flush();
  if (status != cudaSuccess) return MOK_ERR_CUDA;
  status = launch(grad_norm_kernel, dim3(1), dim3(kThreads), 0, 1, parts > 0, s, (const double*)part, parts,
                  max_norm, scale, norm, coef);
  return status == cudaSuccess ? MOK_OK : MOK_ERR_CUDA;
}

extern "C" mok_status mok_adamw_get_sizes(int count, const size_t* n, size_t* elements) {
  using namespace mok;
  if (count < 0 || (count && !n) || !elements) return MOK_ERR_INVALID_ARG;
  size_t sum = 0;
  for (int i = 0; i < count; ++i) {
    if (n[i] > kMaxElements) return MOK_ERR_INVALID_ARG;
    sum += align_up(n[i], kBlock);
    if (sum > kMaxElements) return MOK_ERR_INVALID_ARG;
  }
  *elements = sum;
  return MOK_OK;
}

extern "C" mok_status mok_adamw(const mok_adamw_rule* r, int count, const mok_adamw_tensor* tensors,
                                const mok_adamw_state* st, double lr, const float* lr_dev, int t,
                                const int32_t* t_dev, const float* coef, uint64_t seed,
                                void* stream) {
  using namespace mok;
  if (!r || !st || count < 0 || (count && !tensors)) return MOK_ERR_INVALID_ARG;
  if (!(r->beta1 >= 0. && r->beta1 < 1.) || !(r->beta2 >= 0. && r->beta2 < 1.) ||
      !(r->eps >= FLT_MIN && r->eps <= FLT_MAX) || (r->bits != 8 && r->bits != 32))
    return MOK_ERR_INVALID_ARG;
  if ((!lr_dev && !std::isfinite(lr)) || (!t_dev && t < 1) || !aligned_to(lr_dev, 4) ||
      !aligned_to(t_dev, 4) || !aligned_to(coef, 4))
    return MOK_ERR_INVALID_ARG;
  const bool small = r->bits == 8;
  size_t total = 0;
  bool any = false, masters = false;
  for (int i = 0; i < count; ++i) {
    const mok_adamw_tensor& x = tensors[i];
    if (!is_type(x.p_type) || !is_type(x.g_type) || x.n > kMaxElements || !std::isfinite(x.decay) ||
        (x.n && !x.p) || !aligned_to(x.p, x.p_type == MOK_OUT_BF16 ? 2 : 4) ||
        !aligned_to(x.g, x.g_type == MOK_OUT_BF16 ? 2 : 4))
      return MOK_ERR_INVALID_ARG;
    total += align_up(x.n, kBlock);
    if (total > kMaxElements) return MOK_ERR_INVALID_ARG;
    any |= x.n > 0;
    masters |= x.n > 0 && x.p_type == MOK_OUT_BF16;
  }
  if (!any) return MOK_OK;
  if (!st->m || !st->v || (small && !st->scales) || (masters && !st->master) ||
      !aligned_to(st->m, 16) || !aligned_to(st->v, 16) || !aligned_to(st->scales, 16) ||
      !aligned_to(st->master, 16))
    return MOK_ERR_INVALID_ARG;
  {
    std::unique_ptr<Range[]> ranges(new (std::nothrow) Range[2 * (size_t)count + 4]);
    if (!ranges) return MOK_ERR_UNSUPPORTED;
    Range *written = ranges.get(), *read = written + count + 4;
    size_t n = 0, m = 0;
    auto bytes = [](const void* p, size_t n, mok_out_dtype type) {
      return Range{(uintptr_t)p, (uintptr_t)p + n * (type == MOK_OUT_BF16 ? 2 : 4)};
    };
    for (int i = 0; i < count; ++i) {
      const mok_adamw_tensor& x = tensors[i];
      if (!x.n) continue;
      written[n++] = bytes(x.p, x.n, x.p_type);
      if (x.g) read[m++] = bytes(x.g, x.n, x.g_type);
    }
    const uintptr_t kind = small ? 1 : 4;
    written[n++] = {(uintptr_t)st->m, (uintptr_t)st->m + total * kind};
    written[n++] = {(uintptr_t)st->v, (uintptr_t)st->v + total * kind};
    if (small) written[n++] = {(uintptr_t)st->scales, (uintptr_t)st->scales + total / kBlock * 2};
    if (masters) written[n++] = {(uintptr_t)st->master, (uintptr_t)st->master + total * 4};
    if (!disjoint(written, n, read, m)) return MOK_ERR_INVALID_ARG;
  }
  Step q{};
  q.beta1 = (float)r->beta1; q.beta2 = (float)r->beta2;
  q.rest1 = (float)(1. - r->beta1); q.rest2 = (float)(1. - r->beta2);
  q.eps = (float)r->eps;
  q.lr = (float)lr;
  q.t = t_dev ? 1 : t;
  q.inv_c1 = (float)(1. / (1. - std::pow(r->beta1, (double)q.t)));
  q.inv_sqrt_c2 = (float)(1. / std::sqrt(1. - std::pow(r->beta2, (double)q.t)));
  q.log_beta1 = (float)std::log(r->beta1); q.log_beta2 = (float)std::log(r->beta2);
  q.minus_zero = -0.f;
  q.all_random = r->beta1 > 0.9;
  q.lr_dev = lr_dev; q.t_dev = t_dev; q.coef = coef; q.seed = seed;
  q.master = st->master; q.m = st->m; q.v = st->v; q.scales = st->scales;
  cudaStream_t s = static_cast<cudaStream_t>(stream);

  // chunks of up to four rounds, fewer where that would leave SMs idle
  StepTable<kStepTable> table;
  table.count = 0;
  table.rounds = total / kRound < 152 * 32 ? 1 : total / kRound < 152 * 64 ? 2 : 4;
  const size_t chunk = (size_t)table.rounds * kRound;
  unsigned chunks = 0;
  cudaError_t status = cudaSuccess;
  auto flush = [&] {
    if (!table.count || status != cudaSuccess) return;
    auto go = [&](const auto& tab) {
      constexpr int N = std::extent<decltype(tab.e)>::value;
      status = launch(small ? adamw_kernel<N, true> : adamw_kernel<N, false>, dim3(chunks), dim3(kThreads), 0, 1,
                      false, s, tab, q);
    };
    auto few = [&](auto size) {
      StepTable<decltype(size)::value> part;
      part.count = table.count;
      part.rounds = table.rounds;
      std::copy(table.first, table.first + table.count, part.first);
      std::copy(table.e, table.e + table.count, part.e);
      go(part);
    };
    if (table.count <= 16) few(std::integral_constant<int, 16>{});
    else if (table.count <= 64) few(std::integral_constant<int, 64>{});
    else if (table.count <= 256) few(std::integral_constant<int, 256>{});
    else go(table);
    table.count = 0;
    chunks = 0;
  };
  size_t base = 0;
  for (int i = 0; i < count; ++i) {
    const mok_adamw_tensor& x = tensors[i];
    const size_t own = (x.n + chunk - 1) / chunk;
    if (x.g && x.n) {
      if (table.count == kStepTable || chunks + own > 0x7fffffffu) flush();
      table.first[table.count] = chunks;
      table.e[table.count++] = {x.p, x.g, x.n, base, (float)x.decay,
                                x.p_type == MOK_OUT_BF16, x.g_type == MOK_OUT_BF16,
                                aligned_to(x.p, 16), aligned_to(x.g, 16)};
      chunks += (unsigned)own;
    }
    base += align_up(x.n, kBlock);
  }
  flush();
  return status == cudaSuccess ? MOK_OK : MOK_ERR_CUDA;
}

extern "C" mok_status mok_adamw_moments(size_t elements, const mok_adamw_state* st, void* m,
                                        void* v, void* stream) {
  using namespace mok;
  if (!st || elements % kBlock || elements > kMaxElements) return MOK_ERR_INVALID_ARG;
  if (elements == 0) return MOK_OK;
  if (!st->m || !st->v || !st->scales || !m || !v || !aligned_to(st->m, 16) ||
      !aligned_to(st->v, 16) || !aligned_to(st->scales, 16) || !aligned_to(m, 16) ||
      !aligned_to(v, 16))
    return MOK_ERR_INVALID_ARG;
  const size_t blocks = (elements / 8 + kThreads - 1) / kThreads;
  const cudaError_t e = launch(moments_kernel, dim3((unsigned)blocks), dim3(kThreads), 0, 1, false,
                               static_cast<cudaStream_t>(stream), elements, static_cast<const uint8_t*>(st->m),
                               static_cast<const uint8_t*>(st->v), (const uint8_t*)st->scales,
                               static_cast<__nv_bfloat16*>(m), static_cast<__nv_bfloat16*>(v));
  return e == cudaSuccess ? MOK_OK : MOK_ERR_CUDA;
}
