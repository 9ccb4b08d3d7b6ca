// Layer norm and RMS norm of rows, with the residual sum in front, and their gradients
// (include/mok_ops.h, mok_norm_fwd and mok_norm_bwd).
//
//   h = x + add;  xh = (h - m) r;  y = xh w + b
//   dX = r (t - [mean t] - xh mean(t xh)) + add,  t = dY w;   dW = sum dY xh,  dB = sum dY
//
// Bound by memory. A team of threads, from a warp (H <= 1024) to a whole CTA, goes through rows
// a grid apart, so that a thread keeps the same columns throughout: dW and dB stay in its registers
// and leave as one partial row per CTA, which a second, overlapped kernel sums up. Each thread
// copies its own part of the next row to shared memory (cp.async: asynchronous, and nobody else
// reads it, so there is no barrier and no wait on another thread) while the team reduces this one.
#include <climits>

#include "mok_internal.h"
#include "mok_launch.cuh"
#include "mok_ops.h"
#include "mok_ptx.cuh"
#include "mok_rows.cuh"

namespace mok {
namespace {

constexpr int kMaxH = 32768;
constexpr int kSms = 152;
constexpr int kMaxParts = kSms * 4;    // partial rows of dW and dB
constexpr int kRingBytes = 224 * 1024; // shared memory of an SM for rows in flight

struct NormArgs {
  int T, H;
  float eps;
  bool rms, w_bf16;
  int stages;                    // rows in flight per team; 0: no ring
  const void *x, *add, *w, *b;   // the backward: h in place of x, add the gradient's
  const void* dy;
  void *h, *y;                   // the backward: dX in place of y
  float2* stats;
  float *part_w, *part_b;        // [parts][H]
  void *dw, *db;
  int parts;
};

// V consecutive elements of a tensor or of shared memory
template <int V, typename E>
__device__ __forceinline__ void get(const E* p, float* v) {
  if constexpr (V == 8) {
    load8(p, v);
  } else if constexpr (V == 4 && sizeof(E) == 4) {
    const float4 q = *reinterpret_cast<const float4*>(p);
    v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
  } else if constexpr (V == 4) {
    const uint2 q = *reinterpret_cast<const uint2*>(p);
    v[0] = __uint_as_float(q.x << 16); v[1] = __uint_as_float(q.x & 0xffff0000u);
    v[2] = __uint_as_float(q.y << 16); v[3] = __uint_as_float(q.y & 0xffff0000u);
  } else {
    v[0] = load(p);
  }
}
template <int V, typename E>
__device__ __forceinline__ void put(E* p, const float* v) {
  if constexpr (V == 8) {
    store8(p, v);
  } else if constexpr (V == 4 && sizeof(E) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else if constexpr (V == 4) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    *reinterpret_cast<uint2*>(p) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  } else {
    store(p, v[0]);
  }
}
// ... of a parameter, of type W, or (void) of the type that the call names
template <int V, typename W>
__device__ __forceinline__ void get_w(const NormArgs& q, const void* p, int c, float* v) {
  if constexpr (!std::is_void_v<W>) get<V>(static_cast<const W*>(p) + c, v);
  else if (q.w_bf16) get<V>(static_cast<const __nv_bfloat16*>(p) + c, v);
  else get<V>(static_cast<const float*>(p) + c, v);
}

// V elements as they lie in memory, unpacked when they are used; a thread's place in shared memory
// holds 16 bytes of them, the rest follows in a second place.
constexpr int kPlace = 512;   // one access of a warp
template <int V, typename E>
constexpr int kWPlaces = V * (int)sizeof(E) > 16 ? 2 : 1;
template <int V, typename E>
struct __align__(V * sizeof(E)) Raw {
  E v[V];
  static constexpr int kBytes = V * (int)sizeof(E), kPart = kBytes < 16 ? kBytes : 16;
  using Word = std::conditional_t<kPart == 16, uint4, std::conditional_t<kPart == 8, uint2, uint32_t>>;
  __device__ __forceinline__ void read(const E* p) {
#pragma unroll
    for (int i = 0; i < kBytes / kPart; ++i)
      reinterpret_cast<Word*>(v)[i] = reinterpret_cast<const Word*>(p)[i];
  }
  __device__ __forceinline__ void keep(char* to) const {
#pragma unroll
    for (int i = 0; i < kBytes / kPart; ++i)
      *reinterpret_cast<Word*>(to + i * kPlace) = reinterpret_cast<const Word*>(v)[i];
  }
  __device__ __forceinline__ void fetch(const char* from) {
#pragma unroll
    for (int i = 0; i < kBytes / kPart; ++i)
      reinterpret_cast<Word*>(v)[i] = *reinterpret_cast<const Word*>(from + i * kPlace);
  }
};
// What a backward call needs beyond dX and dW: nothing for an RMS norm, the rows' means, dB as well.
enum { kRms, kMeans, kBias };
// Whether a backward kernel holds w in registers; else the places that it takes.
template <int V, typename W>
constexpr bool keeps_w(int mode) {
  return V == 8 && std::is_same_v<W, __nv_bfloat16> && mode != kBias;
}
template <int N, int V, typename W>
constexpr int w_places(int mode) {
  if constexpr (V == 1) return 0;
  else return keeps_w<V, W>(mode) ? 0 : N * kWPlaces<V, W>;
}

__device__ __forceinline__ void prefetch_l1(const void* p) {
  asm volatile("prefetch.global.L1 [%0];" ::"l"(p));
}
template <int ID>
__device__ __forceinline__ void named_bar_sync(int count) {
  asm volatile("bar.sync %0, %1;" ::"n"(ID), "r"(count) : "memory");
}
// Sums over the threads of a team of a, and of b where `both`. `turn` alternates between two places,
// so that one barrier a sum is enough.
__device__ __forceinline__ float2 row_sum(float a, float b, bool both, int& turn) {
  const int lane = threadIdx.x & 31;
  if (both) {   // the lower half warp goes on with a, the upper with b
    const float other = __shfl_xor_sync(kAll, lane < 16 ? b : a, 16);
    a = (lane < 16 ? a : b) + other;
  } else {
    a += __shfl_xor_sync(kAll, a, 16);
  }
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) a += __shfl_xor_sync(kAll, a, off);
  if (blockDim.x == 32)
    return make_float2(__shfl_sync(kAll, a, 0), __shfl_sync(kAll, a, 16));
  __shared__ float2 s[2][32];
  const int warps = blockDim.x >> 5, first = threadIdx.y * warps;
  turn ^= 1;
  if ((lane & 15) == 0)
    reinterpret_cast<float*>(&s[turn][first + (threadIdx.x >> 5)])[lane >> 4] = a;
  // teams differ in their rows; constant numbers, as a number in a register takes all 16 barriers
  if (blockDim.y == 1) __syncthreads();
  else if (threadIdx.y == 0) named_bar_sync<1>(blockDim.x);
  else if (threadIdx.y == 1) named_bar_sync<2>(blockDim.x);
  else if (threadIdx.y == 2) named_bar_sync<3>(blockDim.x);
  else named_bar_sync<4>(blockDim.x);
  float2 t = make_float2(0.f, 0.f);
  if (warps <= 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 v = s[turn][first + min(i, warps - 1)];
      t.x += i < warps ? v.x : 0.f;
      t.y += i < warps ? v.y : 0.f;
    }
    return t;
  }
  if (lane < warps) t = s[turn][first + lane];
  return make_float2(warp_sum(t.x), warp_sum(t.y));
}

// A thread's part of a row: N accesses, 32 V elements apart, from element c0 on; those below `live`
// lie in the row.
template <int N, int V>
struct Part {
  int c0, live;
  __device__ __forceinline__ explicit Part(int H) {
    c0 = (int)(threadIdx.x >> 5) * (32 * N * V) + (int)(threadIdx.x & 31) * V;
    live = c0 < H ? min(N, (H - c0 + 32 * V - 1) / (32 * V)) : 0;
  }
};
// A thread's places in shared memory, for `stages` rows of K tensors: an access of its warp is 512 bytes
// in one piece (asynchronous copies to places further apart took 1.4 times as long).
// `more` places beyond those.
extern __shared__ __align__(16) char ring[];
template <int N, int K>
__device__ __forceinline__ char* places(int stages, int more) {
  const int warp = (threadIdx.y * blockDim.x + threadIdx.x) >> 5;
  return ring + (size_t)warp * ((stages * K * N + more) * kPlace) + (threadIdx.x & 31) * 16;
}
// Starts the copies of this thread's part of a row (`from`: its first element) to `to` on.
template <int N, int V, typename E>
__device__ __forceinline__ void fetch(uint32_t to, const E* from, int live) {
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (i < live) copy_async<V * (int)sizeof(E)>(to + i * kPlace, from + i * (32 * V));
}

// RING: V elements a copy, 16 bytes at most; else V = 1, any alignment.
template <int N, int V, typename X, typename Y, typename W, int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) norm_fwd_kernel(const NormArgs q) {
  constexpr bool RING = V > 1;
  constexpr int K = 2;
  const Part<N, V> part(q.H);
  const size_t step = (size_t)gridDim.x * blockDim.y;
  size_t row = (size_t)blockIdx.x * blockDim.y + threadIdx.y;
  const float inv_h = 1.f / (float)q.H;
  char* const mine = RING ? places<N, K>(q.stages, 0) : nullptr;
  auto start = [&](size_t r, int stage) {
    if constexpr (RING) {
      if (r < (size_t)q.T) {
        const uint32_t to = smem_u32(mine) + stage * (K * N * kPlace);
        const size_t at = r * q.H + part.c0;
        fetch<N, V>(to, static_cast<const X*>(q.x) + at, part.live);
        if (q.add) fetch<N, V>(to + N * kPlace, static_cast<const X*>(q.add) + at, part.live);
      }
      copies_commit();
    }
  };
  int stage = 0, turn = 0;
  for (int s = 0; s < q.stages; ++s) start(row + s * step, s);
  if constexpr (RING) {   // the first row's second trip to memory, made beside its first
    const int size = q.w_bf16 ? 2 : 4;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i < part.live) {
        const size_t c = (size_t)(part.c0 + i * (32 * V)) * size;
        prefetch_l1(static_cast<const char*>(q.w) + c);
        if (q.b) prefetch_l1(static_cast<const char*>(q.b) + c);
      }
    }
  }
  for (; row < (size_t)q.T; row += step) {
    const size_t at = row * q.H + part.c0;
    const char* here = mine + stage * (K * N * kPlace);
    Vec<V> v[N];
    if constexpr (RING) copies_wait(q.stages - 1);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = Vec<V>::all(0.f);
      if (i < part.live)
        get<V>(RING ? reinterpret_cast<const X*>(here + i * kPlace)
                    : static_cast<const X*>(q.x) + at + i * (32 * V), v[i].v);
    }
    if (q.add) {
      Vec<V> kept[RING ? 1 : N];   // without a ring: all loads before the first store
      if constexpr (!RING) {
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (i < part.live) get<V>(static_cast<const X*>(q.add) + at + i * (32 * V), kept[i].v);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (i < part.live) {
          if constexpr (RING) {
            Vec<V> a;
            get<V>(reinterpret_cast<const X*>(here + (N + i) * kPlace), a.v);
            v[i] = v[i] + a;
          } else {
            v[i] = v[i] + kept[i];
          }
          if constexpr (sizeof(X) == 2) {   // the norm is that of the stored h
#pragma unroll
            for (int j = 0; j < V; ++j) v[i].v[j] = __bfloat162float(__float2bfloat16_rn(v[i].v[j]));
          }
          put<V>(static_cast<X*>(q.h) + at + i * (32 * V), v[i].v);
        }
      }
    }
    start(row + q.stages * step, stage);
    if (++stage >= q.stages) stage = 0;
    float mean = 0.f;
    if (!q.rms) {
      Vec<V> sum = Vec<V>::all(0.f);
#pragma unroll
      for (int i = 0; i < N; ++i) sum = sum + v[i];
      mean = row_sum(sum.sum(), 0.f, false, turn).x * inv_h;
      const Vec<V> minus = Vec<V>::all(-mean);
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i < part.live) v[i] = v[i] + minus;
    }
    Vec<V> sq = Vec<V>::all(0.f);
#pragma unroll
    for (int i = 0; i < N; ++i) sq = fma(v[i], v[i], sq);
    const float r = 1.f / sqrtf(row_sum(sq.sum(), 0.f, false, turn).x * inv_h + q.eps);
    if (q.stats && threadIdx.x == 0) q.stats[row] = make_float2(mean, r);
    const Vec<V> rv = Vec<V>::all(r);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i < part.live) {
        const int c = part.c0 + i * (32 * V);
        Vec<V> w, b = Vec<V>::all(0.f);
        get_w<V, W>(q, q.w, c, w.v);
        if (q.b) get_w<V, W>(q, q.b, c, b.v);
        const Vec<V> y = fma(v[i] * rv, w, b);
        put<V>(static_cast<Y*>(q.y) + at + i * (32 * V), y.v);
      }
    }
  }
}

// The parameters are read once: w stays in registers in the type it has, or, where dB's sums need
// those, in the thread's own places of shared memory. (Read again for every row through L1, twice,
// they made up a fifth of the kernel's time: 8192 x 7168 bf16 with add 95.6 us, now 78.3.)
template <int N, int V, typename X, typename Y, typename W, int MODE, int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) norm_bwd_kernel(const NormArgs q) {
  launch_dependents();
  constexpr bool RING = V > 1, DB = MODE == kBias, WREG = keeps_w<V, W>(MODE);
  const bool rms = MODE == kRms || (MODE == kBias && q.rms);
  constexpr int K = 3;
  const Part<N, V> part(q.H);
  const size_t step = (size_t)gridDim.x * blockDim.y;
  size_t row = (size_t)blockIdx.x * blockDim.y + threadIdx.y;
  const float inv_h = 1.f / (float)q.H;
  constexpr int MORE = w_places<N, V, W>(MODE);
  char* const mine = RING ? places<N, K>(q.stages, MORE) : nullptr;
  auto start = [&](size_t r, int stage) {
    if constexpr (RING) {
      if (r < (size_t)q.T) {
        const uint32_t to = smem_u32(mine) + stage * (K * N * kPlace);
        const size_t at = r * q.H + part.c0;
        fetch<N, V>(to, static_cast<const Y*>(q.dy) + at, part.live);
        fetch<N, V>(to + N * kPlace, static_cast<const X*>(q.x) + at, part.live);
        if (q.add) fetch<N, V>(to + 2 * N * kPlace, static_cast<const X*>(q.add) + at, part.live);
      }
      copies_commit();
    }
  };
  using WT = std::conditional_t<RING, W, float>;
  Raw<V, WT> w_raw[WREG ? N : 1];
  char* const w_mine = mine + q.stages * (K * N * kPlace);
  if constexpr (RING) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      Raw<V, WT> w;
      if (i < part.live) w.read(static_cast<const WT*>(q.w) + part.c0 + i * (32 * V));
      if constexpr (WREG) w_raw[i] = w;
      else w.keep(w_mine + i * (kWPlaces<V, WT> * kPlace));
    }
  }
  auto read_w = [&](int i, Vec<V>& w) {
    if constexpr (!RING) {
      get_w<V, W>(q, q.w, part.c0 + i * (32 * V), w.v);
    } else if constexpr (WREG) {
      get<V>(w_raw[i].v, w.v);
    } else {
      Raw<V, WT> r;
      r.fetch(w_mine + i * (kWPlaces<V, WT> * kPlace));
      get<V>(r.v, w.v);
    }
  };
  Vec<V> acc_w[N], acc_b[DB ? N : 1];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    acc_w[i] = Vec<V>::all(0.f);
    if constexpr (DB) acc_b[i] = acc_w[i];
  }
  int stage = 0, turn = 0;
  for (int s = 0; s < q.stages; ++s) start(row + s * step, s);
  float2 st = row < (size_t)q.T ? q.stats[row] : make_float2(0.f, 0.f);
  for (; row < (size_t)q.T; row += step) {
    const size_t at = row * q.H + part.c0;
    const char* here = mine + stage * (K * N * kPlace);
    const float mean = st.x, r = st.y;
    if (row + step < (size_t)q.T) st = q.stats[row + step];
    Vec<V> s1 = Vec<V>::all(0.f), s2 = s1;
    const Vec<V> minus_mean = Vec<V>::all(-mean), rv = Vec<V>::all(r);
    // what the second pass needs again: kept in registers without a ring
    Vec<V> kept_y[RING ? 1 : N], kept_x[RING ? 1 : N];
    if constexpr (RING) {
      copies_wait(q.stages - 1);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (i < part.live) {
          get<V>(static_cast<const Y*>(q.dy) + at + i * (32 * V), kept_y[i].v);
          get<V>(static_cast<const X*>(q.x) + at + i * (32 * V), kept_x[i].v);
        }
      }
    }
    auto normal = [&](const Vec<V>& x) { return MODE == kRms ? x * rv : (x + minus_mean) * rv; };
    auto read = [&](int i, Vec<V>& dy, Vec<V>& x) {
      if constexpr (RING) {
        get<V>(reinterpret_cast<const Y*>(here + i * kPlace), dy.v);
        get<V>(reinterpret_cast<const X*>(here + (N + i) * kPlace), x.v);
      } else {
        dy = kept_y[i];
        x = kept_x[i];
      }
    };
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i < part.live) {
        Vec<V> dy, x, w;
        read(i, dy, x);
        read_w(i, w);
        const Vec<V> xh = normal(x), t = dy * w;
        acc_w[i] = fma(dy, xh, acc_w[i]);
        if constexpr (DB) acc_b[i] = acc_b[i] + dy;
        if (MODE != kRms) s1 = s1 + t;
        s2 = fma(t, xh, s2);
      }
    }
    const float2 s = row_sum(s2.sum(), s1.sum(), !rms, turn);
    // dX = r t - xh r mean(t xh) - r mean t + add
    const Vec<V> slope = Vec<V>::all(-r * (s.x * inv_h)),
                 shift = Vec<V>::all(rms ? 0.f : -r * (s.y * inv_h));
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i < part.live) {
        Vec<V> dy, x, w;
        read(i, dy, x);
        read_w(i, w);
        Vec<V> d = fma(dy * w, rv, fma(normal(x), slope, shift));
        if (q.add) {
          Vec<V> a;
          if constexpr (RING) get<V>(reinterpret_cast<const X*>(here + (2 * N + i) * kPlace), a.v);
          else get<V>(static_cast<const X*>(q.add) + at + i * (32 * V), a.v);
          d = d + a;
        }
        put<V>(static_cast<X*>(q.y) + at + i * (32 * V), d.v);
      }
    }
    start(row + q.stages * step, stage);
    if (++stage >= q.stages) stage = 0;
  }
  // this CTA's partial rows: its teams' sums one after another through shared memory
  float* sum_w = reinterpret_cast<float*>(ring);
  float* sum_b = sum_w + q.H;
  if (blockDim.y > 1) {
    if constexpr (RING) copies_wait(0);
    __syncthreads();
  }
  for (int team = 0; team < (int)blockDim.y; ++team) {
    if ((int)threadIdx.y == team) {
      const bool last = team + 1 == (int)blockDim.y;
      float* to_w = last ? q.part_w + (size_t)blockIdx.x * q.H : sum_w;
      float* to_b = last ? q.part_b + (size_t)blockIdx.x * q.H : sum_b;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (i < part.live) {
          const int c = part.c0 + i * (32 * V);
          Vec<V> b;
          if (team) {
            get<V>(sum_w + c, b.v);
            acc_w[i] = acc_w[i] + b;
          }
          put<V>(to_w + c, acc_w[i].v);
          if constexpr (DB) {
            if (team) {
              get<V>(sum_b + c, b.v);
              acc_b[i] = acc_b[i] + b;
            }
            put<V>(to_b + c, acc_b[i].v);
          }
        }
      }
    }
    if (blockDim.y > 1) __syncthreads();
  }
}

// dW and dB from the partial rows: 32 columns a CTA, 32 rows at a time, eight of a thread's loads
// in flight (608 partial rows of 1031 columns: 4 of them 9.6 us).
__global__ void __launch_bounds__(1024) norm_dw_kernel(const NormArgs q) {
  wait_prerequisites();
  const int c = blockIdx.x * 32 + threadIdx.x;
  float w = 0.f, b = 0.f;
  if (c < q.H) {
#pragma unroll 8
    for (int i = threadIdx.y; i < q.parts; i += 32) {
      w += q.part_w[(size_t)i * q.H + c];
      if (q.db) b += q.part_b[(size_t)i * q.H + c];
    }
  }
  __shared__ float2 s[32][33];
  s[threadIdx.y][threadIdx.x] = make_float2(w, b);
  __syncthreads();
  const float2 t = s[threadIdx.x][threadIdx.y];   // the warp of a column
  w = warp_sum(t.x);
  b = warp_sum(t.y);
  const int column = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x || column >= q.H) return;
  if (q.w_bf16) {
    store(static_cast<__nv_bfloat16*>(q.dw) + column, w);
    if (q.db) store(static_cast<__nv_bfloat16*>(q.db) + column, b);
  } else {
    store(static_cast<float*>(q.dw) + column, w);
    if (q.db) store(static_cast<float*>(q.db) + column, b);
  }
}

bool check(const mok_norm_dims* d) {
  return d && d->T >= 0 && d->H >= 1 && d->H <= kMaxH &&
         (d->kind == MOK_NORM_LAYER || d->kind == MOK_NORM_RMS) && std::isfinite(d->eps) &&
         d->eps >= 0.f && is_type(d->x_type) && is_type(d->y_type) && is_type(d->w_type);
}
uintptr_t size_of(mok_out_dtype t) { return t == MOK_OUT_BF16 ? 2 : 4; }
bool whole(const void* p) { return aligned_to(p, 16); }


// How a call runs: teams of bx threads a row, by teams a CTA, `stages` rows in flight per team.
struct Form {
  unsigned bx, by, grid;
  int stages;
  size_t smem;
};
// `more`: places of a thread beyond the ring; `threads` a SM is what the registers allow.
template <int N, int V, int K>
Form form(const mok_norm_dims* d, int more, int threads, int most_ctas) {
  Form f{};
  f.bx = ((d->H + N * V - 1) / (N * V) + 31) / 32 * 32;
  f.by = std::max(1u, 256 / f.bx);
  f.stages = V == 1 ? 0 : d->T <= kSms * (int)f.by ? 1 : 2;   // one, where no team has a second row
  f.smem = V == 1 ? 0 : (size_t)(f.bx * f.by / 32) * (f.stages * K * N + more) * kPlace;
  int ctas = std::max(1, threads / (int)(f.bx * f.by));
  if (f.smem) ctas = std::max(1, std::min(ctas, (int)(kRingBytes / f.smem)));
  f.grid = (unsigned)std::min<size_t>(((size_t)d->T + f.by - 1) / f.by,
                                      std::min(kSms * ctas, most_ctas));
  return f;
}
// Partial rows of dW and dB at most.
int most_parts(const mok_norm_dims* d) { return std::min(d->T, d->H <= 2048 ? kMaxParts : kMaxParts / 2); }

template <auto KERNEL>
cudaError_t run(const Form& f, const NormArgs& q, cudaStream_t s) {
  if (f.smem > 40 * 1024) {   // 48 KB with the static part
    const cudaError_t e = allow_smem<KERNEL>();
    if (e != cudaSuccess) return e;
  }
  return launch(KERNEL, dim3(f.grid), dim3(f.bx, f.by), f.smem, 1, false, s, q);
}

template <typename T>
struct Tag {
  using type = T;
};
template <int N, int V, int THREADS, typename F>
cudaError_t by_types(const mok_norm_dims* d, F f) {
  using B = __nv_bfloat16;
  constexpr std::integral_constant<int, N> n{};
  constexpr std::integral_constant<int, V> v{};
  constexpr std::integral_constant<int, THREADS> t{};
  const bool xb = d->x_type == MOK_OUT_BF16, yb = d->y_type == MOK_OUT_BF16;
  auto with = [&](auto x, auto y) {
    if constexpr (V == 1) return f(n, v, t, x, y, Tag<void>{});
    else if (d->w_type == MOK_OUT_BF16) return f(n, v, t, x, y, Tag<B>{});
    else return f(n, v, t, x, y, Tag<float>{});
  };
  if constexpr (V != 4)
    if (xb && yb) return with(Tag<B>{}, Tag<B>{});
  if constexpr (V != 8) {
    if (xb && !yb) return with(Tag<B>{}, Tag<float>{});
    if (yb && !xb) return with(Tag<float>{}, Tag<B>{});
    return with(Tag<float>{}, Tag<float>{});
  }
  return cudaErrorInvalidValue;
}
// f(accesses a thread, elements an access, most threads of a CTA, X, Y, W) for the call's types,
// width and alignment. `vec`: 32 elements a thread (8 for narrow rows; PER, where a type is fp32)
// in accesses of 16 bytes of the widest type, through a ring for K tensors; element by element where
// rows are not aligned, or too wide for the ring and w.
template <int K, int PER, typename F>
cudaError_t by_form(const mok_norm_dims* d, bool vec, F f) {
  const bool wide = d->x_type != MOK_OUT_BF16 || d->y_type != MOK_OUT_BF16;
  // places of 32 elements of each: 4 or 8 accesses of K tensors twice, and of w
  const int places = (wide ? 8 : 4) * (2 * K + (wide || d->w_type == MOK_OUT_BF16 ? 1 : 2));
  if ((size_t)((d->H + 1023) / 1024) * places * kPlace > kRingBytes) vec = false;
  if (!vec) {
    if (d->H <= 1536) return by_types<6, 1, 256>(d, f);   // 2371 x 1031 fp32, bias: 29 us of eight, 25
    if (d->H <= 8192) return by_types<8, 1, 1024>(d, f);
    return by_types<32, 1, 1024>(d, f);
  }
  if (wide) {
    if (d->H <= 256) return by_types<2, 4, 256>(d, f);
    if (d->H <= 8192) return by_types<PER / 4, 4, 8192 / PER>(d, f);
    return by_types<8, 4, 1024>(d, f);
  }
  if (d->H <= 256) return by_types<1, 8, 256>(d, f);
  if (d->H <= 8192) return by_types<4, 8, 256>(d, f);
  return by_types<4, 8, 1024>(d, f);
}

}  // namespace
}  // namespace mok

extern "C" mok_status mok_norm_get_sizes(const mok_norm_dims* d, mok_norm_sizes* out) {
  using namespace mok;
  if (!check(d) || !out) return MOK_ERR_INVALID_ARG;
  out->stats_bytes = (size_t)d->T * sizeof(float2);
  out->workspace_bytes = align_up((size_t)most_parts(d) * d->H * sizeof(float2), 256) + 256;
  return MOK_OK;
}

extern "C" mok_status mok_norm_fwd(const mok_norm_dims* d, const void* x, const void* add,
                                   const void* w, const void* b, void* h, void* y, float* stats,
                                   void* stream) {
  using namespace mok;
  if (!check(d)) return MOK_ERR_INVALID_ARG;
  if (d->T == 0) return MOK_OK;
  if (!x || !w || !y || (add == nullptr) != (h == nullptr)) return MOK_ERR_INVALID_ARG;
  const uintptr_t xs = size_of(d->x_type), ws = size_of(d->w_type);
  if (!aligned_to(x, xs) || !aligned_to(add, xs) || !aligned_to(h, xs) || !aligned_to(w, ws) ||
      !aligned_to(b, ws) || !aligned_to(y, size_of(d->y_type)) || !aligned_to(stats, 8))
    return MOK_ERR_INVALID_ARG;
  NormArgs q{};
  q.T = d->T; q.H = d->H; q.eps = d->eps;
  q.rms = d->kind == MOK_NORM_RMS; q.w_bf16 = d->w_type == MOK_OUT_BF16;
  q.x = x; q.add = add; q.w = w; q.b = b; q.h = h; q.y = y;
  q.stats = reinterpret_cast<float2*>(stats);
  const bool vec = d->H % 8 == 0 && whole(x) && whole(add) && whole(w) && whole(b) && whole(h) &&
                   whole(y);
  const cudaError_t e = by_form<2, 32>(d, vec, [&](auto n, auto v, auto threads, auto xt, auto yt, auto wt) {
    constexpr int N = decltype(n)::value, V = decltype(v)::value, THREADS = decltype(threads)::value;
    constexpr int CTAS = THREADS == 1024 ? 1 : V == 1 ? 5 : 3;
    const Form f = form<N, V, 2>(d, 0, THREADS * CTAS, INT_MAX);
    q.stages = f.stages;
    return run<norm_fwd_kernel<N, V, typename decltype(xt)::type, typename decltype(yt)::type,
                               typename decltype(wt)::type, THREADS, CTAS>>(
        f, q, static_cast<cudaStream_t>(stream));
  });
  return e == cudaSuccess ? MOK_OK : MOK_ERR_CUDA;
}

extern "C" mok_status mok_norm_bwd(const mok_norm_dims* d, const void* dY, const void* h,
                                   const void* w, const float* stats, const void* add, void* dX,
                                   void* dW, void* dB, void* workspace, void* stream) {
  using namespace mok;
  if (!check(d)) return MOK_ERR_INVALID_ARG;
  const uintptr_t xs = size_of(d->x_type), ws = size_of(d->w_type);
  if (!dW || !aligned_to(dW, ws) || !aligned_to(dB, ws)) return MOK_ERR_INVALID_ARG;
  if (d->T > 0) {
    if (!dY || !h || !w || !stats || !dX) return MOK_ERR_INVALID_ARG;
    if (!aligned_to(dY, size_of(d->y_type)) || !aligned_to(h, xs) || !aligned_to(add, xs) ||
        !aligned_to(dX, xs) || !aligned_to(w, ws) || !aligned_to(stats, 8))
      return MOK_ERR_INVALID_ARG;
  }
  if (!workspace || !aligned_to(workspace, 256)) return MOK_ERR_WORKSPACE;
  NormArgs q{};
  q.T = d->T; q.H = d->H;
  q.rms = d->kind == MOK_NORM_RMS; q.w_bf16 = d->w_type == MOK_OUT_BF16;
  q.dy = dY; q.x = h; q.w = w; q.add = add; q.y = dX; q.dw = dW; q.db = dB;
  q.stats = reinterpret_cast<float2*>(const_cast<float*>(stats));
  q.part_w = static_cast<float*>(workspace);
  q.part_b = q.part_w + (size_t)most_parts(d) * d->H;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d->T) {
    const bool vec = d->H % 8 == 0 && whole(dY) && whole(h) && whole(w) && whole(add) && whole(dX);
    const cudaError_t e = by_form<3, 16>(d, vec, [&](auto n, auto v, auto threads, auto xt, auto yt, auto wt) {
      constexpr int N = decltype(n)::value, V = decltype(v)::value, THREADS = decltype(threads)::value;
      constexpr int CTAS = THREADS > 256 ? 1 : V == 1 ? 3 : 2;
      using X = typename decltype(xt)::type;
      using Y = typename decltype(yt)::type;
      using W = typename decltype(wt)::type;
      auto go = [&](auto mode) {
        constexpr int MODE = decltype(mode)::value;
        Form f = form<N, V, 3>(d, w_places<N, V, W>(MODE), THREADS * CTAS, most_parts(d));
        if (f.by > 1) f.smem = std::max(f.smem, (size_t)d->H * sizeof(float2));   // joins the teams
        q.stages = f.stages;
        q.parts = (int)f.grid;
        return run<norm_bwd_kernel<N, V, X, Y, W, MODE, THREADS, CTAS>>(f, q, s);
      };
      if (dB) return go(std::integral_constant<int, kBias>{});
      if (q.rms) return go(std::integral_constant<int, kRms>{});
      return go(std::integral_constant<int, kMeans>{});
    });
    if (e != cudaSuccess) return MOK_ERR_CUDA;
  }
  const cudaError_t e = launch(norm_dw_kernel, dim3((d->H + 31) / 32), dim3(32, 32), 0, 1, d->T > 0, s, q);
  return e == cudaSuccess ? MOK_OK : MOK_ERR_CUDA;
}
