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
  int part_row;                  // elements of a partial row
  unsigned shift_mask;           // a partial row i lies (i H) & shift_mask elements behind its place
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
template <int N, int V, typename W, bool SHIFT>
constexpr int fwd_places() {   // of a forward kernel: for w and b, where rows are shifted
  if constexpr (SHIFT) return 2 * N * kWPlaces<V, W>;
  else return 0;
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
// lie in the row. SHIFT: rows of any length, in accesses of a tensor that begins at a 16-byte boundary. A
// row then begins `shift` elements behind one, and its first and last access hold other rows'
// elements too (edge), which count as 0 and are not written. The rows of a team are a multiple of V
// apart and so have one shift.
template <int N, int V, bool SHIFT>
struct Part {
  int c0, live, shift, end;
  // Long parts: the accesses where a lane of the warp has an edge; the rest branches around what edges
  // take (8192 x 7167 fp32 with add forward 144 us, 157 without). Short ones gain nothing.
  static constexpr bool VOTE = SHIFT && N * V >= 32;
  uint32_t edges = 0;
  __device__ __forceinline__ Part(int H, size_t first_row) {
    shift = SHIFT ? (int)(first_row * H % V) : 0;
    end = H + shift;
    c0 = (int)(threadIdx.x >> 5) * (32 * N * V) + (int)(threadIdx.x & 31) * V;
    live = c0 < end ? min(N, (end - c0 + 32 * V - 1) / (32 * V)) : 0;
    if constexpr (VOTE) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (__any_sync(kAll, outer(i))) edges |= 1u << i;
    }
  }
  __device__ __forceinline__ int at(int i) const { return c0 + i * (32 * V); }
  __device__ __forceinline__ bool outer(int i) const { return at(i) < shift || at(i) + V > end; }
  __device__ __forceinline__ bool edge(int i) const {
    return VOTE ? edges >> i & 1u : SHIFT && outer(i);
  }
  __device__ __forceinline__ bool holds(int i, int j) const {
    return !SHIFT || (at(i) + j >= shift && at(i) + j < end);
  }
  __device__ __forceinline__ void clear(int i, Vec<V>& v) const {
    if (!edge(i)) return;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (!holds(i, j)) v.v[j] = 0.f;
  }
  // p: the row's tensor at c0
  template <typename E>
  __device__ __forceinline__ void write(int i, E* p, const Vec<V>& v) const {
    if (!edge(i) || (VOTE && !outer(i))) {
      put<V>(p + i * (32 * V), v.v);
      return;
    }
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (holds(i, j)) store(p + i * (32 * V) + j, v.v[j]);
  }
  // Starts the copies of a row (p: its tensor at c0) to `to` on; nothing behind its end is read.
  template <typename E>
  __device__ __forceinline__ void fetch(uint32_t to, const E* p) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i >= live) continue;
      constexpr int bytes = V * (int)sizeof(E);
      if (VOTE ? edge(i) : SHIFT)
        copy_async<bytes>(to + i * kPlace, p + i * (32 * V), min(V, end - at(i)) * (int)sizeof(E));
      else copy_async<bytes>(to + i * kPlace, p + i * (32 * V));
    }
  }
  // The parameter's elements of access i.
  template <typename W>
  __device__ __forceinline__ void parameter(int i, const W* w, Raw<V, W>& r) const {
    if constexpr (!SHIFT) {
      r.read(w + at(i));
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) r.v[j] = holds(i, j) ? w[at(i) + j - shift] : W(0.f);
    }
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
// RING: V elements a copy, 16 bytes at most; else V = 1, any alignment. 8192 x 7168 with add: bf16 78.7 us
// (6.0 TB/s, two streams in and two out), fp32 144 us (6.5 TB/s), 8192 x 7167 bf16 76.7 us.
template <int N, int V, typename X, typename Y, typename W, bool SHIFT, int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) norm_fwd_kernel(const NormArgs q) {
  constexpr bool RING = V > 1;
  constexpr int K = 2;
  const size_t step = (size_t)gridDim.x * blockDim.y;
  size_t row = (size_t)blockIdx.x * blockDim.y + threadIdx.y;
  const Part<N, V, SHIFT> part(q.H, row);
  const float inv_h = 1.f / (float)q.H;
  char* const mine = RING ? places<N, K>(q.stages, fwd_places<N, V, W, SHIFT>()) : nullptr;
  auto start = [&](size_t r, int stage) {
    if constexpr (RING) {
      if (r < (size_t)q.T) {
        const uint32_t to = smem_u32(mine) + stage * (K * N * kPlace);
        const size_t at = r * q.H + part.c0 - part.shift;
        part.fetch(to, static_cast<const X*>(q.x) + at);
        if (q.add) part.fetch(to + N * kPlace, static_cast<const X*>(q.add) + at);
      }
      copies_commit();
    }
  };
  int stage = 0, turn = 0;
  for (int s = 0; s < q.stages; ++s) start(row + s * step, s);
  using WT = std::conditional_t<RING, W, float>;
  char* const w_mine = mine + q.stages * (K * N * kPlace);
  constexpr int W_STEP = kWPlaces<V, WT> * kPlace;
  if constexpr (SHIFT) {   // parameters in no row's alignment: taken apart once, kept
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i >= part.live) continue;
      Raw<V, WT> r;
      part.parameter(i, static_cast<const WT*>(q.w), r);
      r.keep(w_mine + i * W_STEP);
      if (q.b) {
        part.parameter(i, static_cast<const WT*>(q.b), r);
        r.keep(w_mine + (N + i) * W_STEP);
      }
    }
  } else if constexpr (RING) {   // the first row's second trip to memory, made beside its first
    const int size = q.w_bf16 ? 2 : 4;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i < part.live) {
        const size_t c = (size_t)part.at(i) * size;
        prefetch_l1(static_cast<const char*>(q.w) + c);
        if (q.b) prefetch_l1(static_cast<const char*>(q.b) + c);
      }
    }
  }
  for (; row < (size_t)q.T; row += step) {
    const size_t at = row * q.H + part.c0 - part.shift;
    const char* here = mine + stage * (K * N * kPlace);
    Vec<V> v[N];
    if constexpr (RING) copies_wait(q.stages - 1);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = Vec<V>::all(0.f);
      if (i < part.live) {
        get<V>(RING ? reinterpret_cast<const X*>(here + i * kPlace)
                    : static_cast<const X*>(q.x) + at + i * (32 * V), v[i].v);
        part.clear(i, v[i]);
      }
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
            part.clear(i, a);
            v[i] = v[i] + a;
          } else {
            v[i] = v[i] + kept[i];
          }
          if constexpr (sizeof(X) == 2) {   // the norm is that of the stored h
#pragma unroll
            for (int j = 0; j < V; ++j) v[i].v[j] = __bfloat162float(__float2bfloat16_rn(v[i].v[j]));
          }
          part.write(i, static_cast<X*>(q.h) + at, v[i]);
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
      for (int i = 0; i < N; ++i) {
        if (i < part.live) {
          v[i] = v[i] + minus;
          part.clear(i, v[i]);
        }
      }
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
        Vec<V> w, b = Vec<V>::all(0.f);
        if constexpr (SHIFT) {
          Raw<V, WT> r;
          r.fetch(w_mine + i * W_STEP);
          get<V>(r.v, w.v);
          if (q.b) {
            r.fetch(w_mine + (N + i) * W_STEP);
            get<V>(r.v, b.v);
          }
        } else {
          get_w<V, W>(q, q.w, part.at(i), w.v);
          if (q.b) get_w<V, W>(q, q.b, part.at(i), b.v);
        }
        part.write(i, static_cast<Y*>(q.y) + at, fma(v[i] * rv, w, b));
      }
    }
  }
}

// Words that the sums of a row take in shared memory.
__host__ __device__ constexpr int join_row(int H) { return H + H / 32 + 1; }

// The parameters are read once: w stays in registers in the type it has, or, where dB's sums need
// those, in the thread's own places of shared memory. (Read again for every row through L1, twice,
// they made up a fifth of the kernel's time: 8192 x 7168 bf16 with add 95.6 us.) With the sum of the
// partial rows that is now 77.0 us (6.1 TB/s), fp32 139 us (6.8 TB/s), 8192 x 7167 bf16 92.4 us.
template <int N, int V, typename X, typename Y, typename W, bool SHIFT, int MODE, int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) norm_bwd_kernel(const NormArgs q) {
  launch_dependents();
  constexpr bool RING = V > 1, DB = MODE == kBias, WREG = keeps_w<V, W>(MODE);
  const bool rms = MODE == kRms || (MODE == kBias && q.rms);
  constexpr int K = 3;
  const size_t step = (size_t)gridDim.x * blockDim.y;
  size_t row = (size_t)blockIdx.x * blockDim.y + threadIdx.y;
  const Part<N, V, SHIFT> part(q.H, row);
  const float inv_h = 1.f / (float)q.H;
  constexpr int MORE = w_places<N, V, W>(MODE);
  char* const mine = RING ? places<N, K>(q.stages, MORE) : nullptr;
  auto start = [&](size_t r, int stage) {
    if constexpr (RING) {
      if (r < (size_t)q.T) {
        const uint32_t to = smem_u32(mine) + stage * (K * N * kPlace);
        const size_t at = r * q.H + part.c0 - part.shift;
        part.fetch(to, static_cast<const Y*>(q.dy) + at);
        part.fetch(to + N * kPlace, static_cast<const X*>(q.x) + at);
        if (q.add) part.fetch(to + 2 * N * kPlace, static_cast<const X*>(q.add) + at);
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
      if (i < part.live) part.parameter(i, static_cast<const WT*>(q.w), w);
      if constexpr (WREG) w_raw[i] = w;
      else w.keep(w_mine + i * (kWPlaces<V, WT> * kPlace));
    }
  }
  auto read_w = [&](int i, Vec<V>& w) {
    if constexpr (!RING) {
      get_w<V, W>(q, q.w, part.at(i), w.v);
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
    const size_t at = row * q.H + part.c0 - part.shift;
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
        part.clear(i, dy);
        part.clear(i, x);
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
        part.write(i, static_cast<X*>(q.y) + at, d);
      }
    }
    start(row + q.stages * step, stage);
    if (++stage >= q.stages) stage = 0;
  }
  // This CTA's partial rows: a single team's as it holds them, several teams' summed up in shared
  // memory, where 33 words hold 32 columns, so that a warp's places lie in different banks.
  if (blockDim.y == 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i >= part.live) continue;
      const size_t to = (size_t)blockIdx.x * q.part_row + part.at(i);
      put<V>(q.part_w + to, acc_w[i].v);
      if constexpr (DB) put<V>(q.part_b + to, acc_b[i].v);
    }
    return;
  }
  const int teams = blockDim.y, threads = blockDim.x * teams, pitch = join_row(q.H);
  float* sum_w = reinterpret_cast<float*>(ring);
  float* sum_b = sum_w + teams * pitch;
  if constexpr (RING) copies_wait(0);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = part.at(i) + j - part.shift, to = threadIdx.y * pitch + c + (c >> 5);
      if (i >= part.live || !part.holds(i, j)) continue;
      sum_w[to] = acc_w[i].v[j];
      if constexpr (DB) sum_b[to] = acc_b[i].v[j];
    }
  }
  __syncthreads();
  for (int c = threadIdx.y * blockDim.x + threadIdx.x; c < q.H; c += threads) {
    float w = 0.f, b = 0.f;
    for (int t = 0; t < teams; ++t) {
      w += sum_w[t * pitch + c + (c >> 5)];
      if constexpr (DB) b += sum_b[t * pitch + c + (c >> 5)];
    }
    q.part_w[(size_t)blockIdx.x * q.part_row + c] = w;
    if constexpr (DB) q.part_b[(size_t)blockIdx.x * q.part_row + c] = b;
  }
}

// dW and dB from the partial rows, COLS columns a CTA. Bound by the latency of its loads: eight of a
// thread's are in flight (with four, 608 partial rows of 1031 columns took 9.6 us).
template <int COLS>
__global__ void __launch_bounds__(1024) norm_dw_kernel(const NormArgs q) {
  constexpr int ROWS = 1024 / COLS;
  wait_prerequisites();
  const int x = threadIdx.x % COLS, y = threadIdx.x / COLS, c = blockIdx.x * COLS + x;
  float w = 0.f, b = 0.f;
  if (c < q.H) {
#pragma unroll 8
    for (int i = y; i < q.parts; i += ROWS) {
      const size_t at = (size_t)i * q.part_row + c + ((unsigned)i * (unsigned)q.H & q.shift_mask);
      w += q.part_w[at];
      if (q.db) b += q.part_b[at];
    }
  }
  __shared__ float2 s[ROWS][COLS + 1];
  s[y][x] = make_float2(w, b);
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;   // a warp of a column
  const int column = blockIdx.x * COLS + warp;
  if (warp >= COLS || column >= q.H) return;
  w = b = 0.f;
#pragma unroll
  for (int i = 0; i < ROWS / 32; ++i) {
    const float2 t = s[i * 32 + lane][warp];
    w += t.x;
    b += t.y;
  }
  w = warp_sum(w);
  b = warp_sum(b);
  if (lane) return;
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
  f.bx = ((d->H + (d->H % 8 ? V - 1 : 0) + N * V - 1) / (N * V) + 31) / 32 * 32;   // room for a shift
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

// Elements of a partial row, with room for a shift.
int part_row(const mok_norm_dims* d) { return (d->H + 15) / 8 * 8; }

template <typename T>
struct Tag {
  using type = T;
};
template <int N, int V, bool SHIFT, int THREADS, typename F>
cudaError_t by_types(const mok_norm_dims* d, F f) {
  using B = __nv_bfloat16;
  constexpr std::integral_constant<int, N> n{};
  constexpr std::integral_constant<int, V> v{};
  constexpr std::integral_constant<int, THREADS> t{};
  constexpr std::bool_constant<SHIFT> shift{};
  const bool xb = d->x_type == MOK_OUT_BF16, yb = d->y_type == MOK_OUT_BF16;
  auto with = [&](auto x, auto y) {
    if constexpr (V == 1) return f(n, v, shift, t, x, y, Tag<void>{});
    else if (d->w_type == MOK_OUT_BF16) return f(n, v, shift, t, x, y, Tag<B>{});
    else return f(n, v, shift, t, x, y, Tag<float>{});
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
// f(accesses a thread, elements an access, shift, most threads of a CTA, X, Y, W) for the call's types,
// width and alignment. `whole_rows`: tensors of rows begin at 16-byte boundaries; then accesses of 16
// bytes of the widest type through a ring for K tensors, PER (where a type is fp32) or 32 elements a
// thread, fewer of narrow rows; shifted where rows begin between boundaries, or the parameters do
// (not `whole_w`). Element by element where tensors begin between boundaries, or rows are too wide for
// the ring: above 2048 elements 32 a thread of 1024, whose 64 registers spill (200 bytes each way forward,
// 440 to 700 out and 800 to 1200 back in backward). Forward and backward, bf16 with add, us: 8192 x 7167 shifted 76 and 92, element by element
// 159 and 289. Shifted rows forward, 16 and 32 elements a thread: 8192 x 2047 bf16 29 and 34, fp32 38
// and 73, 8192 x 7167 bf16 83 and 76, fp32 174 and 145; backward: 32768 x 511 with dB 50 and 72 (spills).
template <int K, int PER, typename F>
cudaError_t by_form(const mok_norm_dims* d, bool whole_rows, bool whole_w, F f) {
  const bool wide = d->x_type != MOK_OUT_BF16 || d->y_type != MOK_OUT_BF16;
  const bool shift = d->H % 8 != 0 || !whole_w;
  // a warp's places for 1024 elements of K tensors twice, and of what a kernel may keep of w and b
  const int kept = K == 3 ? 1 : shift ? 2 : 0;
  const int places = (wide ? 8 : 4) * (2 * K + kept * (wide || d->w_type == MOK_OUT_BF16 ? 1 : 2));
  const int warps = (d->H + (shift ? 7 : 0) + 1023) / 1024;
  const bool vec = whole_rows && (size_t)warps * places * kPlace <= kRingBytes;
  if (!vec) {
    if (d->H <= 2048) return by_types<8, 1, false, 256>(d, f);
    return by_types<32, 1, false, 1024>(d, f);
  }
  const bool broad = warps > 8;
  if (wide) {
    if (shift && d->H <= 2040) return by_types<2, 4, true, 256>(d, f);
    if (shift && (d->H <= 4088 || K == 3) && !broad) return by_types<4, 4, true, 512>(d, f);
    if constexpr (K == 2)
      if (shift && !broad) return by_types<8, 4, true, 256>(d, f);
    if (shift) return by_types<32, 1, false, 1024>(d, f);
    if (d->H <= 256) return by_types<2, 4, false, 256>(d, f);
    if constexpr (K == 2)
      if (broad) return by_types<8, 4, false, 512>(d, f);   // 14 warps at most; the backward's 8 are not broad
    return by_types<PER / 4, 4, false, 8192 / PER>(d, f);
  }
  if constexpr (K == 2)
    if (shift && !broad && d->H > 4088) return by_types<4, 8, true, 256>(d, f);
  if (shift && !broad) return by_types<2, 8, true, 512>(d, f);
  if (shift) return by_types<32, 1, false, 1024>(d, f);
  if (d->H <= 256) return by_types<1, 8, false, 256>(d, f);
  if (d->H <= 512) return by_types<2, 8, false, 256>(d, f);
  if (!broad) return by_types<4, 8, false, 256>(d, f);
  return by_types<4, 8, false, K == 2 ? 1024 : 512>(d, f);   // the backward's w takes it to 16 warps at most
}

}  // namespace
}  // namespace mok

extern "C" mok_status mok_norm_get_sizes(const mok_norm_dims* d, mok_norm_sizes* out) {
  using namespace mok;
  if (!check(d) || !out) return MOK_ERR_INVALID_ARG;
  out->stats_bytes = (size_t)d->T * sizeof(float2);
  out->workspace_bytes = align_up((size_t)most_parts(d) * part_row(d) * sizeof(float2), 256) + 256;
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
  const bool whole_rows = whole(x) && whole(add) && whole(h) && whole(y), whole_w = whole(w) && whole(b);
  const cudaError_t e = by_form<2, 32>(d, whole_rows, whole_w, [&](auto n, auto v, auto sh, auto threads, auto xt, auto yt,
                                                                auto wt) {
    constexpr int N = decltype(n)::value, V = decltype(v)::value, THREADS = decltype(threads)::value;
    constexpr bool SHIFT = decltype(sh)::value;
    using W = typename decltype(wt)::type;
    constexpr int CTAS = THREADS > 512 ? 1 : SHIFT ? (N * V == 32 ? 2 : 1024 / THREADS)
                         : THREADS > 256 ? 1 : V == 1 ? 5 : N < 4 ? 4 : 3;
    const Form f = form<N, V, 2>(d, fwd_places<N, V, W, SHIFT>(), THREADS * CTAS, INT_MAX);
    q.stages = f.stages;
    return run<norm_fwd_kernel<N, V, typename decltype(xt)::type, typename decltype(yt)::type, W, SHIFT,
                               THREADS, CTAS>>(f, q, static_cast<cudaStream_t>(stream));
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
  q.part_row = part_row(d);
  q.part_b = q.part_w + (size_t)most_parts(d) * q.part_row;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d->T) {
    const bool whole_rows = whole(dY) && whole(h) && whole(add) && whole(dX);
    const cudaError_t e = by_form<3, 16>(d, whole_rows, whole(w), [&](auto n, auto v, auto sh, auto threads, auto xt,
                                                                  auto yt, auto wt) {
      constexpr int N = decltype(n)::value, V = decltype(v)::value, THREADS = decltype(threads)::value;
      constexpr bool SHIFT = decltype(sh)::value;
      constexpr int CTAS = THREADS > 256 ? 1 : V == 1 || N * V == 8 ? 3 : 2;
      using X = typename decltype(xt)::type;
      using Y = typename decltype(yt)::type;
      using W = typename decltype(wt)::type;
      auto go = [&](auto mode) {
        constexpr int MODE = decltype(mode)::value;
        Form f = form<N, V, 3>(d, w_places<N, V, W>(MODE), THREADS * CTAS, most_parts(d));
        if (f.by > 1)   // joins the teams
          f.smem = std::max(f.smem, f.by * join_row(d->H) * (MODE == kBias ? sizeof(float2) : sizeof(float)));
        q.stages = f.stages;
        q.parts = (int)f.grid;
        q.shift_mask = SHIFT && f.by == 1 ? V - 1 : 0;   // several teams are joined at their places
        return run<norm_bwd_kernel<N, V, X, Y, W, SHIFT, MODE, THREADS, CTAS>>(f, q, s);
      };
      if (dB) return go(std::integral_constant<int, kBias>{});
      if (q.rms) return go(std::integral_constant<int, kRms>{});
      return go(std::integral_constant<int, kMeans>{});
    });
    if (e != cudaSuccess) return MOK_ERR_CUDA;
  }
  // backward with 16 columns a CTA and with 32, us: 2371 x 1031 fp32 11.3 and 13.2, 8192 x 4096 bf16 39.2 and
  // 39.8, 512 x 7168 13.2 and 11.1
  const bool narrow = d->H <= 4096;
  const cudaError_t e = launch(narrow ? norm_dw_kernel<16> : norm_dw_kernel<32>,
                               dim3(narrow ? (d->H + 15) / 16 : (d->H + 31) / 32), dim3(1024), 0, 1, d->T > 0, s, q);
  return e == cudaSuccess ? MOK_OK : MOK_ERR_CUDA;
}
