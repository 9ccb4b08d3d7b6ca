// Low-rank adapters of many requests beside a shared projection (include/mok_ops.h,
// mok_lora_fwd and mok_lora_bwd).
//
//   u_t = scale_a xa_t A_a^T     y_t  = x_t W    + u_t B_a          (a = ids[t])
//   v_t = scale_a dY_t B_a^T     dX_t = dY_t W^T + v_t A_a
//   dA_a = sum_t v_t^T xa_t      dB_a = sum_t u_t^T dY_t            (t with ids[t] = a)
//
// Two kernels serve both directions, because A [n][r][K] and B [n][r][N] have one form:
//
//   shrink_kernel   the r values of every row (u or v): 128 rows against the A (or B) rows of
//                   the distinct adapters among them, side by side in one MMA; each row keeps
//                   the columns of its own adapter.
//   proj_kernel     the shared projection, whose K loop simply goes on after W: one step per
//                   distinct adapter of the row tile, [hi(u) | lo(u)] against that adapter's
//                   B (or A) rows, into the same TMEM accumulator. The MMA's lane mask
//                   (disable-output-lane) confines a step to the rows of its adapter. So rows
//                   of different requests share a tile in any order, with no sorting and no
//                   padding, the projection is one pass, and an adapter with an inf or NaN
//                   cannot reach another request's rows.
//
// (shrink_rows_kernel finds u for small batches.) The weight gradients sum over the rows of one
// adapter: bucket_kernel lists each adapter's rows in ascending order, wgrad_kernel gathers them.
//
// u and v are kept as two bf16 values, hi = u cut to bf16 and lo = bf16(u - hi): the tensor
// cores take bf16, and the pair carries 16 significant bits, so the low-rank path adds no
// visible rounding to the bf16 inputs and results. Per 32 ranks a row holds 128 bytes: 32 hi,
// then 32 lo values.
//
// Every mbarrier wait is bounded (kTimeoutNs); on expiry the kernel sets the status word,
// lets its copies and MMAs in flight finish, and returns.
#include <algorithm>
#include <atomic>
#include <mutex>
#include <type_traits>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "mok_internal.h"
#include "mok_ops.h"
#include "mok_profile.h"
#include "mok_ptx.cuh"

namespace mok {
namespace {

constexpr int BM = 128;                 // rows of a tile (TMEM lanes)
constexpr int BK = 64;                  // contraction elements per pipeline stage
constexpr int A_BYTES = BM * BK * 2;    // 16 KB: 128 rows x 128 bytes
constexpr int kThreads = 192;           // producer warp, MMA warp, four epilogue warps
constexpr int kMaxStages = 16;
constexpr int kStagingBox = 4096;       // 32 rows x 128 bytes, one epilogue store
constexpr int kBarBytes = 512;
constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr size_t kMaxSmem = 227 * 1024;

// A distinct adapter of a row tile (or of a pair of them): its id and the lanes (rows) that do
// NOT use it, four words for each of the row tiles.
struct Slot {
  int32_t id;
  int32_t pad[3];
  uint4 off[2];
};

__device__ __forceinline__ void flag_timeout(uint32_t* status) {
  if (status != nullptr) atomicOr(status, kErrTimeout);
}
// mbar_wait whose deadline is taken only when the wait turns out long
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity) {
  for (int i = 0; i < 64; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return mbar_wait(bar, parity, globaltimer_ns() + kTimeoutNs);
}
// One lane of a converged warp, always the same one. The roles that issue TMA and MMA run as
// whole warps and elect a lane only around those instructions: everything else is then
// provably uniform, so their operands sit in uniform registers. (With the loops themselves
// under "lane == 0" one step took 650 clocks to issue, longer than its MMAs: 0.33 us in every
// shape.)
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred P;\n\t"
      "elect.sync _|P, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, P;\n\t}"
      : "=r"(p));
  return p != 0;
}

// tcgen05.mma (kind::f16) that leaves the accumulator rows (TMEM lanes) of `off` untouched:
// bit i of word j stands for lane 32 j + i.
__device__ __forceinline__ void umma_bf16_rows(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc,
                                               uint32_t idesc, const uint4 off,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, {%5, %6, %7, %8}, p;\n\t}" ::"r"(
          tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(off.x), "r"(off.y), "r"(off.z),
      "r"(off.w)
      : "memory");
}
// The same for an SM pair (M = 256): words 0-3 are the even CTA's lanes, 4-7 the odd one's.
__device__ __forceinline__ void umma_bf16_rows_pair(uint32_t tmem_d, uint64_t adesc,
                                                    uint64_t bdesc, uint32_t idesc,
                                                    const uint4 off0, const uint4 off1,
                                                    uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, {%5, %6, %7, %8, %9, %10, %11, "
      "%12}, p;\n\t}" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(off0.x), "r"(off0.y), "r"(off0.z),
      "r"(off0.w), "r"(off1.x), "r"(off1.y), "r"(off1.z), "r"(off1.w)
      : "memory");
}
// 3-D tiled load: c0 innermost (elements), then c1, c2.
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* m, uint64_t* bar,
                                            int32_t c0, int32_t c1, int32_t c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
      : "memory");
}
// ... completing on an mbarrier of either CTA of a pair (bar: from mapa_rank).
__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* m, uint32_t bar,
                                                 int32_t c0, int32_t c1, int32_t c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}
// Programmatic dependent launch: let the next kernel of the stream start its own set-up, and
// wait until the kernels before this one have finished and their writes are visible.
__device__ __forceinline__ void launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_prerequisites() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
// 16 consecutive TMEM columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float* v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
// 4 floats from the shared memory of CTA `rank` of the cluster (p: this CTA's address).
// Volatile, so it stays between the cluster barriers around it; several may be in flight.
__device__ __forceinline__ float4 ld_rank4(const float* p, uint32_t rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(mapa_rank(p, rank)));
  return v;
}
// Sum over the ranks 0 .. n - 1 (n <= 8) in rank order, all loads issued before the first add.
__device__ __forceinline__ float4 sum_ranks(const float* p, int n) {
  float4 v[8];
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (k < n) v[k] = ld_rank4(p, k);
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (k < n) {
      s.x += v[k].x; s.y += v[k].y; s.z += v[k].z; s.w += v[k].w;
    }
  return s;
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// hi and lo of two neighbours. hi is cut towards zero, and lo, which then has hi's sign, is never 0
// beside a hi that is not (2^-24 of it, below fp32's rounding, where nothing is left), and is
// infinite with hi: so hi x + lo x is infinite where u x is, and NaN only where that is NaN.
__device__ __forceinline__ float low_part(float a, float hi) {
  const float rest = a - hi;
  return isinf(a) ? a : rest != 0.f ? rest : hi * 0x1p-24f;
}
__device__ __forceinline__ void split_pair(float a, float b, uint32_t& hi, uint32_t& lo) {
  const uint32_t ha = __float_as_uint(a) & 0xffff0000u, hb = __float_as_uint(b) & 0xffff0000u;
  hi = ha >> 16 | hb;
  lo = pack_bf16(low_part(a, __uint_as_float(ha)), low_part(b, __uint_as_float(hb)));
}

// ------------------------------------------------------------------ barriers of a CTA
struct Bars {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drain;
  uint32_t tmem;
  volatile int abort;
};
static_assert(sizeof(Bars) <= kBarBytes, "barrier area");

// pair: one arrival per epilogue warp of both CTAs hands an accumulator back
__device__ __forceinline__ void init_bars(Bars* b, bool pair = false) {
  for (int s = 0; s < kMaxStages; ++s) {
    mbar_init(&b->full[s], 1);
    mbar_init(&b->empty[s], 1);
  }
  for (int a = 0; a < 2; ++a) {
    mbar_init(&b->acc_full[a], 1);
    mbar_init(&b->acc_empty[a], pair ? 8 : 128);
  }
  mbar_init(&b->drain, 1);
  b->abort = 0;
  fence_mbar_init();
}

// The ring of pipeline stages as one role (producer or MMA warp) walks it.
struct Ring {
  int stages;
  int stage = 0;
  uint32_t phase = 0;
  uint32_t used = 0;     // stages filled so far (producer)
  __device__ explicit Ring(int n) : stages(n) {}
  __device__ __forceinline__ void next() {
    ++used;
    if (++stage == stages) {
      stage = 0;
      phase ^= 1;
    }
  }
};

// A wait of a whole warp; every lane gets the same answer. False: the wait passed its bound
// (the status word is set) or another warp's did.
__device__ __noinline__ bool warp_wait_long(Bars* b, uint64_t* bar, uint32_t parity,
                                            uint32_t* status) {
  uint64_t deadline = 0;
  bool done = false;
  for (uint32_t i = 1;; ++i) {
    done = done || mbar_try_wait(bar, parity);
    if (__all_sync(0xffffffffu, done)) return true;
    if (i % 64 == 0) {
      const uint64_t now = globaltimer_ns();
      if (deadline == 0) deadline = now + kTimeoutNs;
      const bool late = now > deadline;
      if (late && !b->abort) flag_timeout(status);
      if (late) b->abort = 1;
      if (__any_sync(0xffffffffu, late || b->abort)) return false;
    }
  }
}
__device__ __forceinline__ bool warp_wait(Bars* b, uint64_t* bar, uint32_t parity,
                                          uint32_t* status) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return warp_wait_long(b, bar, parity, status);
}
// After an abort: every copy that was issued has landed (bounded), so that the shared memory
// may go away.
__device__ void drain_copies(Bars* b, const Ring& r) {
  for (uint32_t s = 0; s < (uint32_t)r.stages && s < r.used; ++s) {
    const uint32_t last = (r.used - 1 - s) / r.stages;   // last round that filled stage s
    wait_bar(&b->full[s], last & 1);
  }
}
template <bool PAIR>
__device__ void drain_mmas(Bars* b) {   // from the lane that issued them
  if constexpr (PAIR) umma_commit_pair(&b->drain);
  else umma_commit(&b->drain);
  wait_bar(&b->drain, 0);
}
// Descriptor of the operand at shared-memory address `at`, from one with address 0. The mask
// matters: in a cluster the address carries the CTA's rank above its 18 bits, which would
// otherwise land in the descriptor's byte offsets.
__device__ __forceinline__ uint64_t desc_at(uint64_t base, uint32_t at) {
  return base + ((at & 0x3ffffu) >> 4);
}

// ------------------------------------------------------------------ distinct adapters
// The distinct adapters among the 128 rows of a tile in order of first use, from 128 threads
// (et = 0 .. 127, one row each; others et = -1). sync: a barrier of every thread that calls it.
struct TileSlots {
  int32_t id[BM];        // adapter of each row, -1: none
  int32_t slot[BM];      // slot of each row's adapter, -1: none
  int32_t slot_id[BM];   // adapter of each slot
  uint4 off[BM];         // rows outside each slot
  int32_t warp_count[4];
  int32_t count;
};

template <class Sync>
__device__ void find_slots(TileSlots& s, int et, const int32_t* ids, int n, int T, int row0,
                           Sync sync) {
  int id = -1;
  if (et >= 0) {
    id = row0 + et < T ? ids[row0 + et] : -1;
    if (id < 0 || id >= n) id = -1;
    s.id[et] = id;
  }
  sync();
  uint32_t eq[4] = {0, 0, 0, 0};
  int first = -1;
  bool leads = false;
  if (et >= 0 && id >= 0) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int4* v = reinterpret_cast<const int4*>(&s.id[32 * w]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int4 x = v[j];
        eq[w] |= (uint32_t)(x.x == id) << (4 * j) | (uint32_t)(x.y == id) << (4 * j + 1) |
                 (uint32_t)(x.z == id) << (4 * j + 2) | (uint32_t)(x.w == id) << (4 * j + 3);
      }
    }
#pragma unroll
    for (int w = 3; w >= 0; --w)
      if (eq[w]) first = 32 * w + __ffs(eq[w]) - 1;
    leads = first == et;
  }
  const unsigned lead = __ballot_sync(0xffffffffu, leads);
  if (et >= 0 && (et & 31) == 0) s.warp_count[et >> 5] = __popc(lead);
  sync();
  if (et >= 0 && leads) {
    int pos = __popc(lead & ((1u << (et & 31)) - 1));
    for (int w = 0; w < (et >> 5); ++w) pos += s.warp_count[w];
    s.slot_id[pos] = id;
    s.slot[et] = pos;
    s.off[pos] = make_uint4(~eq[0], ~eq[1], ~eq[2], ~eq[3]);
  }
  if (et == 0) s.count = s.warp_count[0] + s.warp_count[1] + s.warp_count[2] + s.warp_count[3];
  sync();
  int mine = -1;
  if (et >= 0 && id >= 0) mine = s.slot[first];
  sync();
  if (et >= 0) s.slot[et] = mine;
  sync();
}

// What proj_kernel reads: the list of row tile m (128 entries each), or, where it runs SM pairs,
// one list per pair of row tiles (256 entries each, from the even tile's CTA), in which an
// adapter of both tiles stands once. Called by the 128 threads et = 0 .. 127, which share named
// barrier 2; `even` holds row tile m's slots, `odd` is scratch.
__device__ void publish_slots(bool pairs, int m, int et, const int32_t* ids, int n, int T,
                              const TileSlots& even, TileSlots& odd, int32_t* n_slots,
                              Slot* slots) {
  const uint4 none = make_uint4(~0u, ~0u, ~0u, ~0u);
  Slot s;
  s.pad[0] = s.pad[1] = s.pad[2] = 0;
  s.off[1] = none;
  if (!pairs) {
    if (et == 0) n_slots[m] = even.count;
    if (et < even.count) {
      s.id = even.slot_id[et];
      s.off[0] = even.off[et];
      slots[(size_t)m * BM + et] = s;
    }
    return;
  }
  if (m & 1) return;
  auto sync = [] { named_bar_sync(2, 128); };
  find_slots(odd, et, ids, n, T, (m + 1) * BM, sync);
  Slot* out = slots + (size_t)m * BM;
  if (et < even.count) {
    s.id = even.slot_id[et];
    s.off[0] = even.off[et];
    for (int j = 0; j < odd.count; ++j)
      if (odd.slot_id[j] == s.id) s.off[1] = odd.off[j];
    out[et] = s;
  }
  bool fresh = et < odd.count;   // the odd tile's own adapters follow
  for (int j = 0; j < even.count; ++j) fresh = fresh && even.slot_id[j] != odd.slot_id[et];
  const unsigned f = __ballot_sync(0xffffffffu, fresh);
  sync();
  if ((et & 31) == 0) odd.warp_count[et >> 5] = __popc(f);
  sync();
  int pos = even.count + __popc(f & ((1u << (et & 31)) - 1));
  for (int w = 0; w < (et >> 5); ++w) pos += odd.warp_count[w];
  if (fresh) {
    s.id = odd.slot_id[et];
    s.off[0] = none;
    s.off[1] = odd.off[et];
    out[pos] = s;
  }
  if (et == 0)
    n_slots[m / 2] = even.count + odd.warp_count[0] + odd.warp_count[1] + odd.warp_count[2] +
                     odd.warp_count[3];
}

// ------------------------------------------------------------------ shrink
// u = scale (x A_a^T), as hi | lo. One cluster of `split` CTAs per row tile (and per `cy`-th
// chunk of its adapters): each CTA takes a share of the contraction, the partial sums meet
// through distributed shared memory in rank order. A chunk is at most p.cols accumulator
// columns: cols / rp adapters side by side, each rp columns wide. The ring's stages are as large
// as the tile's adapters need, and as many as then fit.
struct ShrinkParams {
  int T, n, r, rp, nb;
  int kiters, split, cy, cols, a_bytes, ring_bytes, tail;
  int pairs;          // lists for pairs of row tiles
  const int32_t* ids;
  const float* scale;
  uint8_t* uq;        // [T][nb] blocks of 128 bytes
  int32_t* n_slots;
  Slot* slots;
  uint32_t* status;
};

__global__ void __launch_bounds__(kThreads, 1)
    shrink_kernel(const __grid_constant__ CUtensorMap xmap,
                  const __grid_constant__ CUtensorMap amap, const ShrinkParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(16) TileSlots ts, ts_odd;
  float* red = reinterpret_cast<float*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                        ~uintptr_t(1023));   // [128][rp + 4], whole KB
  const int rs = p.rp + 4;
  uint8_t* smem = reinterpret_cast<uint8_t*>(red + BM * rs);
  Bars* bars = reinterpret_cast<Bars*>(smem + p.ring_bytes + p.tail);

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);   // known uniform
  const int lane = threadIdx.x & 31;
  const int et = (int)threadIdx.x - 64;
  const int q = (int)(blockIdx.x % p.split);
  const int c0 = (int)(blockIdx.x / p.split) % p.cy;
  const int m = (int)(blockIdx.x / p.split) / p.cy;
  const int row0 = m * BM;

  launch_dependents();
  if (threadIdx.x == 0) {
    init_bars(bars);
    tma_prefetch_desc(&xmap);
    tma_prefetch_desc(&amap);
  }
  if (warp == 1) tmem_alloc(&bars->tmem, p.cols);
  tc_fence_before();
  find_slots(ts, et, p.ids, p.n, p.T, row0, [] { __syncthreads(); });
  tc_fence_after();
  const uint32_t tmem = bars->tmem;
  const int count = ts.count, per = p.cols / p.rp;
  const int stage_bytes = p.a_bytes + min(count, per) * p.rp * 128;

  if (c0 == 0 && q == 0 && warp >= 2)   // while the others start the ring
    publish_slots(p.pairs, m, et, p.ids, p.n, p.T, ts, ts_odd, p.n_slots, p.slots);

  const int kb0 = (int)((long long)p.kiters * q / p.split);
  const int kb1 = (int)((long long)p.kiters * (q + 1) / p.split);
  Ring ring(min(kMaxStages, p.ring_bytes / stage_bytes));
  uint32_t parity = 0;
  for (int c = c0; c * per < count; c += p.cy, parity ^= 1) {   // the same chunks in every rank
    const int s0 = c * per, ns = min(per, count - s0);
    if (warp == 0) {
      for (int kb = kb0; kb < kb1; ++kb, ring.next()) {
        if (!warp_wait(bars, &bars->empty[ring.stage], ring.phase ^ 1, p.status)) break;
        uint8_t* sa = smem + ring.stage * stage_bytes;
        uint64_t* bar = &bars->full[ring.stage];
        if (elect_one()) {
          mbar_arrive_expect_tx(bar, p.a_bytes + ns * p.rp * 128);
          tma_load_2d(sa, &xmap, bar, kb * BK, row0);
        }
        __syncwarp();
        if (elect_one())
          for (int j = 0; j < ns; ++j)   // rp rows of 128 bytes per adapter (zeros past rank r)
            tma_load_3d(sa + p.a_bytes + j * p.rp * 128, &amap, bar, kb * BK, 0, ts.slot_id[s0 + j]);
        __syncwarp();
      }
    } else if (warp == 1) {
      const uint32_t idesc = idesc_bf16(BM, ns * p.rp, false, false);
      const uint64_t km = umma_desc_sw128(0, 16, 1024);
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb, ring.next()) {
        ok = warp_wait(bars, &bars->full[ring.stage], ring.phase, p.status);
        if (!ok) break;
        tc_fence_after();
        const uint32_t sa = smem_u32(smem + ring.stage * stage_bytes);
        const uint64_t ad = desc_at(km, sa), bd = desc_at(km, sa + p.a_bytes);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_bf16(tmem, ad + 2 * kk, bd + 2 * kk, idesc, (kb > kb0 || kk > 0) ? 1u : 0u);
          umma_commit(&bars->empty[ring.stage]);
        }
        __syncwarp();
      }
      if (ok && elect_one()) umma_commit(&bars->acc_full[0]);
      __syncwarp();
    } else {
      bool ok = !bars->abort && wait_bar(&bars->acc_full[0], parity);
      if (!ok) {
        if (!bars->abort) flag_timeout(p.status);
        bars->abort = 1;
      }
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      // rows of this warp's TMEM lanes, adapter by adapter
      const int quarter = warp & 3, row = quarter * 32 + lane;
      const int sl = ts.slot[row];
      unsigned todo = ok ? __ballot_sync(0xffffffffu, sl >= s0 && sl < s0 + ns) : 0u;
      while (todo) {
        const int cur = __shfl_sync(0xffffffffu, sl, __ffs(todo) - 1);
        todo &= ~__ballot_sync(0xffffffffu, sl == cur);
        for (int i0 = 0; i0 < p.rp; i0 += 16) {
          float v[16];
          tmem_ld16(tmem + ((uint32_t)(quarter * 32) << 16) + (cur - s0) * p.rp + i0, v);
          if (sl == cur) {
#pragma unroll
            for (int i = 0; i < 16; i += 4)
              *reinterpret_cast<float4*>(&red[row * rs + i0 + i]) =
                  make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
    }
    cluster_sync_all();
    if (et >= 0) {
      const int rows = BM / p.split, quads = p.rp / 4;
      for (int it = et; it < rows * quads; it += 128) {
        const int row = q * rows + it / quads, i = 4 * (it % quads);
        const int sl = ts.slot[row];
        if (sl < s0 || sl >= s0 + ns) continue;
        const float4 v = sum_ranks(&red[row * rs + i], p.split);
        const float f = p.scale[ts.id[row]];
        // ranks r .. rp - 1 are padding: 0 also where a row with an inf met A's zero fill
        uint2 hi, lo;
        split_pair(i < p.r ? f * v.x : 0.f, i + 1 < p.r ? f * v.y : 0.f, hi.x, lo.x);
        split_pair(i + 2 < p.r ? f * v.z : 0.f, i + 3 < p.r ? f * v.w : 0.f, hi.y, lo.y);
        uint8_t* dst = p.uq + ((size_t)(row0 + row) * p.nb + i / 32) * 128 + (i % 32) * 2;
        *reinterpret_cast<uint2*>(dst) = hi;
        *reinterpret_cast<uint2*>(dst + 64) = lo;
      }
    }
    cluster_sync_all();   // the partial sums may be overwritten, the accumulator reused
    tc_fence_after();
  }
  if (bars->abort) {
    if (warp == 0) drain_copies(bars, ring);
    if (warp == 1 && elect_one()) drain_mmas<false>(bars);
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, p.cols);
  }
  if (threadIdx.x == 0) wait_prerequisites();   // what waits for this kernel waits for them too
}

// The same for a few rows: a CTA takes RG ranks of one row, its warps share the contraction in
// pieces of 256 elements (RG independent 16-byte loads per lane, so the CTA costs about one
// trip to memory), on the CUDA cores; no MMA tile to fill, no ring to start. Fewer rows, fewer
// ranks a CTA: one SM takes in about 50 GB/s, so one row's 16 ranks of 7168 in one CTA took
// 8 us, spread over eight they take 3.6 (96 rows of 2048: 5.5). The last CTAs list the row
// tiles' adapters for proj_kernel.
constexpr int kRowThreads = 1024;
constexpr int kRowMaxPieces = 64;    // contraction up to 16384
// A batch goes this way up to 256 rows and 24 M products (rows x ranks x C): each row reads its
// adapter by itself. Forward with 32 adapters, this way against the tiles, in us:
//   7168 to 2048  rank 16: 16 rows 14.5 and 19.2, 192 rows 23.5 and 27.3, 384 rows 36.9 and 27.4
//                 rank 64: 16 rows 18.5 and 19.0, 64 rows 26.2 and 23.8
//   1024 to 1024  rank 16: 64 rows 10.2 and 13.4, 256 rows 15.6 and 16.1, 384 rows 18.1 and 16.5
// The bounds are too wide at high ranks of short contractions (1024 to 1024, rank 64: 64 rows 13.0
// and 13.5, 128 rows 18.3 and 15.2, 256 rows 35.1 and 24.4) and beside wide outputs (2048 to 7168,
// rank 16: 64 rows 18.1 and 19.5, 128 rows 21.8 and 19.8).
constexpr int kRowsMost = 256;
constexpr long long kRowsProducts = 24 << 20;

struct ShrinkRowsParams {
  int T, C, n, r, nb, groups;   // groups of RG ranks
  const __nv_bfloat16* x;      // [T][C]
  const __nv_bfloat16* w;      // [n][r][C]
  const int32_t* ids;
  const float* scale;
  uint8_t* uq;
  int32_t* n_slots;
  Slot* slots;
  int pairs;
};

__device__ __forceinline__ void unpack8(const uint4 q, float* v) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

template <int RG>
__global__ void __launch_bounds__(kRowThreads) shrink_rows_kernel(const ShrinkRowsParams p) {
  __shared__ __align__(16) TileSlots ts, ts_odd;
  __shared__ float part[kRowMaxPieces][RG];
  launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t = (int)blockIdx.x / p.groups;
  if (t >= p.T) {
    const int m = (int)blockIdx.x - p.T * p.groups;
    find_slots(ts, tid < BM ? tid : -1, p.ids, p.n, p.T, m * BM, [] { __syncthreads(); });
    if (tid < BM)
      publish_slots(p.pairs, m, tid, p.ids, p.n, p.T, ts, ts_odd, p.n_slots, p.slots);
    if (tid == 0) wait_prerequisites();   // what waits for this kernel waits for them too
    return;
  }
  const int id = p.ids[t];
  if (id < 0 || id >= p.n) return;
  const int i0 = (int)blockIdx.x % p.groups * RG;
  const __nv_bfloat16* x = p.x + (size_t)t * p.C;
  const __nv_bfloat16* w = p.w + ((size_t)id * p.r + i0) * p.C;
  const int pieces = (p.C + 255) / 256;
  const float scale = p.scale[id];
  for (int c = warp; c < pieces; c += kRowThreads / 32) {
    const int k = c * 256 + lane * 8;
    uint4 wq[RG];
    const uint4 none = make_uint4(0, 0, 0, 0);
    const uint4 xq = k < p.C ? *reinterpret_cast<const uint4*>(x + k) : none;
#pragma unroll
    for (int i = 0; i < RG; ++i)
      wq[i] = k < p.C && i0 + i < p.r ? *reinterpret_cast<const uint4*>(w + (size_t)i * p.C + k)
                                      : none;
    float xv[8], sum[RG];
    unpack8(xq, xv);
#pragma unroll
    for (int i = 0; i < RG; ++i) {
      float wv[8];
      unpack8(wq[i], wv);
      sum[i] = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[i] = fmaf(xv[j], wv[j], sum[i]);
    }
    // RG sums over 32 lanes: a step halves the sums, then the rest is added up; lane l ends
    // with sum l RG / 32
    int dist = 16;
#pragma unroll
    for (int h = RG / 2; h > 0; h >>= 1, dist >>= 1) {
      const bool up = lane & dist;
#pragma unroll
      for (int i = 0; i < h; ++i) {
        const float give = up ? sum[i] : sum[i + h];
        const float keep = up ? sum[i + h] : sum[i];
        sum[i] = keep + __shfl_xor_sync(0xffffffffu, give, dist);
      }
    }
#pragma unroll
    for (; dist > 0; dist >>= 1) sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], dist);
    if (lane % (32 / RG) == 0) part[c][lane / (32 / RG)] = sum[0];
  }
  __syncthreads();
  if (tid < RG / 2) {
    float v[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      v[j] = 0.f;
      for (int c = 0; c < pieces; ++c) v[j] += part[c][2 * tid + j];
      // ranks past r are padding: 0 also where a row with an inf met their zero fill
      v[j] = i0 + 2 * tid + j < p.r ? scale * v[j] : 0.f;
    }
    uint32_t hi, lo;
    split_pair(v[0], v[1], hi, lo);
    const int i = i0 + 2 * tid;
    uint8_t* dst = p.uq + ((size_t)t * p.nb + i / 32) * 128 + i % 32 * 2;
    *reinterpret_cast<uint32_t*>(dst) = hi;
    *reinterpret_cast<uint32_t*>(dst + 64) = lo;
  }
}

// ------------------------------------------------------------------ projection
// out tile [128][NT] = X W (TRANS: X W^T) + the adapters' steps. Three forms:
//   PAIR       large batches: the two CTAs of a cluster share M = 256 MMAs, each with its own
//              128 rows of X and half of the tile's columns of W, which takes a third off the
//              bytes a tile moves into its SM's shared memory (what bounds single CTAs);
//   split = 1  one CTA per tile;
//   split > 1  too few tiles for the SMs: a cluster of `split` CTAs shares one tile's
//              contraction, W's and the adapters' steps alike, and the partial sums meet in
//              rank order through distributed shared memory.
// The first two are persistent, with two accumulators, so that a tile's epilogue overlaps the
// next tile's MMAs; results are staged in shared memory and stored by TMA. Where the last wave
// of pairs would be at most half full, its tiles are halved in width and fill it.
//
// The adapters' part of a tile goes 32 ranks (a block of u) at a time. Its first stage holds
// that block of u for the tile's rows, and B rows of as many adapters as fit; further stages
// hold B rows only. The stage with u is handed back last, so a group is at most stages - 1
// stages long; a longer list loads u again for its next group.
//
// Launched with programmatic dependence on u's kernel: the steps over W need nothing from it, so
// only the adapters' part waits. A CTA can start only where it has room: shrink_kernel takes its
// SM's shared memory and shrink_rows_kernel<16> its registers, so that is on the SMs that they do
// not use (24 of 152 beside the 128 tiles of 8192 rows) or have left.
//
// By itself under a profiler, 8192 rows of 7168 to 2048 with a dozen adapters of rank 32 take 132
// us, 1.82 PFLOP/s, 0.95 of cuBLAS's burst rate (the transposed product, rank 16, 127 us, 0.98):
// bound by the tensor cores, whose pipe is 84% (86%) busy. The whole forward of one such row, rank
// 16, takes 11.6 us, where W's 29 MB need 4.4: the rest is the start, the join and the launches.
// 96 rows with 48 adapters, 2048 to 7168: 19.9 us, u and then the adapters' steps and the join.
struct ProjParams {
  int T, out_cols, n;
  int kiters;               // steps over W (0: the adapters' part alone)
  int NT, n_tiles, m_tiles, split, stages, a_bytes, stage_bytes;
  int whole;                // PAIR: tiles from here on are run as two halves of NT / 2 columns
  int rp, nb, rb;           // padded rank, 32-rank blocks, ranks per adapter step
  int out_bf16;
  const int32_t* ids;
  const int32_t* n_slots;   // null: no adapters' part
  const Slot* slots;
  void* out;
  uint32_t* status;
};

// The adapters that a CTA (or pair) runs for one tile, in a fixed order, 32 at a time in the
// lanes of a warp. split: every split-th slot from rank q.
template <bool PAIR>
struct SlotList {
  const Slot* base;
  int count, q, split, window;
  int id;
  uint4 off0, off1;
  __device__ void open(const ProjParams& p, int m, int rank) {   // m: (first) row tile
    base = p.slots + (size_t)m * BM;
    const int n = p.n_slots[PAIR ? m / 2 : m];
    q = PAIR ? 0 : rank;
    split = PAIR ? 1 : p.split;
    count = n > q ? (n - q + split - 1) / split : 0;
    window = -1;
    if (count > 0) load(0);
  }
  __device__ void load(int w) {
    window = w;
    const int i = 32 * w + (int)(threadIdx.x & 31);
    if (i >= count) return;
    const Slot* s = base + (q + i * split);
    id = s->id;
    off0 = s->off[0];
    if (PAIR) off1 = s->off[1];
  }
  // whole warp: adapter and lane masks of entry i
  __device__ int get_id(int i) {
    if (i >> 5 != window) load(i >> 5);
    return __shfl_sync(0xffffffffu, id, i & 31);
  }
  __device__ static uint4 pick(const uint4& v, int lane) {
    return make_uint4(__shfl_sync(0xffffffffu, v.x, lane), __shfl_sync(0xffffffffu, v.y, lane),
                      __shfl_sync(0xffffffffu, v.z, lane), __shfl_sync(0xffffffffu, v.w, lane));
  }
  __device__ void get_off(int i, uint4& a, uint4& b) {
    if (i >> 5 != window) load(i >> 5);
    a = pick(off0, i & 31);
    if (PAIR) b = pick(off1, i & 31);
  }
};

template <bool TRANS, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    proj_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
                const __grid_constant__ CUtensorMap umap, const __grid_constant__ CUtensorMap emap,
                const __grid_constant__ CUtensorMap omap, const ProjParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* staging = smem + p.stages * p.stage_bytes;
  // split > 1: no staging boxes; the partial tile reuses the pipeline stages
  Bars* bars = reinterpret_cast<Bars*>(staging + (p.split == 1 ? 8 * kStagingBox : 0));

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);   // known uniform
  const int lane = threadIdx.x & 31;
  const int csize = PAIR ? 2 : p.split;
  const int q = (int)(blockIdx.x % csize);                  // rank in the cluster
  const int m_step = PAIR ? 2 : 1;                          // row tiles of a tile
  const int all = (p.m_tiles + m_step - 1) / m_step * p.n_tiles;
  const int tiles = PAIR ? p.whole + 2 * (all - p.whole) : all;
  const int t0 = (int)(blockIdx.x / csize), tstep = (int)(gridDim.x / csize);
  const int kb0 = PAIR ? 0 : (int)((long long)p.kiters * q / p.split);
  const int kb1 = PAIR ? p.kiters : (int)((long long)p.kiters * (q + 1) / p.split);
  const uint32_t tmem_cols = p.NT <= 64 ? 128 : p.NT <= 128 ? 256 : 512;   // two accumulators
  const int per_stage = 64 / p.rb;                          // adapters of an adapter stage
  const int group = p.stages - 1;

  if (threadIdx.x == 0) {
    init_bars(bars, PAIR);
    tma_prefetch_desc(&xmap);
    tma_prefetch_desc(&wmap);
    tma_prefetch_desc(&umap);
    tma_prefetch_desc(&emap);
  }
  if (warp == 1) {
    if constexpr (PAIR) tmem_alloc_pair(&bars->tmem, tmem_cols);
    else tmem_alloc(&bars->tmem, tmem_cols);
  }
  tc_fence_before();
  if constexpr (PAIR) cluster_sync_all();   // the other CTA's barriers are initialised
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem;

  // tile -> its (first) row tile, first column and width
  auto place = [&](int tile, int& m, int& n0, int& width) {
    width = p.NT;
    int half = 0;
    if (PAIR && tile >= p.whole) {
      const int h = tile - p.whole;
      tile = p.whole + h / 2;
      width = p.NT / 2;
      half = (h & 1) * width;
    }
    m = tile / p.n_tiles * m_step;
    n0 = tile % p.n_tiles * p.NT + half;
  };

  if (warp == 0) {
    // ---- producer
    Ring ring(p.stages);
    SlotList<PAIR> list;
    bool ok = true;
    // one box of X's (or u's) rows, or of the columns of W (or B) for this CTA
    auto load2 = [&](void* dst, const CUtensorMap* m, int c0, int c1) {
      if constexpr (PAIR) tma_load_2d_pair(dst, m, mapa_rank(&bars->full[ring.stage], 0), c0, c1);
      else tma_load_2d(dst, m, &bars->full[ring.stage], c0, c1);
    };
    auto load3 = [&](void* dst, const CUtensorMap* m, int c0, int c1, int c2) {
      if constexpr (PAIR) tma_load_3d_pair(dst, m, mapa_rank(&bars->full[ring.stage], 0), c0, c1, c2);
      else tma_load_3d(dst, m, &bars->full[ring.stage], c0, c1, c2);
    };
    auto announce = [&](uint32_t bytes) {   // PAIR: rank 0 announces both CTAs' bytes
      if (!PAIR || q == 0) mbar_arrive_expect_tx(&bars->full[ring.stage], PAIR ? 2 * bytes : bytes);
    };
    for (int tile = t0; ok && tile < tiles; tile += tstep) {
      int m, n0, width;
      place(tile, m, n0, width);
      const int row0 = (m + (PAIR ? q : 0)) * BM;
      const int nc = PAIR ? width / 2 : width;   // columns this CTA loads
      if (PAIR) n0 += q * nc;
      if (p.n_slots != nullptr && tile != t0) list.open(p, m, q);   // ahead of the steps over W
      for (int kb = kb0; kb < kb1; ++kb, ring.next()) {
        ok = warp_wait(bars, &bars->empty[ring.stage], ring.phase ^ 1, p.status);
        if (!ok) break;
        uint8_t* sa = smem + ring.stage * p.stage_bytes;
        uint8_t* sb = sa + p.a_bytes;
        if (elect_one()) {
          announce(p.a_bytes + nc * 128);
          load2(sa, &xmap, kb * BK, row0);
          for (int j = 0; j < nc / 64; ++j) {
            if (TRANS) load2(sb + j * 64 * 128, &wmap, kb * BK, n0 + j * 64);   // 64 rows of W (K-major)
            else load2(sb + j * 64 * 128, &wmap, n0 + j * 64, kb * BK);         // 64 columns (MN-major)
          }
        }
        __syncwarp();
      }
      if (tile == t0) {
        wait_prerequisites();
        if (p.n_slots != nullptr) list.open(p, m, q);
      }
      if (!ok || p.n_slots == nullptr) continue;
      for (int b = 0; b < p.nb && ok; ++b) {
        int in_group = 0;
        for (int i0 = 0; i0 < list.count; i0 += per_stage, ring.next()) {
          const int cnt = min(per_stage, list.count - i0);
          const bool head = in_group == 0;
          ok = warp_wait(bars, &bars->empty[ring.stage], ring.phase ^ 1, p.status);
          if (!ok) break;
          uint8_t* sa = smem + ring.stage * p.stage_bytes;
          if (elect_one()) {
            announce((head ? p.a_bytes : 0) + cnt * nc * p.rb * 2);
            if (head) load2(sa, &umap, b * 64, row0);
          }
          __syncwarp();
          for (int j = 0; j < cnt; ++j) {
            const int id = list.get_id(i0 + j);
            uint8_t* sb = sa + p.a_bytes + j * nc * p.rb * 2;
            if (elect_one())
              for (int c = 0; c < nc / 64; ++c)   // rb ranks x 64 columns (zeros past rank r)
                load3(sb + c * p.rb * 128, &emap, n0 + c * 64, b * 32, id);
            __syncwarp();
          }
          if (++in_group == group) in_group = 0;
        }
      }
    }
    if (bars->abort && (!PAIR || q == 0)) drain_copies(bars, ring);
  } else if (warp == 1 && (!PAIR || q == 0)) {
    // ---- MMA
    const int rows = PAIR ? 2 * BM : BM;
    auto commit = [&](uint64_t* bar) {
      if constexpr (PAIR) umma_commit_pair(bar);
      else umma_commit(bar);
    };
    const uint64_t km = umma_desc_sw128(0, 16, 1024);              // K-major operand
    const uint64_t wm = TRANS ? km : umma_desc_sw128(0, 64 * 128, 1024);
    const uint64_t em = umma_desc_sw128(0, p.rb * 128, 1024);      // MN-major, rb rows a chunk
    constexpr uint32_t wstep = TRANS ? 32 / 16 : 2048 / 16;        // 16 contraction elements on
    Ring ring(p.stages);
    SlotList<PAIR> list;
    bool ok = true;
    int local = 0;
    for (int tile = t0; tile < tiles; tile += tstep, ++local) {
      int m, n0, width;
      place(tile, m, n0, width);
      const int nc = PAIR ? width / 2 : width;
      const uint32_t idesc = idesc_bf16(rows, width, false, !TRANS);
      const uint32_t idesc_e = idesc_bf16(rows, width, false, true);
      const int acc = local & 1;
      const uint32_t d = tmem + acc * (tmem_cols / 2);
      if (p.n_slots != nullptr && tile != t0) list.open(p, m, q);
      ok = warp_wait(bars, &bars->acc_empty[acc], ((local >> 1) & 1) ^ 1, p.status);
      tc_fence_after();
      for (int kb = kb0; ok && kb < kb1; ++kb) {
        ok = warp_wait(bars, &bars->full[ring.stage], ring.phase, p.status);
        if (!ok) break;
        tc_fence_after();
        const uint32_t sa = smem_u32(smem + ring.stage * p.stage_bytes);
        const uint64_t ad = desc_at(km, sa), bd = desc_at(wm, sa + p.a_bytes);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint32_t accumulate = (kb > kb0 || kk > 0) ? 1u : 0u;
            if constexpr (PAIR) umma_bf16_pair(d, ad + 2 * kk, bd + wstep * kk, idesc, accumulate);
            else umma_bf16(d, ad + 2 * kk, bd + wstep * kk, idesc, accumulate);
          }
          commit(&bars->empty[ring.stage]);
        }
        __syncwarp();
        ring.next();
      }
      if (tile == t0) {
        wait_prerequisites();
        if (p.n_slots != nullptr) list.open(p, m, q);
      }
      if (!ok) break;
      if (p.n_slots != nullptr) {
        for (int b = 0; b < p.nb && ok; ++b) {
          int in_group = 0, head_stage = 0;
          for (int i0 = 0; i0 < list.count; i0 += per_stage) {
            const int cnt = min(per_stage, list.count - i0);
            ok = warp_wait(bars, &bars->full[ring.stage], ring.phase, p.status);
            if (!ok) break;
            tc_fence_after();
            if (in_group == 0) head_stage = ring.stage;
            const uint32_t su = smem_u32(smem + head_stage * p.stage_bytes);
            const uint32_t sb = smem_u32(smem + ring.stage * p.stage_bytes) + p.a_bytes;
            for (int j = 0; j < cnt; ++j) {
              uint4 off, off_odd;
              list.get_off(i0 + j, off, off_odd);
              const uint64_t hi = desc_at(km, su), bd = desc_at(em, sb + j * nc * p.rb * 2);
              if (elect_one()) {
                for (int kk = 0; kk < p.rb / 16; ++kk) {   // hi and lo of 16 ranks, same rows of B
                  // without W a row's first step starts its sum (a row is in one slot only)
                  const uint32_t first = (p.kiters > 0 || b > 0 || kk > 0) ? 1u : 0u;
                  const uint64_t h = hi + 2 * kk, l = h + 4, e = bd + 128 * kk;
                  if constexpr (PAIR) {
                    umma_bf16_rows_pair(d, h, e, idesc_e, off, off_odd, first);
                    umma_bf16_rows_pair(d, l, e, idesc_e, off, off_odd, 1u);
                  } else {
                    umma_bf16_rows(d, h, e, idesc_e, off, first);
                    umma_bf16_rows(d, l, e, idesc_e, off, 1u);
                  }
                }
              }
              __syncwarp();
            }
            const bool last = i0 + per_stage >= list.count || in_group + 1 == group;
            if (elect_one()) {
              if (in_group > 0) commit(&bars->empty[ring.stage]);
              if (last) commit(&bars->empty[head_stage]);
            }
            __syncwarp();
            ring.next();
            if (++in_group == group) in_group = 0;
          }
        }
      }
      if (!ok) break;
      if (elect_one()) commit(&bars->acc_full[acc]);
      __syncwarp();
    }
    if (bars->abort && elect_one()) drain_mmas<PAIR>(bars);
    __syncwarp();
  } else if (warp == 1) {
    wait_prerequisites();
  } else {
    // ---- epilogue
    const int quarter = warp & 3, row = quarter * 32 + lane;
    uint8_t* box = staging + quarter * 2 * kStagingBox;
    int local = 0, stored = 0;
    for (int tile = t0; tile < tiles; tile += tstep, ++local) {
      const int acc = local & 1;
      int m, n0, width;
      place(tile, m, n0, width);
      const int row0 = (m + (PAIR ? q : 0)) * BM;
      bool ok = !bars->abort && wait_bar(&bars->acc_full[acc], (local >> 1) & 1);
      if (!ok) {
        if (!bars->abort) flag_timeout(p.status);
        bars->abort = 1;
      }
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const uint32_t d = tmem + acc * (tmem_cols / 2) + ((uint32_t)(quarter * 32) << 16);
      const bool rows_here = row0 + quarter * 32 < p.T;
      bool zero = false;   // adapters' part alone: rows without an adapter were never written
      if (p.kiters == 0) {
        const int id = row0 + row < p.T ? p.ids[row0 + row] : -1;
        zero = id < 0 || id >= p.n;
      }
      if (!PAIR && p.split > 1) {
        float* red = reinterpret_cast<float*>(smem) + row * (p.NT + 4);
        for (int c = 0; rows_here && c < p.NT; c += 32) {
          float v[32];
          tmem_ld32(d + c, v);
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<float4*>(red + c + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        }
        continue;
      }
      const int step = p.out_bf16 ? 64 : 32;   // columns of a 128-byte box row
      for (int c = 0; rows_here && c < width && n0 + c < p.out_cols; c += step, ++stored) {
        uint8_t* dst = box + (stored & 1) * kStagingBox;
        float v[32];
        if (stored >= 2) {
          if (lane == 0) bulk_wait_read<1>();
          __syncwarp();
        }
        for (int h = 0; h < step / 32; ++h) {
          tmem_ld32(d + c + 32 * h, v);
          if (zero) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0.f;
          }
          if (p.out_bf16) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              *reinterpret_cast<uint4*>(dst + lane * 128 + (((4 * h + j) ^ (lane & 7)) * 16)) =
                  make_uint4(pack_bf16(v[8 * j], v[8 * j + 1]), pack_bf16(v[8 * j + 2], v[8 * j + 3]),
                             pack_bf16(v[8 * j + 4], v[8 * j + 5]),
                             pack_bf16(v[8 * j + 6], v[8 * j + 7]));
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              *reinterpret_cast<float4*>(dst + lane * 128 + ((j ^ (lane & 7)) * 16)) =
                  make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(&omap, dst, n0 + c, row0 + quarter * 32);
          bulk_commit();
        }
      }
      tc_fence_before();
      if constexpr (PAIR) {
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(mapa_rank(&bars->acc_empty[acc], 0));
      } else {
        mbar_arrive(&bars->acc_empty[acc]);
      }
    }
    if (lane == 0) bulk_wait_all();
  }
  __syncwarp();

  if (!PAIR && p.split > 1) {   // one tile per cluster
    cluster_sync_all();
    if (warp >= 2) {
      const int et = (int)threadIdx.x - 64, tile = t0;
      const int row0 = tile / p.n_tiles * BM, n0 = tile % p.n_tiles * p.NT;
      const int rows = min(BM, p.T - row0), groups = p.NT / 4;
      const float* red = reinterpret_cast<const float*>(smem);
      for (int it = q * 128 + et; it < rows * groups; it += 128 * p.split) {
        const int r = it / groups, c = it % groups * 4;
        if (n0 + c >= p.out_cols) continue;
        const float4 a = sum_ranks(red + r * (p.NT + 4) + c, p.split);
        const size_t at = (size_t)(row0 + r) * p.out_cols + n0 + c;
        if (p.out_bf16)
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + at) =
              make_uint2(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w));
        else
          *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = a;
      }
    }
    cluster_sync_all();   // no rank leaves while another reads its partial tile
  }
  tc_fence_before();
  if constexpr (PAIR) cluster_sync_all();   // no copy or commit of either CTA is on its way
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    if constexpr (PAIR) tmem_dealloc_pair(tmem, tmem_cols);
    else tmem_dealloc(tmem, tmem_cols);
  }
}

// ------------------------------------------------------------------ row lists
// One CTA per adapter: its rows in ascending order at rows[off[a] .. off[a + 1]), where off[a]
// counts the rows of lower adapters. Each CTA reads all ids, so that no CTA waits for another, and
// the work grows with n T: 8192 rows take 10 us for 48 adapters, 53 for 1024, 200 for 4096 and 790
// for 16384 (of backwards of 73, 414, 1208 and 2950 us, 512 to 512, rank 8). Runs beside
// shrink_kernel, which needs nothing from it.
constexpr int kBucketThreads = 1024;

__global__ void __launch_bounds__(kBucketThreads)
    bucket_kernel(int T, int n, const int32_t* __restrict__ ids, int32_t* __restrict__ off,
                  int32_t* __restrict__ rows) {
  __shared__ int s_less[32], s_eq[32];
  launch_dependents();
  const int a = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int less = 0;
  for (int t = tid; t < T; t += kBucketThreads) {
    const int id = ids[t];
    less += id >= 0 && id < a;
  }
  less = __reduce_add_sync(0xffffffffu, less);
  if (lane == 0) s_less[warp] = less;
  __syncthreads();
  int base = 0;
  for (int w = 0; w < 32; ++w) base += s_less[w];
  const int start = base;
  for (int t0 = 0; t0 < T; t0 += kBucketThreads) {
    const int t = t0 + tid;
    const bool mine = t < T && ids[t] == a;
    const unsigned b = __ballot_sync(0xffffffffu, mine);
    if (lane == 0) s_eq[warp] = __popc(b);
    __syncthreads();
    int pos = base, all = 0;
    for (int w = 0; w < 32; ++w) {
      const int c = s_eq[w];
      if (w < warp) pos += c;
      all += c;
    }
    if (mine) rows[pos + __popc(b & ((1u << lane) - 1))] = t;
    base += all;
    __syncthreads();
  }
  if (tid == 0) {
    off[a] = start;
    if (a == n - 1) off[n] = base;
  }
}

// ------------------------------------------------------------------ weight gradients
// dA[a] = sum over adapter a's rows t of vq[t]^T xa[t], and dB[a] the same of uq and dY, in one
// launch. A CTA owns N columns of one of the two and an equal share of the row list (adapter
// by adapter), whatever the adapters' sizes; the `split` shares of a block of columns are the
// ranks of a cluster. An adapter that lies inside a share is finished there. One that goes on
// into the next ranks' shares leaves partial sums in their shared memory, which the rank where
// it starts adds up in rank order.
//
// One pass over xa and dY, memory bound: 64 rows of the list a stage, gathered by eight warps
// (four: 368 against 353 us for a training step at rank 64) with 16-byte asynchronous copies
// (TMA's row gather, four rows of 128 bytes an instruction, reached half the rate). A stage
// holds xa or dY [64 rows][N], the rows' hi values [64][ranks] and their lo values, all
// contraction-row by contraction-row (MN-major operands), so two MMAs per 16 rows, hi and lo,
// sum D[rank][column] in TMEM. Two accumulators: an adapter's results leave while the next one's
// rows are multiplied. Rows past an adapter's end are filled with zeros in both operands, so
// that no other adapter's value can meet a zero; ranks past RP and the duplicate half of a short
// M are accumulator rows that nothing reads.
//
// 8192 rows, 7168 and 2048 columns, four adapters: 37 us at rank 16 (4.1 TB/s), 49 at rank 64,
// 89 at rank 128, where 128 columns a CTA read u twice as often. (On warp-level MMAs the launch
// grew with the rank, to 199 us at rank 128.)
constexpr int kWgRows = 64;
constexpr int kWgGather = 256;       // threads that gather (whole warps, a multiple of four)
constexpr int kWgThreads = kWgGather + 160;   // + one MMA warp, four epilogue warps
constexpr int kWgBox = kWgRows * 128;

template <int RP, int NCOLS>
struct WgShape {
  static constexpr int N = NCOLS;                       // columns of a CTA
  static constexpr int UT = RP <= 64 ? 1 : 2;           // 64-rank tiles of hi (and of lo)
  static constexpr int STAGE = (N / 64 + 2 * UT) * kWgBox;
  static constexpr int STAGES = RP <= 32 ? 4 : 3;
  static constexpr int LAG = STAGES - 2;                // copies in flight behind the newest
  static constexpr int RS = N + 4;                      // floats per row of the partial sums
  static constexpr int PART = RP * RS * 4;
  static constexpr int SMEM = STAGES * STAGE + PART + kBarBytes + 1024;
  static_assert(STAGES * STAGE >= PART && SMEM <= (int)kMaxSmem, "shared memory");
};

__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(on ? 16 : 0)
               : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

struct WgradSide {
  const uint8_t* uq;             // [T][nb] blocks of 128 bytes
  const __nv_bfloat16* g;        // [T][C]
  void* out;                     // [n][r][C]
  int C, ctiles;
};
struct WgradParams {
  WgradSide side[2];
  int r, n, split, out_bf16;
  const int32_t* off;            // [n + 1]
  const int32_t* rows;           // [off[n]]
  uint32_t* status;
};

template <int RP, int NCOLS>
__global__ void __launch_bounds__(kWgThreads, 1) wgrad_kernel(const WgradParams p) {
  using S = WgShape<RP, NCOLS>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  float* tail = reinterpret_cast<float*>(smem);    // over the stages, when they are done
  float* head = reinterpret_cast<float*>(smem + S::STAGES * S::STAGE);   // [RP][RS]
  Bars* bars = reinterpret_cast<Bars*>(smem + S::STAGES * S::STAGE + S::PART);
  __shared__ int s_last, s_more;
  launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // known uniform
  const int q = (int)(blockIdx.x % p.split);
  int ct = (int)(blockIdx.x / p.split);
  const bool second = ct >= p.side[0].ctiles;
  if (second) ct -= p.side[0].ctiles;
  const uint8_t* uq = second ? p.side[1].uq : p.side[0].uq;
  const __nv_bfloat16* g = second ? p.side[1].g : p.side[0].g;
  void* out = second ? p.side[1].out : p.side[0].out;
  const int C = second ? p.side[1].C : p.side[0].C;
  const int c0 = ct * S::N;
  if (tid == 0) {
    for (int i = 0; i < S::STAGES; ++i) {
      mbar_init(&bars->full[i], kWgGather);
      mbar_init(&bars->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->acc_full[i], 1);
      mbar_init(&bars->acc_empty[i], 128);
    }
    mbar_init(&bars->drain, 1);
    bars->abort = 0;
    s_last = -1;
    s_more = 0;
    fence_mbar_init();
  }
  if (warp == kWgGather / 32) tmem_alloc(&bars->tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem;
  wait_prerequisites();

  const int total = p.off[p.n];
  const int r0 = (int)((long long)total * q / p.split);
  const int r1 = (int)((long long)total * (q + 1) / p.split);
  // adapter of list row r0: the last one whose rows start at or before it
  int a = 0;
  if (r0 < r1) {
    int lo = 0, hi = p.n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (p.off[mid] <= r0) lo = mid;
      else hi = mid - 1;
    }
    a = lo;
  }

  if (warp < kWgGather / 32) {
    // ---- gather: a thread copies one 16-byte column of the stage's rows (and its pieces of
    // u); the lanes of a warp hold the 64 row numbers, the next stage's already on their way
    constexpr int GC = S::N / 8;                       // 16-byte columns of a row
    constexpr int GI = kWgRows * GC / kWgGather, UP = RP / 4;
    constexpr int UI = kWgRows * UP / kWgGather;
    static_assert(GI * kWgGather == kWgRows * GC && UI * kWgGather == kWgRows * UP, "whole passes");
    const int gc = tid % GC;
    const bool col_on = c0 + gc * 8 < C;
    Ring ring(S::STAGES);
    int done = 0, pending = 0;                         // next stage to hand over, stages before it
    bool ok = true;
    for (int at = r0; ok && at < r1; ++a) {
      const int end = min(p.off[a + 1], r1);
      int n0 = at + lane < end ? p.rows[at + lane] : -1;
      int n1 = at + 32 + lane < end ? p.rows[at + 32 + lane] : -1;
      for (int b = at; b < end; b += kWgRows) {
        const int i0 = n0, i1 = n1;
        const int nx = b + kWgRows + lane;
        n0 = nx < end ? p.rows[nx] : -1;
        n1 = nx + 32 < end ? p.rows[nx + 32] : -1;
        ok = warp_wait(bars, &bars->empty[ring.stage], ring.phase ^ 1, p.status);
        if (!ok) break;
        uint8_t* sg = smem + ring.stage * S::STAGE;
        uint8_t* su = sg + S::N / 64 * kWgBox;
#pragma unroll
        for (int i = 0; i < GI; ++i) {
          const int rr = tid / GC + kWgGather / GC * i;
          const int row = __shfl_sync(0xffffffffu, rr < 32 ? i0 : i1, rr & 31);
          const bool on = row >= 0 && col_on;
          cp_async16(sg + (gc >> 3) * kWgBox + rr * 128 + (((gc & 7) ^ (rr & 7)) * 16),
                     on ? g + (size_t)row * C + c0 + gc * 8 : g, on);
        }
#pragma unroll
        for (int i = 0; i < UI; ++i) {
          const int rr = tid / UP + kWgGather / UP * i, pc = tid % UP;
          const int row = __shfl_sync(0xffffffffu, rr < 32 ? i0 : i1, rr & 31);
          const int h = pc % (RP / 8), lo = pc / (RP / 8);   // eight ranks, hi or lo
          cp_async16(su + (lo * S::UT + (h >> 3)) * kWgBox + rr * 128 + (((h & 7) ^ (rr & 7)) * 16),
                     row >= 0 ? uq + ((size_t)row * ((RP + 31) / 32) + (h >> 2)) * 128 + lo * 64 +
                                    (h & 3) * 16
                              : uq,
                     row >= 0);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        ring.next();
        if (++pending > S::LAG) {                      // the oldest has landed: hand it over
          cp_async_wait<S::LAG>();
          fence_proxy_async_smem();
          mbar_arrive(&bars->full[done]);
          done = done + 1 == S::STAGES ? 0 : done + 1;
          --pending;
        }
      }
      at = max(at, end);
    }
    cp_async_wait<0>();
    fence_proxy_async_smem();
    for (; pending > 0; --pending) {
      mbar_arrive(&bars->full[done]);
      done = done + 1 == S::STAGES ? 0 : done + 1;
    }
  } else if (warp == kWgGather / 32) {
    // ---- MMA
    const uint32_t idesc = idesc_bf16(128, S::N, true, true);
    const uint64_t mn = umma_desc_sw128(0, kWgBox, 1024);
    Ring ring(S::STAGES);
    bool ok = true;
    int seg = 0;
    for (int at = r0; ok && at < r1; ++a) {
      const int begin = p.off[a], end = p.off[a + 1], stop = min(end, r1);
      if (begin == end) continue;
      const int buf = seg & 1;
      const uint32_t d = tmem + buf * 256;
      ok = warp_wait(bars, &bars->acc_empty[buf], ((seg >> 1) & 1) ^ 1, p.status);
      tc_fence_after();
      for (int b = at; ok && b < stop; b += kWgRows) {
        ok = warp_wait(bars, &bars->full[ring.stage], ring.phase, p.status);
        if (!ok) break;
        tc_fence_after();
        const uint32_t sg = smem_u32(smem + ring.stage * S::STAGE);
        const uint32_t su = sg + S::N / 64 * kWgBox;
        const uint64_t bd = desc_at(mn, sg), hi = desc_at(mn, su),
                       lo = desc_at(mn, su + S::UT * kWgBox);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            umma_bf16(d, hi + 128 * kk, bd + 128 * kk, idesc, (b > at || kk > 0) ? 1u : 0u);
            umma_bf16(d, lo + 128 * kk, bd + 128 * kk, idesc, 1u);
          }
          umma_commit(&bars->empty[ring.stage]);
        }
        __syncwarp();
        ring.next();
      }
      at = stop;
      if (!ok) break;
      if (elect_one()) umma_commit(&bars->acc_full[buf]);
      __syncwarp();
      ++seg;
    }
    if (bars->abort && elect_one()) drain_mmas<false>(bars);
    __syncwarp();
  } else {
    // ---- epilogue: lane = rank
    const int quarter = warp & 3, rank = quarter * 32 + lane;
    int seg = 0;
    for (int at = r0; at < r1; ++a) {
      const int begin = p.off[a], end = p.off[a + 1], stop = min(end, r1);
      if (begin == end) continue;
      const int buf = seg & 1;
      if (!warp_wait(bars, &bars->acc_full[buf], (seg >> 1) & 1, p.status)) break;
      tc_fence_after();
      at = stop;
      const bool began = begin >= r0, ends = end <= r1;
      if (began && !ends && quarter == 0 && lane == 0) {   // goes on in the next ranks
        int more = 0;
        while (q + more + 1 < p.split && (int)((long long)total * (q + more + 1) / p.split) < end)
          ++more;
        s_last = a;
        s_more = more;
      }
      const uint32_t d = tmem + buf * 256 + ((uint32_t)(quarter * 32) << 16);
      for (int c = 0; quarter * 32 < RP && c < S::N && c0 + c < C; c += 32) {
        float v[32];
        tmem_ld32(d + c, v);
        if (began && ends) {   // finished here
          const size_t o = ((size_t)a * p.r + rank) * C + c0 + c;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (rank < p.r && c0 + c + 8 * j < C) {
              if (p.out_bf16) {
                *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(out) + o + 8 * j) =
                    make_uint4(pack_bf16(v[8 * j], v[8 * j + 1]), pack_bf16(v[8 * j + 2], v[8 * j + 3]),
                               pack_bf16(v[8 * j + 4], v[8 * j + 5]),
                               pack_bf16(v[8 * j + 6], v[8 * j + 7]));
              } else {
                float4* dst = reinterpret_cast<float4*>(static_cast<float*>(out) + o + 8 * j);
                dst[0] = make_float4(v[8 * j], v[8 * j + 1], v[8 * j + 2], v[8 * j + 3]);
                dst[1] = make_float4(v[8 * j + 4], v[8 * j + 5], v[8 * j + 6], v[8 * j + 7]);
              }
            }
          }
        } else if (rank < RP) {   // to this rank's head, or (its last adapter) its tail
          float* dst = (began ? tail : head) + rank * S::RS + c;
#pragma unroll
          for (int j = 0; j < 32; j += 4)
            *reinterpret_cast<float4*>(dst + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        }
        __syncwarp();
      }
      tc_fence_before();
      mbar_arrive(&bars->acc_empty[buf]);
      ++seg;
    }
    if (r0 == r1)                     // fewer rows than ranks: nothing to add here
      for (int i = tid - kWgGather - 32; i < RP * S::RS; i += 128) head[i] = 0.f;
  }
  __syncwarp();
  // out[z] = this CTA's tail (or zeros) + the heads of the next ranks
  auto write = [&](int z, bool own, int ranks) {
    for (int it = tid; it < p.r * (S::N / 4); it += kWgThreads) {
      const int rr = it / (S::N / 4), cc = it % (S::N / 4) * 4;
      if (c0 + cc >= C) continue;
      float4 v[8];
#pragma unroll
      for (int k = 1; k < 8; ++k)
        if (k <= ranks) v[k] = ld_rank4(head + rr * S::RS + cc, q + k);
      float4 s = own ? *reinterpret_cast<const float4*>(tail + rr * S::RS + cc)
                     : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 1; k < 8; ++k)
        if (k <= ranks) {
          s.x += v[k].x; s.y += v[k].y; s.z += v[k].z; s.w += v[k].w;
        }
      const size_t o = ((size_t)z * p.r + rr) * C + c0 + cc;
      if (p.out_bf16)
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out) + o) =
            make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
      else
        *reinterpret_cast<float4*>(static_cast<float*>(out) + o) = s;
    }
  };
  tc_fence_before();
  cluster_sync_all();                 // every head is in place
  if (s_last >= 0) write(s_last, true, s_more);
  for (int z = q; z < p.n; z += p.split)   // adapters without rows
    if (p.off[z] == p.off[z + 1]) write(z, false, 0);
  cluster_sync_all();                 // no rank leaves while another reads its head
  if (warp == kWgGather / 32) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ host side
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static std::atomic<EncodeTiledFn> fn{nullptr};
  EncodeTiledFn f = fn.load(std::memory_order_acquire);
  if (f) return f;
  void* p = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
          cudaSuccess || q != cudaDriverEntryPointSuccess)
    return nullptr;
  f = reinterpret_cast<EncodeTiledFn>(p);
  fn.store(f, std::memory_order_release);
  return f;
}

// Map of a dense row-major tensor [d2][d1][d0] (d2 = 0: a matrix) with boxes of 128 bytes x
// box1 rows, 128-byte swizzle; loads outside read zeros, stores outside are dropped.
bool make_map(CUtensorMap* m, const void* base, bool bf16, uint64_t d0, uint64_t d1, uint64_t d2,
              int box1) {
  EncodeTiledFn enc = encode_fn();
  if (!enc || !base) return false;
  const uint64_t es = bf16 ? 2 : 4;
  cuuint64_t dims[3] = {d0, d1, d2};
  cuuint64_t strides[2] = {d0 * es, d0 * d1 * es};
  cuuint32_t box[3] = {(cuuint32_t)(128 / es), (cuuint32_t)box1, 1};
  cuuint32_t step[3] = {1, 1, 1};
  return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
             d2 ? 3 : 2, const_cast<void*>(base), dims, strides, box, step,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int padded_rank(int r) { return r <= 16 ? 16 : r <= 32 ? 32 : r <= 64 ? 64 : 128; }

// Parts of `saved`: the slots of each row tile, then u. The backward's workspace holds the
// same for v, then the row lists.
struct SavedParts {
  size_t n_slots, slots, uq, total;
};
SavedParts saved_parts(const mok_lora_dims& d) {
  const size_t mt = (size_t)(d.T + 2 * BM - 1) / (2 * BM) * 2, nb = (padded_rank(d.r) + 31) / 32;
  SavedParts s;
  s.n_slots = 0;
  s.slots = align_up(mt * 4, 256);
  s.uq = s.slots + align_up(mt * BM * sizeof(Slot), 256);
  s.total = s.uq + align_up((size_t)d.T * nb * 128, 256);
  return s;
}
struct WorkParts {
  SavedParts v;
  size_t off, rows, total;
};
WorkParts work_parts(const mok_lora_dims& d) {
  WorkParts w;
  w.v = saved_parts(d);
  w.off = w.v.total;
  w.rows = w.off + align_up(((size_t)d.n + 1) * 4, 256);
  w.total = w.rows + align_up((size_t)d.T * 4, 256);
  return w;
}

// The current device's SMs, and how many clusters of 1, 2, 4, 8 CTAs of proj_kernel (one CTA
// per SM) it holds at once. Also raises the kernels' shared-memory limits. Once per device.
struct Device {
  int sms = 0;
  int clusters[4];
};
template <typename K>
int max_clusters(K kernel, int cluster, size_t smem) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)cluster * 64);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  return cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess ? n : 0;
}
bool init_device(Device& d, int dev) {
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return false;
  const void* fns[] = {(const void*)shrink_kernel,
                       (const void*)proj_kernel<false, false>, (const void*)proj_kernel<true, false>,
                       (const void*)proj_kernel<false, true>, (const void*)proj_kernel<true, true>,
                       (const void*)wgrad_kernel<16, 256>, (const void*)wgrad_kernel<16, 128>,
                       (const void*)wgrad_kernel<32, 256>, (const void*)wgrad_kernel<32, 128>,
                       (const void*)wgrad_kernel<64, 256>, (const void*)wgrad_kernel<64, 128>,
                       (const void*)wgrad_kernel<128, 128>};
  for (const void* f : fns) {
    cudaFuncAttributes a;
    if (cudaFuncGetAttributes(&a, f) != cudaSuccess) return false;
    if (cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)(kMaxSmem - a.sharedSizeBytes)) != cudaSuccess)
      return false;
  }
  for (int i = 0; i < 4; ++i) {
    d.clusters[i] = max_clusters(proj_kernel<false, false>, 1 << i, kMaxSmem);
    if (d.clusters[i] <= 0) return false;
  }
  d.sms = n;
  return true;
}
const Device* current_device() {
  constexpr int kMaxDevices = 64;
  static Device devices[kMaxDevices];
  static std::once_flag once[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  std::call_once(once[dev], [&] { init_device(devices[dev], dev); });
  return devices[dev].sms > 0 ? &devices[dev] : nullptr;
}

template <typename... Params, typename... Args>
cudaError_t launch(void (*kernel)(Params...), int grid, int threads, size_t smem, int cluster,
                   bool early, cudaStream_t s, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // early: may start before
  attr[1].val.programmaticStreamSerializationAllowed = 1;            // the last kernel ends
  cfg.attrs = attr;
  cfg.numAttrs = early ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Rows of X (or u) that a tile loads: all 128, or the batch's own rounded up to 8 (the rows of
// a swizzle atom).
int tile_rows(int T) { return T >= BM ? BM : (T + 7) / 8 * 8; }

// How the r values of [T][C] are found: by rows on the CUDA cores (rg ranks a CTA), or in tiles, whose
// contraction `split` CTAs of a cluster share and whose adapters' chunks `cy` clusters do.
struct ShrinkForm {
  int rg, split, cy, cols;
};
ShrinkForm shrink_form(const mok_lora_dims& d, int C, const Device& dev) {
  const int mt = (d.T + BM - 1) / BM, rp = padded_rank(d.r);
  ShrinkForm f = {};
  if (d.T <= kRowsMost && C <= 256 * kRowMaxPieces && (long long)d.T * rp * C <= kRowsProducts) {
    f.rg = 16;   // the fewest CTAs that still keep the SMs busy
    while (f.rg > 2 && d.T * (rp / f.rg) < dev.sms / 2) f.rg /= 2;
    return f;
  }
  const int distinct = std::min(std::min(d.n, d.T), BM);   // adapters of a tile, at most
  f.cols = distinct * rp <= 64 ? 64 : distinct * rp <= 128 ? 128 : 256;
  // How many ranks share a tile's contraction (a rank takes at least two steps), against how many
  // clusters share its chunks: the least estimated time in microseconds, 0.35 a step and 5 for
  // the start and the join of a chunk, over a batch whose tiles hold every adapter they can and
  // one of long runs (a single chunk), which the host cannot tell apart.
  const int kiters = (C + BK - 1) / BK, chunks = (distinct * rp + f.cols - 1) / f.cols;
  double best = 0;
  for (int i = 0; i < 4; ++i) {
    const int split = 1 << i, fit = dev.clusters[i];
    if (i > 0 && 2 * split > kiters) break;
    const int cy = std::max(1, std::min(chunks, fit / mt));
    const double waves = (mt + fit - 1) / fit, rounds = (chunks + cy - 1) / cy;
    const double t = waves * (rounds + 1) * ((kiters + split - 1) / split * 0.35 + 5.0);
    if (best == 0 || t < best) {
      best = t;
      f.split = split;
      f.cy = cy;
    }
  }
  return f;
}

// The r values of every row: in [T][C] against w [n][r][C]. early: the launch may start before
// the stream's last kernel ends.
mok_status run_shrink(const mok_lora_dims& d, int C, const void* in, const void* w,
                      const float* scale, const int32_t* ids, char* saved, bool pairs,
                      uint32_t* status, bool early, const Device& dev, cudaStream_t s) {
  const SavedParts sp = saved_parts(d);
  const int mt = (d.T + BM - 1) / BM;
  const int rp = padded_rank(d.r), nb = (rp + 31) / 32;
  const ShrinkForm f = shrink_form(d, C, dev);
  uint8_t* uq = reinterpret_cast<uint8_t*>(saved + sp.uq);
  int32_t* n_slots = reinterpret_cast<int32_t*>(saved + sp.n_slots);
  Slot* slots = reinterpret_cast<Slot*>(saved + sp.slots);
  if (f.rg > 0) {
    auto go = [&](auto rg) {
      constexpr int RG = decltype(rg)::value;
      // every rank that the MMAs read is written, padding too
      const int groups = rp / RG;
      ShrinkRowsParams p = {d.T, C, d.n, d.r, nb, groups, static_cast<const __nv_bfloat16*>(in),
                            static_cast<const __nv_bfloat16*>(w), ids, scale, uq, n_slots, slots, pairs};
      return launch(shrink_rows_kernel<RG>, d.T * groups + mt, kRowThreads, 0, 1, early, s, p);
    };
    const cudaError_t e = f.rg == 16  ? go(std::integral_constant<int, 16>{})
                          : f.rg == 8 ? go(std::integral_constant<int, 8>{})
                          : f.rg == 4 ? go(std::integral_constant<int, 4>{})
                                      : go(std::integral_constant<int, 2>{});
    return e == cudaSuccess ? MOK_OK : MOK_ERR_CUDA;
  }
  ShrinkParams p = {};
  p.T = d.T;
  p.n = d.n;
  p.r = d.r;
  p.rp = rp;
  p.nb = nb;
  p.kiters = (C + BK - 1) / BK;
  p.cols = f.cols;
  p.split = f.split;
  p.cy = f.cy;
  p.a_bytes = tile_rows(d.T) * BK * 2;
  // an MMA reads 128 rows from a stage's start, past a short batch's own: in bounds for the
  // last stage too
  p.tail = A_BYTES - p.a_bytes;
  const int fixed = BM * (rp + 4) * 4 + p.tail + kBarBytes + 1024;
  p.ring_bytes = (int)((kMaxSmem - 2 * sizeof(TileSlots) - fixed) / 1024 * 1024);
  p.pairs = pairs;
  p.ids = ids;
  p.scale = scale;
  p.uq = uq;
  p.n_slots = n_slots;
  p.slots = slots;
  p.status = status;
  CUtensorMap xm, am;
  if (!make_map(&xm, in, true, C, d.T, 0, tile_rows(d.T)) || !make_map(&am, w, true, C, d.r, d.n, p.rp))
    return MOK_ERR_CUDA;
  const size_t smem = (size_t)p.ring_bytes + fixed;
  return launch(shrink_kernel, mt * p.cy * p.split, kThreads, smem, p.split, early, s, xm, am, p) ==
                 cudaSuccess
             ? MOK_OK
             : MOK_ERR_CUDA;
}

// Form of the projection for [T][C] x [C][cols]: the candidate with the least estimated time,
// in microseconds: waves x (steps x time of a step + fixed) + the last epilogue. A step's time
// is the largest of the tensor core's, its bytes' way into the SM's shared memory, all SMs'
// out of L2, W's out of HBM (narrow 64-column pieces of its rows at two thirds of the rate),
// and the memory's latency over the ring's stages. The constants are fitted to the times of
// every form, 1 to 8192 rows and 256 x 256 to 7168 x 2048. At 96 shapes of that range (eight
// adapters of rank 16, in any order up to 128 rows and packed above) the choice costs 2.1% against
// the best form on average, at most 3% at 82 of them and 26% at the worst (2048 rows, 4096 to 1000:
// 192 columns 35.5 us, pairs 28.2). ext: the adapters' stages of a tile, an estimate.
struct ProjForm {
  int NT, split, pair, stages, stage_bytes;
  size_t smem;
};
// Tiles of the last wave of pairs that are run as halves: all of them if they then still fit
// one wave.
int pair_tail(int tiles, const Device& dev) {
  const int rest = tiles % dev.clusters[1];
  return 2 * rest <= dev.clusters[1] ? rest : 0;
}
ProjForm choose_form(int T, int kiters, int ext, int cols, const Device& dev) {
  const int mt = (T + BM - 1) / BM, a_bytes = tile_rows(T) * BK * 2;
  ProjForm best = {};
  double best_t = 0;
  for (int nt : {256, 192, 128, 64}) {
    for (int pair = 0; pair <= 1; ++pair) {
      for (int i = 0; i < 4; ++i) {
        const int split = 1 << i;
        if (pair && (nt != 256 || split > 1 || mt < 2)) continue;
        if (split > 1 && (kiters < 2 * split || nt > 128)) continue;
        ProjForm f;
        f.NT = nt;
        f.split = split;
        f.pair = pair;
        f.stage_bytes = a_bytes + (pair ? nt / 2 : nt) * 128;
        const size_t fixed = (split == 1 ? 8 * kStagingBox : 0) + kBarBytes + 1024;
        const size_t tail = A_BYTES - a_bytes;   // an MMA reads 128 rows (see run_shrink)
        // a cluster's partial tile lies over the stages
        const size_t red = split == 1 ? 0 : (size_t)std::min(BM, (T + 31) / 32 * 32) * (nt + 4) * 4;
        f.stages = std::min<int>(kMaxStages, (int)((kMaxSmem - fixed - tail) / f.stage_bytes));
        if (f.stages < 3 || (size_t)f.stages * f.stage_bytes < red) continue;
        f.smem = (size_t)f.stages * f.stage_bytes + tail + fixed;
        const double tiles = (double)((cols + nt - 1) / nt) * (pair ? (mt + 1) / 2 : mt);
        const double cap = dev.clusters[pair ? 1 : i];
        const double waves = std::ceil(tiles / cap);
        const double live = std::min(tiles, cap) * (pair ? 2 : split);   // CTAs at once
        const double w_bytes = (pair ? nt / 2 : nt) * 128;
        double hbm = w_bytes / mt * std::max(live / 5.2e6, 1 / 6.6e4);
        if (mt == 1 && nt == 64) hbm *= 1.5;
        const double step = std::max({0.0014 * nt, f.stage_bytes / 1.8e5, live * f.stage_bytes / 1.32e7,
                                      hbm, 0.42 / f.stages});
        const double fill = std::min(T, BM) / (double)BM;   // of a tile's rows
        const double fixed_t = pair ? 2.1 : split == 1 ? 1.7 : 2.8 + 4.3 * fill * nt / 128;
        const double t = waves * (std::ceil((double)(kiters + ext) / split) * step + fixed_t) +
                         (split == 1 ? 2.75 * fill * nt / 256 : 0.0);
        if (best_t == 0 || t < best_t) {
          best_t = t;
          best = f;
        }
      }
    }
  }
  return best;
}

// The form of [T][C] W (C = 0: no W), with or without the adapters' part.
ProjForm form_of(const mok_lora_dims& d, int C, int cols, bool adapters, const Device& dev) {
  const int rp = padded_rank(d.r), nb = (rp + 31) / 32, rb = std::min(rp, 32);
  // Short batches are mostly rows of different requests, long ones mostly long runs of one; an
  // adapter stage takes about as long as two steps over W. A long batch of many adapters in any
  // order runs more steps than it is counted for here.
  const int slots = adapters ? (d.T <= BM ? std::min(d.n, d.T) : 2) : 0;
  return choose_form(d.T, (C + BK - 1) / BK, 2 * nb * ((slots * rb + 63) / 64), cols, dev);
}

int form_tiles(const mok_lora_dims& d, const ProjForm& f, int cols) {
  const int mt = (d.T + BM - 1) / BM;
  return (f.pair ? (mt + 1) / 2 : mt) * ((cols + f.NT - 1) / f.NT);
}

// out [T][cols] = in [T][C] W (trans: W^T) + the low-rank part. W == null: that part alone;
// parts == null: no such part.
mok_status run_proj(const mok_lora_dims& d, const ProjForm& f, int C, int cols, bool trans,
                    const void* in, const void* W, const char* parts, const void* expand,
                    const int32_t* ids, void* out, mok_out_dtype type, uint32_t* status, bool early,
                    const Device& dev, cudaStream_t s) {
  const SavedParts sp = saved_parts(d);
  ProjParams p = {};
  p.T = d.T;
  p.out_cols = cols;
  p.n = d.n;
  p.kiters = W ? (C + BK - 1) / BK : 0;
  p.m_tiles = (d.T + BM - 1) / BM;
  p.rp = padded_rank(d.r);
  p.nb = (p.rp + 31) / 32;
  p.rb = std::min(p.rp, 32);
  p.out_bf16 = type == MOK_OUT_BF16;
  p.NT = f.NT;
  p.split = f.split;
  p.n_tiles = (cols + p.NT - 1) / p.NT;
  p.a_bytes = tile_rows(d.T) * BK * 2;
  p.stage_bytes = f.stage_bytes;
  p.stages = f.stages;
  if (parts) {
    p.n_slots = reinterpret_cast<const int32_t*>(parts + sp.n_slots);
    p.slots = reinterpret_cast<const Slot*>(parts + sp.slots);
  }
  p.ids = ids;
  p.out = out;
  p.status = status;
  const int rows = tile_rows(d.T);
  CUtensorMap xm, wm, um, em, om;
  bool ok = make_map(&om, out, p.out_bf16, cols, d.T, 0, 32);
  if (W) {
    ok = ok && make_map(&xm, in, true, C, d.T, 0, rows);
    ok = ok && (trans ? make_map(&wm, W, true, C, cols, 0, 64) : make_map(&wm, W, true, cols, C, 0, BK));
  } else {
    xm = wm = om;   // not read
  }
  if (parts) {
    ok = ok && make_map(&um, parts + sp.uq, true, (uint64_t)p.nb * 64, d.T, 0, rows);
    ok = ok && make_map(&em, expand, true, cols, d.r, d.n, p.rb);
  } else {
    um = em = om;
  }
  if (!ok) return MOK_ERR_CUDA;
  const int csize = f.pair ? 2 : f.split;
  int tiles = form_tiles(d, f, cols);
  if (f.pair) {
    p.whole = tiles - pair_tail(tiles, dev);
    tiles += tiles - p.whole;
  }
  const int grid = f.split > 1 ? tiles * csize
                               : std::min(tiles, dev.clusters[f.pair]) * csize;
  auto go = [&](auto kernel) {
    return launch(kernel, grid, kThreads, f.smem, csize, early, s, xm, wm, um, em, om, p);
  };
  const cudaError_t e =
      trans ? (f.pair ? go(proj_kernel<true, true>) : go(proj_kernel<true, false>))
            : (f.pair ? go(proj_kernel<false, true>) : go(proj_kernel<false, false>));
  return e == cudaSuccess ? MOK_OK : MOK_ERR_CUDA;
}

// Columns of a CTA of the weight gradients, and the row shares of a block of columns: one wave of
// clusters, at least two stages a share. 256 columns read u half as often, 128 make more CTAs of few
// rows. Backward with four packed adapters, 128 against 256 columns, in us:
//   7168 and 2048  rank 16: 512 rows 31.7 and 33.6, 1536 rows 52.6 and 52.9, 2048 rows 60.4 and
//                  60.1, 8192 rows 181.7 and 170.1; rank 64: 512 rows 36.5 and 38.8, 2048 rows 66.8
//                  and 65.7, 8192 rows 193.5 and 181.0
//   1000 and 1000  rank 16: 512 rows 18.7 and 21.1, 2048 rows 30.0 and 28.8, 8192 rows 53.7 and 50.0
// At 2048 and 2048 the columns also decide how many CTAs share the rows, and the rule is off by up to
// 20%: rank 16, 512 rows 24.7 and 21.0, 1024 rows 28.4 and 23.8, 2048 rows 34.3 and 35.5, 8192 rows
// 77.5 and 80.2.
struct WgradForm {
  int cols, split;
};
WgradForm wgrad_form(const mok_lora_dims& d, const Device& dev) {
  WgradForm f;
  f.cols = d.T >= 2048 && padded_rank(d.r) <= 64 ? 256 : 128;
  const int tiles = (d.K + f.cols - 1) / f.cols + (d.N + f.cols - 1) / f.cols;
  int i = 0;
  while (i < 3 && d.T > (2 << i) * kWgRows && tiles <= dev.clusters[i + 1]) ++i;
  f.split = 1 << i;
  return f;
}

mok_status run_wgrad(const mok_lora_dims& d, const char* uq, const char* vq, const void* xa,
                     const void* dY, const char* ws, const WorkParts& wp, void* dA, void* dB,
                     mok_out_dtype type, uint32_t* status, const Device& dev, cudaStream_t s) {
  const WgradForm f = wgrad_form(d, dev);
  auto go = [&](auto rp, auto cols) {
    using S = WgShape<decltype(rp)::value, decltype(cols)::value>;
    WgradParams p = {};
    p.side[0] = WgradSide{reinterpret_cast<const uint8_t*>(vq), static_cast<const __nv_bfloat16*>(xa),
                          dA, d.K, (d.K + S::N - 1) / S::N};
    p.side[1] = WgradSide{reinterpret_cast<const uint8_t*>(uq), static_cast<const __nv_bfloat16*>(dY),
                          dB, d.N, (d.N + S::N - 1) / S::N};
    p.r = d.r;
    p.n = d.n;
    p.split = f.split;
    p.out_bf16 = type == MOK_OUT_BF16;
    p.off = reinterpret_cast<const int32_t*>(ws + wp.off);
    p.rows = reinterpret_cast<const int32_t*>(ws + wp.rows);
    p.status = status;
    const int tiles = p.side[0].ctiles + p.side[1].ctiles;
    return launch(wgrad_kernel<decltype(rp)::value, decltype(cols)::value>, tiles * p.split,
                  kWgThreads, S::SMEM, p.split, true, s, p);
  };
  using std::integral_constant;
  auto width = [&](auto rp) {
    return f.cols == 256 ? go(rp, integral_constant<int, 256>{}) : go(rp, integral_constant<int, 128>{});
  };
  cudaError_t e;
  switch (padded_rank(d.r)) {
    case 16: e = width(integral_constant<int, 16>{}); break;
    case 32: e = width(integral_constant<int, 32>{}); break;
    case 64: e = width(integral_constant<int, 64>{}); break;
    default: e = go(integral_constant<int, 128>{}, integral_constant<int, 128>{}); break;
  }
  return e == cudaSuccess ? MOK_OK : MOK_ERR_CUDA;
}

bool ok_dims(const mok_lora_dims* d) {
  return d && d->T >= 0 && d->T <= (1 << 24) && d->K >= 8 && d->N >= 8 && d->K % 8 == 0 &&
         d->N % 8 == 0 && d->K <= (1 << 20) && d->N <= (1 << 20) && d->n >= 1 &&
         d->n <= (1 << 20) && d->r >= 1 && d->r <= 128;
}
bool ok_ptr(const void* p, uintptr_t align) {
  return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (align - 1)) == 0;
}
bool ok_weights(const mok_lora_weights* w) {
  return w && ok_ptr(w->W, 16) && ok_ptr(w->A, 16) && ok_ptr(w->B, 16) && ok_ptr(w->scale, 4);
}
bool ok_type(mok_out_dtype t) { return t == MOK_OUT_BF16 || t == MOK_OUT_F32; }

}  // namespace
}  // namespace mok

extern "C" mok_status mok_lora_get_sizes(const mok_lora_dims* dims, mok_lora_sizes* out) {
  using namespace mok;
  if (!ok_dims(dims) || !out) return MOK_ERR_INVALID_ARG;
  out->saved_bytes = saved_parts(*dims).total;
  out->workspace_bytes = work_parts(*dims).total;
  return MOK_OK;
}

extern "C" mok_status mok_lora_fwd(const mok_lora_dims* dims, const mok_lora_weights* w,
                                   const void* x, const void* x_ad, const int32_t* ids, void* y,
                                   mok_out_dtype out, void* saved, uint32_t* status,
                                   void* stream) {
  using namespace mok;
  if (!ok_dims(dims) || !ok_weights(w) || !ok_type(out)) return MOK_ERR_INVALID_ARG;
  if (dims->T == 0) return MOK_OK;
  if (!ok_ptr(x, 16) || (x_ad && !ok_ptr(x_ad, 16)) || !ok_ptr(ids, 4) || !ok_ptr(y, 16) ||
      (status && !ok_ptr(status, 4)))
    return MOK_ERR_INVALID_ARG;
  if (!ok_ptr(saved, 256)) return MOK_ERR_WORKSPACE;
  const Device* dev = current_device();
  if (!dev) return MOK_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* sv = static_cast<char*>(saved);
  const ProjForm f = form_of(*dims, dims->K, dims->N, true, *dev);
  mok_status st = run_shrink(*dims, dims->K, x_ad ? x_ad : x, w->A, w->scale, ids, sv, f.pair, status,
                             false, *dev, s);
  if (st != MOK_OK) return st;
  return run_proj(*dims, f, dims->K, dims->N, false, x, w->W, sv, w->B, ids, y, out, status, true,
                  *dev, s);
}

extern "C" mok_status mok_lora_bwd(const mok_lora_dims* dims, const mok_lora_weights* w,
                                   const void* x, const void* x_ad, const int32_t* ids,
                                   const void* saved, const void* dY, void* dX, void* dXa,
                                   void* dA, void* dB, mok_out_dtype out, void* workspace,
                                   uint32_t* status, void* stream) {
  using namespace mok;
  if (!ok_dims(dims) || !ok_weights(w) || !ok_type(out)) return MOK_ERR_INVALID_ARG;
  if (!ok_ptr(dA, 16) || !ok_ptr(dB, 16)) return MOK_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dims->T == 0) {
    const size_t es = out == MOK_OUT_BF16 ? 2 : 4, nr = (size_t)dims->n * dims->r;
    if (cudaMemsetAsync(dA, 0, nr * dims->K * es, s) != cudaSuccess ||
        cudaMemsetAsync(dB, 0, nr * dims->N * es, s) != cudaSuccess)
      return MOK_ERR_CUDA;
    return MOK_OK;
  }
  if (!ok_ptr(x, 16) || !ok_ptr(ids, 4) || !ok_ptr(dY, 16) || !ok_ptr(dX, 16) ||
      (status && !ok_ptr(status, 4)))
    return MOK_ERR_INVALID_ARG;
  if (x_ad ? (!ok_ptr(x_ad, 16) || !ok_ptr(dXa, 16)) : dXa != nullptr) return MOK_ERR_INVALID_ARG;
  if (!ok_ptr(saved, 256) || !ok_ptr(workspace, 256)) return MOK_ERR_WORKSPACE;
  const Device* dev = current_device();
  if (!dev) return MOK_ERR_CUDA;
  const mok_lora_dims& d = *dims;
  const char* sv = static_cast<const char*>(saved);
  char* ws = static_cast<char*>(workspace);
  const WorkParts wp = work_parts(d);
  // row lists, v, weight gradients, dX: each launch starts its set-up while the one before it
  // drains, and waits for it before it reads or writes anything that it produced
  bucket_kernel<<<d.n, kBucketThreads, 0, s>>>(d.T, d.n, ids, reinterpret_cast<int32_t*>(ws + wp.off),
                                               reinterpret_cast<int32_t*>(ws + wp.rows));
  if (cudaGetLastError() != cudaSuccess) return MOK_ERR_CUDA;
  // with x_ad the adapters' part is a product of its own
  const ProjForm f = form_of(d, d.N, d.K, !x_ad, *dev);
  const ProjForm fa = x_ad ? form_of(d, 0, d.K, true, *dev) : f;
  mok_status st = run_shrink(d, d.N, dY, w->B, w->scale, ids, ws, fa.pair, status, true, *dev, s);
  if (st != MOK_OK) return st;
  st = run_wgrad(d, sv + wp.v.uq, ws + wp.v.uq, x_ad ? x_ad : x, dY, ws, wp, dA, dB, out,
                 status, *dev, s);
  if (st != MOK_OK) return st;
  st = run_proj(d, f, d.N, d.K, true, dY, w->W, x_ad ? nullptr : ws, w->A, ids, dX, out, status, true,
                *dev, s);
  if (st != MOK_OK || !x_ad) return st;
  return run_proj(d, fa, 0, d.K, true, nullptr, nullptr, ws, w->A, ids, dXa, out, status, false, *dev,
                  s);
}

extern "C" mok_status mok_lora_get_status(uint32_t* status, void* stream) {
  using namespace mok;
  if (!ok_ptr(status, 4)) return MOK_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint32_t bits = 0;
  if (cudaMemcpyAsync(&bits, status, 4, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaMemsetAsync(status, 0, 4, s) != cudaSuccess || cudaStreamSynchronize(s) != cudaSuccess)
    return MOK_ERR_CUDA;
  return (bits & kErrTimeout) ? MOK_ERR_TIMEOUT : MOK_OK;
}

extern "C" mok_status mok_lora_get_forms(const mok_lora_dims* dims, int backward, int own_input,
                                         mok_lora_forms* out) {
  using namespace mok;
  if (!ok_dims(dims) || !out) return MOK_ERR_INVALID_ARG;
  const Device* dev = current_device();
  if (!dev) return MOK_ERR_CUDA;
  *out = {};
  if (dims->T == 0) return MOK_OK;
  const mok_lora_dims& d = *dims;
  const int C = backward ? d.N : d.K, cols = backward ? d.K : d.N;
  auto describe = [&](const ProjForm& f) {
    mok_lora_proj_form o = {f.NT, f.split, f.pair, 0};
    if (f.pair) o.halved = pair_tail(form_tiles(d, f, cols), *dev);
    return o;
  };
  const bool apart = backward && own_input;
  out->proj = describe(form_of(d, C, cols, !apart, *dev));
  if (apart) out->adapters = describe(form_of(d, 0, cols, true, *dev));
  const ShrinkForm s = shrink_form(d, C, *dev);
  out->u_ranks = s.rg;
  out->u_split = s.split;
  out->u_chunks = s.cy;
  if (backward) {
    const WgradForm w = wgrad_form(d, *dev);
    out->grad_columns = w.cols;
    out->grad_split = w.split;
  }
  return MOK_OK;
}
