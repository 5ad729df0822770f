// What the gated scan's kernels that carry a state along the tokens share: tiles of a row,
// handed out in order, and the states that enter them (see gated_scan.cu).
#pragma once

#include <algorithm>
#include <type_traits>

#include "gated_scan.cuh"

namespace m2 {

static __device__ unsigned int g_gs_errors = 0;
static __device__ unsigned int g_gs_stall = 0;  // mamba2_debug_stall_waits

namespace {

// Channels of a tile: half a warp takes two each.  (Wider tiles would be shorter: more of
// a row's tiles, each waiting for the one before, would be under way at once.  64 channels
// by 64 tokens: 475 against 447 us at 32768 tokens of 7168 channels with z, before the power cap.)
constexpr int kWidth = 32;
constexpr int kLanes = kWidth / 2;
constexpr int kWarps = 4;           // that compute
constexpr int kSegs = 2 * kWarps;   // segments of a tile's tokens: one for each half warp
constexpr int kThreads = 32 * (kWarps + 1);
// The state entering a tile is put together from that left by the `back`th tile before
// it and the maps of those between, one after the other: E(t + 1) = A(t) E(t) + H(t),
// rounded the same whatever `back` is.  8 where a step has many tiles (that state is then
// there, and only the maps of tiles under way are waited for: 43 against 47 us with 32 at
// 4096 tokens of 5120 channels, 126 against 149 for four such rows); 32 where a narrow row's
// tiles are nearly all under way at once, for a chain of fewer links (37 against 45 us at
// 32768 tokens of 64 channels; equal at 768).
constexpr int kNear = 8, kFar = 32;
constexpr int kFarBelow = 24;  // tiles of a step
constexpr int kBatch = 4;      // maps read at once

// Bits of a token's mark in packed rows: (sequence << 2) | last << 1 | first.
constexpr int kFirst = 1, kLast = 2;

struct Maps {
  CUtensorMap m[5];
};

// Division of numbers below 2^30 by one known on the host.
struct Divide {
  unsigned long long m;
  __device__ __forceinline__ int of(int t) const {
    return m == 0 ? t : (int)__umul64hi((unsigned long long)t, m);
  }
};
inline Divide divide_by(int d) {  // floor(2^64 / d) + 1: exact while t d < 2^64
  return Divide{d == 1 ? 0 : ~0ull / (unsigned)d + 1};
}

struct Scan {
  const float *ncs;  // -c softplus(lam) log2(e) of each channel, padded with zeros
  int64_t L;
  int D, nblk, steps, rows, tiles, back;  // steps: tiles along a row's tokens
  const int *marks;         // packed rows: [L], else null
  const unsigned int *bad;  // packed rows: wrong offsets
  const float *first;       // [rows][D] the states entering the rows, or null (packed: each sequence's)
  float4 *maps;             // [tiles][kLanes]: the tiles' maps
  float2 *states;           // [tiles][kLanes]: the states they leave
  unsigned int *ticket;
  Divide by_nblk, by_rows;
};

struct Tile {
  int cb, row, step, left;
};

template <typename T_, int TENSORS, int TOKENS> struct Shared {
  using T = T_;
  static_assert(kWarps == 4, "resets");
  static constexpr int kTensors = TENSORS, kTile = TOKENS, kStages = 2;
  static constexpr int kTokens = TOKENS / kSegs;        // of a thread
  static constexpr int kRow = kWidth * (int)sizeof(T);  // bytes of a token
  static constexpr int kTensor = kTile * kRow;
  alignas(128) unsigned char in[kStages][kTensors * kTensor];
  alignas(16) int marks[kStages][kTile];
  alignas(16) float ncs[kStages][kWidth];
  float4 seg[2][kSegs][kLanes];
  float2 enter[2][kLanes];
  alignas(16) int resets[2][kWarps];  // packed rows: a sequence begins among the warp's tokens
  uint64_t full[kStages], segs[2];
  Tile tile[kStages];
  int dead;  // a wait ran out: everybody leaves after the next `entered`
};

// The counter and the records reset, the decays' factor per channel, and for packed rows the
// offsets checked, the tokens marked and the states of empty sequences written (those of
// `empty_in`, or zero).
__global__ void gs_prep_kernel(const float *lam, float c, int D, float *ncs, uint4 *records,
                               int64_t nrecords, unsigned int *ticket, const int32_t *cu, int64_t batch,
                               int64_t L, int *marks, unsigned int *bad,
                               const float *empty_in, float *empty_out) {
  launch_dependents();
  grid_dependency_wait();
  const int64_t at = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t all = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = at; i < (D + 63) / 64 * 64; i += all)
    ncs[i] = i < D ? -c * softplus_f(lam[i]) * kLog2e : 0.0f;
  for (int64_t i = at; i < nrecords; i += all)
    records[i] = make_uint4(kUnset, kUnset, kUnset, kUnset);
  if (at == 0) *ticket = 0;
  if (cu == nullptr) return;
  // every block looks at all offsets, so that none acts on wrong ones
  int wrong = 0;
  for (int64_t s = threadIdx.x; s < batch; s += blockDim.x) wrong |= cu[s + 1] < cu[s];
  if (threadIdx.x == 0) wrong |= cu[0] != 0 || cu[batch] != L;
  wrong = __syncthreads_or(wrong);
  if (at == 0) {
    *bad = wrong ? 1u : 0u;
    if (wrong) atomicOr(&g_gs_errors, kErrSeqlens);
  }
  if (wrong) return;
  for (int64_t t = at; t < L; t += all) {
    int64_t lo = 0, hi = batch - 1;  // the sequence of token t: the first that ends after it
    while (lo < hi) {
      const int64_t mid = (lo + hi) >> 1;
      if (cu[mid + 1] > t) hi = mid;
      else lo = mid + 1;
    }
    marks[t] = (int)(lo << 2) | (cu[lo] == t ? kFirst : 0) | (cu[lo + 1] - 1 == t ? kLast : 0);
  }
  if (empty_out == nullptr) return;
  // a warp for 1024 channels of a sequence, all read before any is written: one warp for a whole
  // row, 32 channels after the other, took 54 us for one empty sequence of 4096 channels
  constexpr int kQuads = 8;
  const int pieces = (D + 128 * kQuads - 1) / (128 * kQuads);
  const int64_t warp = at / 32, together = all / 32 / pieces;  // sequences looked at at once
  const int d0 = (int)(warp % pieces) * (128 * kQuads) + 4 * (threadIdx.x % 32);
  if (warp >= together * pieces) return;
  for (int64_t s = warp / pieces; s < batch; s += together) {
    if (cu[s + 1] != cu[s]) continue;
    float4 v[kQuads];
#pragma unroll
    for (int k = 0; k < kQuads; ++k) {
      v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (empty_in != nullptr && d0 + 128 * k < D)
        v[k] = *reinterpret_cast<const float4 *>(empty_in + s * D + d0 + 128 * k);
    }
#pragma unroll
    for (int k = 0; k < kQuads; ++k)
      if (d0 + 128 * k < D) *reinterpret_cast<float4 *>(empty_out + s * D + d0 + 128 * k) = v[k];
  }
}

// The block's named barriers.  All wait in hardware: warps that ask an mbarrier again and
// again took a third of the instructions issued.
__device__ __forceinline__ void segments_done() {  // the computing warps
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory");
}
__device__ __forceinline__ void entered_wait(int half) {  // the computing warps, for the fifth
  asm volatile("bar.sync %0, %1;" ::"r"(2 + half), "n"(kThreads) : "memory");
}
__device__ __forceinline__ void entered_signal(int half) {
  asm volatile("bar.arrive %0, %1;" ::"r"(2 + half), "n"(kThreads) : "memory");
}

// A block's start: false if there is nothing to do.
template <typename S, bool PACKED> __device__ __forceinline__ bool begin(S &sm, const Scan &p) {
  const bool stalled = test_stall(&g_gs_stall, &g_gs_errors);
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) mbar_init(&sm.full[s], 1);
    for (int s = 0; s < 2; ++s) mbar_init(&sm.segs[s], kWarps);
    sm.dead = 0;
    fence_mbar_init();
  }
  __syncthreads();
  // (every block waits, so that what waits for this kernel has waited for the one before)
  grid_dependency_wait();
  return !(stalled || (PACKED && *p.bad));
}

// The segments before `seg` (in the order of the scan) as one map.
template <bool PACKED, typename S>
__device__ __forceinline__ float4 compose_before(const S &sm, int half, int seg, int lane) {
  if (PACKED) {
    const int4 r = *reinterpret_cast<const int4 *>(sm.resets[half]);
    if (r.x | r.y | r.z | r.w) {
      float4 pre = make_float4(1.0f, 1.0f, 0.0f, 0.0f);
#pragma unroll
      for (int k = 0; k < kSegs - 1; ++k)
        if (k < seg) pre = gs_then(pre, sm.seg[half][k][lane]);
      return pre;
    }
  }
  F2 A = f2(1.0f), H = f2(0.0f);
#pragma unroll
  for (int k = 0; k < kSegs - 1; ++k)
    if (k < seg) {
      const float4 m = sm.seg[half][k][lane];
      A = mul2(A, f2(m.x, m.y));
      H = fma2(f2(m.x, m.y), H, f2(m.z, m.w));
    }
  const float2 x = unpack(A), y = unpack(H);
  return make_float4(x.x, x.y, y.x, y.y);
}

// Between the segments' maps and the states that enter them: the last segment's threads
// publish the tile's map and the state it leaves; every thread gets the state entering
// its segment.  False if a wait ran out.
template <bool PACKED, typename S>
__device__ __forceinline__ bool exchange(S &sm, const Scan &p, const Tile &q, int half, int seg,
                                         int lane, float4 map, float2 *h) {
  segments_done();
  const float4 pre = compose_before<PACKED>(sm, half, seg, lane);
  const int64_t at = (int64_t)((q.step * p.rows + q.row) * p.nblk + q.cb) * kLanes + lane;
  const bool tells = seg == kSegs - 1 && q.step < p.steps - 1;
  if (tells) {
    map = gs_then(pre, map);  // of the tile
    if (q.step > 0) record_put(p.maps + at, map);
  }
  entered_wait(half);
  if (*reinterpret_cast<volatile int *>(&sm.dead)) return false;
  const float2 enter = sm.enter[half][lane];
  if (tells) {
    const float2 leave = gs_through(map, enter);
    record_put(p.states + at, leave);
    if (q.step == 0)  // known whole: nothing before it counts
      record_put(p.maps + at, make_float4(-0.0f, -0.0f, leave.x, leave.y));
  }
  *h = gs_through(pre, enter);
  return true;
}

// The warp beside the computing ones: it fetches the tiles and looks up the states that
// enter them.  REVERSE: the steps go from the rows' last tokens to the first.
template <typename S, bool PACKED, bool REVERSE>
__device__ __forceinline__ void look_up(S &sm, const Maps &in, const Scan &p) {
  const int lane = threadIdx.x & 31, l = lane % kLanes;  // (both halves read the same records)
  const int per_step = p.rows * p.nblk;
  // one lane: tile t's copies, into stage s
  auto fetch = [&](int s, int t) {
    Tile q;
    const int of_rows = p.by_nblk.of(t);
    q.left = p.tiles - t;
    q.cb = t - of_rows * p.nblk;
    q.step = p.by_rows.of(of_rows);
    q.row = of_rows - q.step * p.rows;
    sm.tile[s] = q;
    if (q.left <= 0) {
      mbar_arrive(&sm.full[s]);
      return;
    }
    const int t0 = (REVERSE ? p.steps - 1 - q.step : q.step) * S::kTile;
    const int n = (int)min((int64_t)S::kTile, p.L - t0);
    // (whole 16-byte groups of marks; the array is padded)
    const uint32_t mark_bytes = PACKED ? (n * 4 + 15) / 16 * 16 : 0;
    mbar_arrive_expect_tx(&sm.full[s], S::kTensors * S::kTensor + kWidth * 4 + mark_bytes);
#pragma unroll
    for (int k = 0; k < S::kTensors; ++k)
      tma_load_3d(sm.in[s] + k * S::kTensor, &in.m[k], q.cb * kWidth, t0, q.row, &sm.full[s]);
    bulk_g2s(sm.ncs[s], p.ncs + q.cb * kWidth, kWidth * 4, &sm.full[s]);
    if (PACKED) bulk_g2s(sm.marks[s], p.marks + t0, mark_bytes, &sm.full[s]);
  };
  if (lane == 0) {
    fetch(0, (int)atomicAdd(p.ticket, 1u));
    // by then the other blocks have their first tile too: no block holds two neighbours
    // that it would work on one after the other while others wait for the second
    mbar_wait_parked(&sm.full[0], 0, &g_gs_errors);
    fetch(1, (int)atomicAdd(p.ticket, 1u));
  }
  __syncwarp();

  for (int it = 0;; ++it) {
    const int s = it % S::kStages, half = it & 1;
    const uint32_t phase = (it >> 1) & 1;
    const Tile q = sm.tile[s];
    if (q.left <= 0) return;  // so is every later tile's: no copy is under way
    int next = 0;
    if (lane == 0) next = (int)atomicAdd(p.ticket, 1u);  // wanted when the segments are there
    const int d = q.cb * kWidth + 2 * l;
    const int tile = q.step * per_step + q.row * p.nblk + q.cb;
    const int between = min(q.step, p.back - 1);
    bool fetched = false, entered = false, based = q.step < p.back, alive = true;
    int folded = 0;  // maps, of those between
    const int64_t stride = (int64_t)per_step * kLanes;
    const float2 *base = p.states + (int64_t)tile * kLanes + l - p.back * stride;
    const float4 *maps = p.maps + (int64_t)tile * kLanes + l - between * stride;
    float2 h = make_float2(0.0f, 0.0f);
    if (!PACKED && q.step == 0 && p.first != nullptr && d < p.D)
      h = *reinterpret_cast<const float2 *>(p.first + (int64_t)q.row * p.D + d);
    // asks for the next maps (and the base), and folds those that are there without a gap
    auto ask = [&]() {
      float2 b = make_float2(0.0f, 0.0f);
      float4 m[kBatch];
      if (!based) b = record_get(base);
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (folded + k < between) m[k] = record_get(maps + k * stride);
      unsigned int there = based || is_set(b) ? 1u << 31 : 0u;
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (folded + k < between && is_set(m[k])) there |= 1u << k;
      there = __reduce_and_sync(0xffffffffu, there);
      if (!(there >> 31)) return;
      if (!based) h = b;
      based = true;
      const int run = __ffs(~there) - 1;
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (k < run) h = gs_through(m[k], h);
      folded += run;
      maps += run * stride;
      entered = folded == between;
      if (entered) {
        sm.enter[half][l] = h;
        entered_signal(half);
      }
    };
    auto refill = [&]() {
      if (lane == 0) fetch(s, next);  // every warp is done with the stage
      __syncwarp();
      fetched = true;
    };
    // Few instructions here count, and short code: this warp shares its scheduler with a
    // computing one, for which the others wait, and the instruction cache with all.
    unsigned long long since = 0;
    for (int asked = 0; !entered && alive; ++asked) {
      if (!fetched && __all_sync(0xffffffffu, mbar_test(&sm.segs[half], phase))) refill();
      ask();
      if (asked % 64 == 63) {
        const unsigned long long now = __shfl_sync(0xffffffffu, globaltimer_ns(), 0);
        if (since == 0) since = now;
        alive = now - since <= kWaitLimitNs;
      }
    }
    if (alive && !fetched) {
      alive = __all_sync(0xffffffffu, mbar_wait_bounded(&sm.segs[half], phase, &g_gs_errors));
      if (alive) refill();
    }
    if (!alive) {
      // what this block has under way lands before the warp leaves, and nobody waits for it
      sm.dead = 1;
      __syncwarp();
      entered_signal(entered ? half ^ 1 : half);
      if (lane == 0) {
        atomicOr(&g_gs_errors, kErrWaitTimeout);
        for (int i = it + fetched; i < it + fetched + S::kStages; ++i)
          mbar_wait_bounded(&sm.full[i % S::kStages], (i / S::kStages) & 1, &g_gs_errors);
      }
      return;
    }
  }
}

// Where the parts of a scan's workspace are.
struct Plan {
  int nblk, steps;
  int64_t tiles;
  size_t ncs, maps, states, marks, total;
};
inline Plan plan_of(int64_t rows, int64_t L, int D, int tile_tokens, bool packed) {
  Plan p;
  p.nblk = (int)ceil_div(D, kWidth);
  p.steps = (int)ceil_div(L, tile_tokens);
  p.tiles = rows * p.steps * p.nblk;
  const size_t records = p.steps > 1 ? (size_t)align_up(p.tiles, 2) * kLanes : 0;
  p.ncs = 256;  // after the counter and the flag of wrong offsets
  p.maps = p.ncs + align_up((size_t)D * 4, 256);
  p.states = p.maps + records * 16;
  p.marks = p.states + records * 8;
  p.total = p.marks + (packed ? align_up((size_t)L * 4, 256) : 0);
  return p;
}

// Launches a kernel whose blocks may start while the one before drains (they wait for it; so
// none of its pointers may be __restrict__, which lets them be read before).  The first
// kernel of a call too: 2 us less for calls in turn, prefill 46.3 against 44.3 us at 4096
// tokens of 5120 channels.
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, size_t smem,
                             cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), ContextOnce &once, unsigned grid, int threads,
                             size_t smem, cudaStream_t stream, A... args) {
  if (!once.done()) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    once.set();
  }
  return launch_dependent(kernel, grid, threads, smem, stream, args...);
}

// The parameters of a scan over `a`'s rows whose workspace is at ws, and the launch that
// prepares it.
inline cudaError_t prepare(const GatedScanArgs &a, const Plan &w, char *ws, const float *first,
                           const float *empty_in, float *empty_out, Scan *p) {
  const bool packed = a.cu != nullptr;
  p->ncs = reinterpret_cast<float *>(ws + w.ncs);
  p->L = a.L;
  p->D = a.D;
  p->nblk = w.nblk;
  p->steps = w.steps;
  p->rows = (int)a.rows();
  p->tiles = (int)w.tiles;
  p->back = a.rows() * w.nblk < kFarBelow ? kFar : kNear;
  p->marks = packed ? reinterpret_cast<int *>(ws + w.marks) : nullptr;
  p->ticket = reinterpret_cast<unsigned int *>(ws);
  p->bad = p->ticket + 1;
  p->first = first;
  p->by_nblk = divide_by(w.nblk);
  p->by_rows = divide_by(p->rows);
  p->maps = reinterpret_cast<float4 *>(ws + w.maps);
  p->states = reinterpret_cast<float2 *>(ws + w.states);
  const int64_t nrecords = (int64_t)(w.marks - w.maps) / 16;  // maps and states, side by side
  const int64_t work = std::max(std::max<int64_t>(a.D, nrecords), packed ? a.L : 0);
  return launch_dependent(gs_prep_kernel, (unsigned)std::min<int64_t>(ceil_div(work, 256), 148 * 4), 256, 0,
                          a.stream, a.lam, a.c, a.D, const_cast<float *>(p->ncs),
                          reinterpret_cast<uint4 *>(ws + w.maps), nrecords, p->ticket, a.cu, a.batch,
                          a.L, const_cast<int *>(p->marks), const_cast<unsigned int *>(p->bad),
                          empty_in, empty_out);
}

inline int sm_count() {
  static std::atomic<int> known[64] = {};
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  n = known[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 148;
    known[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

}  // namespace
}  // namespace m2
