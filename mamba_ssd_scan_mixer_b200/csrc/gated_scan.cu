// Prefill and decode step of the gated linear recurrence (gated_scan.cuh).
//
// Prefill reads every input once.  A tile is 128 (fp32: 64) tokens of 64 channels of a
// row; resident blocks take tiles in order, all channels of a stretch of tokens before
// the next stretch, from a counter:
//   1. the tile's x, r and g arrive by TMA, two tiles ahead of the arithmetic;
//   2. each thread of the eight computing warps turns the 16 (8) tokens of its two
//      channels into h_t = a_t h_{t-1} + b_t, keeps a and b in registers, and composes
//      them into the map of its segment, (A, H), in shared memory; the last of the
//      warps publishes the whole tile's map;
//   3. meanwhile a ninth warp looks up the state entering the tile: it folds the maps of
//      the tiles before it onto the state that one further back left.  When the
//      segments are there it fetches the tile after next;
//   4. each thread runs its tokens from that state and writes y; the last of the warps
//      has published the state that the tile leaves.
// Nothing makes the whole block wait: warps meet at mbarriers only.  Every state is put
// together in an order fixed by the tiles' numbers alone, so that results do not depend
// on timing.  A block waits only for tiles of lower numbers, whose blocks are running:
// the tiles are handed out in order.
#include <algorithm>
#include <type_traits>

#include "gated_scan.cuh"

namespace m2 {

static __device__ unsigned int g_gs_errors = 0;
static __device__ unsigned int g_gs_stall = 0;  // mamba2_debug_stall_waits

namespace {

constexpr int kWidth = 64;  // channels of a tile: two for each lane
constexpr int kWarps = 4;   // that compute
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kStages = 2;
// The state entering a tile is put together from that left by the `back`th tile before
// it and the maps of those between, one after the other: E(t + 1) = A(t) E(t) + H(t),
// rounded the same whatever `back` is.  8 where a step has many tiles (that state is then
// there, and only the maps of tiles under way are waited for); 32 where a narrow row's
// tiles are nearly all under way at once, for a chain of fewer links.
constexpr int kNear = 8, kFar = 32;
constexpr int kFarBelow = 24;  // tiles of a step
constexpr int kBatch = 8;      // maps read at once

// Blocks on an SM at once: what shared memory holds.
template <bool GATED> constexpr int kResident = GATED ? 3 : 4;
// Tokens of a tile: what the registers of a block's threads and the shared memory of
// two blocks to an SM hold.
template <typename T> constexpr int kTile = sizeof(T) == 2 ? 64 : 32;
template <typename T> constexpr int kTokens = kTile<T> / kWarps;  // of a thread

// Bits of a token's mark in packed rows: (sequence << 2) | last << 1 | first.
constexpr int kFirst = 1, kLast = 2;

struct Scan {
  const float *ncs;  // [nblk][64] -c softplus(lam) log2(e)
  int64_t L;
  int D, nblk, steps, rows, tiles, back;  // steps: tiles along a row's tokens
  const int *marks;         // packed rows: [L], else null
  const unsigned int *bad;  // packed rows: wrong offsets
  void *y;                  // or null: only the states entering the chunks are wanted
  const float *h_in;        // or null
  float *h_out, *ck;        // or null
  float4 *maps;             // [tiles][32]: the tiles' maps
  float2 *states;           // [tiles][32]: the states they leave
  unsigned int *ticket;
};

struct Tile {
  int cb, row, step, left;
};

template <typename T, bool GATED> struct Shared {
  static constexpr int kTensors = GATED ? 4 : 3;
  static constexpr int kRow = kWidth * (int)sizeof(T);  // bytes of a token
  static constexpr int kTensor = kTile<T> * kRow;
  alignas(128) unsigned char in[kStages][kTensors * kTensor];
  alignas(16) int marks[kStages][kTile<T>];
  alignas(16) float ncs[kStages][kWidth];
  float4 seg[2][kWarps][32];
  float2 enter[2][32];
  uint64_t full[kStages], segs[2];
  Tile tile[kStages];
  int dead;  // a wait ran out: everybody leaves after the next `entered`
};

// The counter and the records reset, the decays' factor per channel, and for packed rows the
// offsets checked, the tokens marked and the states of empty sequences written.
__global__ void gs_prep_kernel(const float *lam, float c, int D, float *ncs, uint4 *records,
                               int64_t nrecords, unsigned int *ticket, const int32_t *cu, int64_t batch,
                               int64_t L, int *marks, unsigned int *bad, float *h_out,
                               int states_in) {
  launch_dependents();
  const int64_t at = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t all = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = at; i < (D + kWidth - 1) / kWidth * kWidth; i += all)
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
  if (h_out != nullptr && !states_in)
    for (int64_t s = at / 32; s < batch; s += all / 32)  // a warp for a sequence
      if (cu[s + 1] == cu[s])
        for (int d = threadIdx.x % 32; d < D; d += 32) h_out[s * D + d] = 0.0f;
}

// The block's named barriers.  All wait in hardware: warps that ask an mbarrier again and
// again took a third of the instructions issued.
__device__ __forceinline__ void segments_done() {  // the computing warps
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory");
}
__device__ __forceinline__ void entered_wait(int half) {  // the computing warps, for the ninth
  asm volatile("bar.sync %0, %1;" ::"r"(2 + half), "n"(kThreads) : "memory");
}
__device__ __forceinline__ void entered_signal(int half) {
  asm volatile("bar.arrive %0, %1;" ::"r"(2 + half), "n"(kThreads) : "memory");
}

// Step 2: a and b of the thread's tokens, and their composition.  `begins`: the tokens (a
// bit each) that begin a sequence of packed rows.
template <typename T, bool FULL, bool RESETS, bool NEAR>
__device__ __forceinline__ float4 make_maps(const unsigned char *in, const int *marks,
                                            unsigned int begins, F2 ncs, int n, const Scan &p,
                                            int d, F2 (&a)[kTokens<T>], F2 (&b)[kTokens<T>]) {
  constexpr int kRow = Shared<T, false>::kRow, kTensor = Shared<T, false>::kTensor;
  F2 A = f2(1.0f), H = f2(0.0f);
#pragma unroll
  for (int i = 0; i < kTokens<T>; ++i) {
    const unsigned char *row = in + i * kRow;
    const Coeffs c =
        coefficients<NEAR>(gs_pair<T>(row), gs_clamped<T>(row + kTensor),
                           gs_clamped<T>(row + 2 * kTensor), ncs);
    a[i] = c.a;
    b[i] = c.b;
    if (!FULL && i >= n) {
      a[i] = f2(1.0f);
      b[i] = f2(0.0f);
    }
    if (RESETS && (begins >> i & 1)) {
      if (p.h_in != nullptr && d < p.D) {
        const float2 h =
            *reinterpret_cast<const float2 *>(p.h_in + (int64_t)(marks[i] >> 2) * p.D + d);
        b[i] = fma2(a[i], f2(h.x, h.y), b[i]);
      }
      A = f2(-0.0f);
      H = b[i];
    } else {
      A = mul2(A, a[i]);
      H = fma2(a[i], H, b[i]);
    }
  }
  const float2 x = unpack(A), y = unpack(H);
  return make_float4(x.x, x.y, y.x, y.y);
}

__device__ __forceinline__ void store_pair(float *p, float2 v) {
  *reinterpret_cast<float2 *>(p) = v;
}
__device__ __forceinline__ void store_pair(__nv_bfloat16 *p, float2 v) {
  *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(v.x, v.y);
}

// The ninth warp: step 3, and the copies of step 1.
template <typename T, bool PACKED, bool GATED>
__device__ __forceinline__ void look_up(Shared<T, GATED> &sm, const CUtensorMap &map_x,
                                        const CUtensorMap &map_r, const CUtensorMap &map_g,
                                        const CUtensorMap &map_z, const Scan &p) {
  using S = Shared<T, GATED>;
  const int lane = threadIdx.x & 31;
  const int per_step = p.rows * p.nblk;
  // one lane: tile t's copies, into stage s
  auto fetch = [&](int s, int t) {
    Tile q;
    q.left = p.tiles - t;
    q.cb = t % p.nblk;
    q.row = t / p.nblk % p.rows;
    q.step = t / per_step;
    sm.tile[s] = q;
    if (q.left <= 0) {
      mbar_arrive(&sm.full[s]);
      return;
    }
    const int t0 = q.step * kTile<T>, n = (int)min((int64_t)kTile<T>, p.L - t0);
    // (whole 16-byte groups of marks; the array is padded)
    const uint32_t mark_bytes = PACKED ? (n * 4 + 15) / 16 * 16 : 0;
    mbar_arrive_expect_tx(&sm.full[s], S::kTensors * S::kTensor + kWidth * 4 + mark_bytes);
    unsigned char *in = sm.in[s];
    tma_load_3d(in, &map_x, q.cb * kWidth, t0, q.row, &sm.full[s]);
    tma_load_3d(in + S::kTensor, &map_r, q.cb * kWidth, t0, q.row, &sm.full[s]);
    tma_load_3d(in + 2 * S::kTensor, &map_g, q.cb * kWidth, t0, q.row, &sm.full[s]);
    if (GATED) tma_load_3d(in + 3 * S::kTensor, &map_z, q.cb * kWidth, t0, q.row, &sm.full[s]);
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
    const int s = it % kStages, half = it & 1;
    const uint32_t phase = (it >> 1) & 1;
    const Tile q = sm.tile[s];
    if (q.left <= 0) return;  // so is every later tile's: no copy is under way
    int next = 0;
    if (lane == 0) next = (int)atomicAdd(p.ticket, 1u);  // wanted when the segments are there
    const int d = q.cb * kWidth + 2 * lane;
    const int tile = q.step * per_step + q.row * p.nblk + q.cb;
    const int between = min(q.step, p.back - 1);
    bool fetched = false, entered = false, based = q.step < p.back;
    int folded = 0;  // maps, of those between
    const float2 *base = p.states + ((int64_t)tile - (int64_t)p.back * per_step) * 32 + lane;
    const float4 *maps = p.maps + ((int64_t)tile - (int64_t)between * per_step) * 32 + lane;
    float2 h = make_float2(0.0f, 0.0f);
    if (!PACKED && q.step == 0 && p.h_in != nullptr && d < p.D)
      h = *reinterpret_cast<const float2 *>(p.h_in + (int64_t)q.row * p.D + d);
    unsigned long long since = 0;
    for (;;) {
      if (!entered) {
        float2 b = make_float2(0.0f, 0.0f);
        float4 m[kBatch];
        if (!based) b = record_get(base);
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
          if (folded + k < between) m[k] = record_get(maps + (int64_t)(folded + k) * per_step * 32);
        unsigned int there = based || is_set(b) ? 1u << 31 : 0u;
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
          if (folded + k < between && is_set(m[k])) there |= 1u << k;
        there = __reduce_and_sync(0xffffffffu, there);
        if (there >> 31) {
          if (!based) h = b;
          based = true;
          const int run = __ffs(~there) - 1;  // maps there without a gap
#pragma unroll
          for (int k = 0; k < kBatch; ++k)
            if (k < run) h = gs_through(m[k], h);
          folded += run;
          entered = folded == between;
        }
        if (entered) {
          sm.enter[half][lane] = h;
          entered_signal(half);
          constexpr int kPer = kGsChunk / kTile<T>;
          if (p.ck != nullptr && q.step % kPer == 0 && d < p.D) {
            const int64_t nch = (p.L + kGsChunk - 1) / kGsChunk;
            *reinterpret_cast<float2 *>(p.ck + ((int64_t)q.row * nch + q.step / kPer) * p.D + d) =
                h;
          }
        }
      }
      if (!fetched && __all_sync(0xffffffffu, entered ? mbar_try_wait(&sm.segs[half], phase)
                                                      : mbar_test(&sm.segs[half], phase))) {
        if (lane == 0) fetch(s, next);  // every warp is done with the stage
        __syncwarp();
        fetched = true;
      }
      if (fetched && entered) break;
      const unsigned long long now = globaltimer_ns();
      if (since == 0) since = now;
      if (__any_sync(0xffffffffu, now - since > kWaitLimitNs)) {
        // what this block has under way lands before the warp leaves, and nobody waits for it
        sm.dead = 1;
        __syncwarp();
        entered_signal(entered ? half ^ 1 : half);
        if (lane == 0) {
          atomicOr(&g_gs_errors, kErrWaitTimeout);
          for (int i = it + fetched; i < it + fetched + kStages; ++i)
            mbar_wait_bounded(&sm.full[i % kStages], (i / kStages) & 1, &g_gs_errors);
        }
        return;
      }
    }
  }
}

template <typename T, bool PACKED, bool GATED>
__global__ void __launch_bounds__(kThreads, kResident<GATED>)
    gs_prefill_kernel(const __grid_constant__ CUtensorMap map_x,
                      const __grid_constant__ CUtensorMap map_r,
                      const __grid_constant__ CUtensorMap map_g,
                      const __grid_constant__ CUtensorMap map_z, const Scan p) {
  extern __shared__ __align__(128) unsigned char raw[];
  using S = Shared<T, GATED>;
  S &sm = *reinterpret_cast<S *>(raw);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (test_stall(&g_gs_stall, &g_gs_errors)) return;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&sm.full[s], 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.segs[s], kWarps);
    }
    sm.dead = 0;
    fence_mbar_init();
  }
  __syncthreads();
  grid_dependency_wait();
  if (PACKED && *p.bad) return;
  if (warp == kWarps) {
    look_up<T, PACKED, GATED>(sm, map_x, map_r, map_g, map_z, p);
    return;
  }

  const int first = warp * kTokens<T>;
  for (int it = 0;; ++it) {
    const int s = it % kStages, half = it & 1;
    if (!mbar_wait_parked(&sm.full[s], (it / kStages) & 1, &g_gs_errors)) sm.dead = 1;
    const Tile q = sm.tile[s];
    if (q.left <= 0) return;
    const int t0 = q.step * kTile<T>, n = (int)min((int64_t)kTile<T>, p.L - t0);
    const int d = q.cb * kWidth + 2 * lane;
    const bool real = d < p.D;
    const float2 ncs = *reinterpret_cast<const float2 *>(&sm.ncs[s][2 * lane]);
    F2 a[kTokens<T>], b[kTokens<T>];
    const unsigned char *in = sm.in[s] + first * S::kRow + lane * (2 * (int)sizeof(T));
    const int *marks = sm.marks[s] + first;
    // packed rows: which of the warp's tokens begin and end a sequence
    unsigned int begins = 0, ends = 0;
    if (PACKED) {
      const int mark = lane < min(kTokens<T>, n - first) ? marks[lane] : 0;
      begins = __ballot_sync(0xffffffffu, mark & kFirst);
      ends = __ballot_sync(0xffffffffu, p.h_out != nullptr && (mark & kLast));
    }
    const F2 k = f2(ncs.x, ncs.y);
    float4 map;
    if (__all_sync(0xffffffffu, fminf(ncs.x, ncs.y) >= -0.5f) && begins == 0)
      map = n == kTile<T>
                ? make_maps<T, true, false, true>(in, marks, 0, k, n - first, p, d, a, b)
                : make_maps<T, false, false, true>(in, marks, 0, k, n - first, p, d, a, b);
    else
      map = make_maps<T, false, PACKED, false>(in, marks, begins, k, n - first, p, d, a, b);
    sm.seg[half][warp][lane] = map;
    typename Pair<T>::V gate[GATED ? kTokens<T> : 1];
    if (GATED) {
#pragma unroll
      for (int i = 0; i < kTokens<T>; ++i)
        gate[i] = *reinterpret_cast<const typename Pair<T>::V *>(in + i * S::kRow + 3 * S::kTensor);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.segs[half]);
    const int64_t token = (int64_t)q.row * p.L + t0 + first;
    segments_done();
    // the segments before this one as one map
    float4 pre = make_float4(1.0f, 1.0f, 0.0f, 0.0f);
    if (PACKED) {
      for (int k = 0; k < warp; ++k) pre = gs_then(pre, sm.seg[half][k][lane]);
    } else {
      F2 A = f2(1.0f), H = f2(0.0f);
#pragma unroll
      for (int k = 0; k < kWarps - 1; ++k)
        if (k < warp) {
          const float4 m = sm.seg[half][k][lane];
          A = mul2(A, f2(m.x, m.y));
          H = fma2(f2(m.x, m.y), H, f2(m.z, m.w));
        }
      const float2 x = unpack(A), y = unpack(H);
      pre = make_float4(x.x, x.y, y.x, y.y);
    }
    const int tile = (q.step * p.rows + q.row) * p.nblk + q.cb;
    const bool tells = warp == kWarps - 1 && q.step < p.steps - 1;
    if (tells) map = gs_then(pre, map);  // of the tile
    if (tells && q.step > 0) record_put(p.maps + (int64_t)tile * 32 + lane, map);
    entered_wait(half);
    if (*reinterpret_cast<volatile int *>(&sm.dead)) return;
    const float2 enter = sm.enter[half][lane];
    if (tells) {
      const float2 leave = gs_through(map, enter);
      record_put(p.states + (int64_t)tile * 32 + lane, leave);
      if (q.step == 0)  // known whole: nothing before it counts
        record_put(p.maps + (int64_t)tile * 32 + lane,
                   make_float4(-0.0f, -0.0f, leave.x, leave.y));
    }
    const float2 h = gs_through(pre, enter);
    F2 hh = f2(h.x, h.y);
    if (p.y != nullptr) {
      T *y = static_cast<T *>(p.y) + token * p.D + d;
      auto run = [&](auto all) {  // all: every token of every lane is stored, no sequence's end
#pragma unroll
        for (int i = 0; i < kTokens<T>; ++i) {
          if (!decltype(all)::value && PACKED && (begins >> i & 1)) hh = b[i];
          else hh = fma2(a[i], hh, b[i]);
          F2 o = hh;
          if (GATED) {
            const float2 z = Pair<T>::get(gate[i]);
            o = mul2(hh, mul2(f2(z.x, z.y), sigmoid2(f2(z.x, z.y))));
          }
          if (decltype(all)::value) {
            store_pair(y, unpack(o));
          } else if (real && i < n - first) {
            store_pair(y, unpack(o));
            if (PACKED && (ends >> i & 1))
              *reinterpret_cast<float2 *>(
                  p.h_out + (int64_t)(p.marks[t0 + first + i] >> 2) * p.D + d) = unpack(hh);
          }
          y += p.D;
        }
      };
      if (__all_sync(0xffffffffu, real && n - first >= kTokens<T> && (begins | ends) == 0))
        run(std::true_type());
      else run(std::false_type());
    }
    if (!PACKED && p.h_out != nullptr && q.step == p.steps - 1 && real && first < n &&
        n <= first + kTokens<T>)
      // (tokens behind the last leave the state as it is)
      *reinterpret_cast<float2 *>(p.h_out + (int64_t)q.row * p.D + d) = unpack(hh);
  }
}

template <typename T> struct In {
  const T *x, *r, *g, *z;
  int64_t ld_x, ld_r, ld_g, ld_z;
};

template <typename T>
__global__ void gs_step_kernel(In<T> in, const float *lam, float c, int64_t n2, int D, float *h,
                               T *y) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= n2) return;
  const int64_t b = i / (D / 2);
  const int d = 2 * (int)(i % (D / 2));
  const float2 x = ld2(in.x + b * in.ld_x + d), r = ld2(in.r + b * in.ld_r + d),
               g = ld2(in.g + b * in.ld_g + d);
  const Gate p = gs_gate(r.x, g.x, -c * softplus_f(lam[d])),
             q = gs_gate(r.y, g.y, -c * softplus_f(lam[d + 1]));
  float2 *hp = reinterpret_cast<float2 *>(h + b * D + d);
  float2 v = *hp;
  v.x = p.a * v.x + p.m * p.G * x.x;
  v.y = q.a * v.y + q.m * q.G * x.y;
  *hp = v;
  if (in.z != nullptr) {
    const float2 z = ld2(in.z + b * in.ld_z + d);
    v.x *= z.x * gs_sigmoid(z.x);
    v.y *= z.y * gs_sigmoid(z.y);
  }
  st2(y + b * D + d, v.x, v.y);
}

template <typename T> In<T> inputs(const GatedScanArgs &a) {
  return In<T>{static_cast<const T *>(a.x), static_cast<const T *>(a.r),
               static_cast<const T *>(a.g), static_cast<const T *>(a.z),
               a.ld_x,                      a.ld_r,
               a.ld_g,                      a.ld_z};
}

// Where the parts of the workspace are.
struct Plan {
  int nblk, steps;
  int64_t tiles;
  size_t ncs, maps, states, marks, total;
};
Plan plan_of(int64_t rows, int64_t L, int D, int io, bool packed) {
  Plan p;
  p.nblk = (int)ceil_div(D, kWidth);
  p.steps = (int)ceil_div(L, io == MAMBA2_BF16 ? kTile<__nv_bfloat16> : kTile<float>);
  p.tiles = rows * p.steps * p.nblk;
  const size_t records = p.steps > 1 ? (size_t)p.tiles * 32 : 0;
  p.ncs = 256;  // after the counter and the flag of wrong offsets
  p.maps = p.ncs + align_up((size_t)p.nblk * kWidth * 4, 256);
  p.states = p.maps + records * 16;
  p.marks = p.states + records * 8;
  p.total = p.marks + (packed ? align_up((size_t)L * 4, 256) : 0);
  return p;
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 148;
  return n;
}

template <typename T, bool PACKED, bool GATED>
cudaError_t launch(const GatedScanArgs &a, const CUtensorMap (&m)[4], const Scan &p) {
  constexpr size_t smem = sizeof(Shared<T, GATED>);
  static_assert(kResident<GATED> * (smem + 1024 + 256) <= 228 * 1024, "blocks to an SM");
  static ContextOnce once;
  if (!once.done()) {
    const cudaError_t e = cudaFuncSetAttribute(
        gs_prefill_kernel<T, PACKED, GATED>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    once.set();
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min(p.tiles, kResident<GATED> * sm_count()), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, gs_prefill_kernel<T, PACKED, GATED>, m[0], m[1], m[2], m[3], p);
}

template <typename T> cudaError_t prefill(const GatedScanArgs &a) {
  const int64_t rows = a.rows();
  const bool packed = a.cu != nullptr;
  const Plan w = plan_of(rows, a.L, a.D, a.io, packed);
  Scan p;
  p.ncs = reinterpret_cast<float *>(a.ws + w.ncs);
  p.L = a.L;
  p.D = a.D;
  p.nblk = w.nblk;
  p.steps = w.steps;
  p.rows = (int)rows;
  p.tiles = (int)w.tiles;
  p.back = rows * w.nblk < kFarBelow ? kFar : kNear;
  p.marks = packed ? reinterpret_cast<int *>(a.ws + w.marks) : nullptr;
  p.ticket = reinterpret_cast<unsigned int *>(a.ws);
  p.bad = p.ticket + 1;
  p.y = a.y;
  p.h_in = a.states_in ? a.h : nullptr;
  p.h_out = a.no_state_out ? nullptr : a.h;
  p.ck = a.ck;
  p.maps = reinterpret_cast<float4 *>(a.ws + w.maps);
  p.states = reinterpret_cast<float2 *>(a.ws + w.states);
  const bool gated = a.z != nullptr && a.y != nullptr;
  CUtensorMap m[4];
  if (!gs_tensor_map(&m[0], a.io, a.x, rows, a.L, a.D, a.ld_x) ||
      !gs_tensor_map(&m[1], a.io, a.r, rows, a.L, a.D, a.ld_r) ||
      !gs_tensor_map(&m[2], a.io, a.g, rows, a.L, a.D, a.ld_g) ||
      !gs_tensor_map(&m[3], a.io, gated ? a.z : a.x, rows, a.L, a.D, gated ? a.ld_z : a.ld_x))
    return cudaErrorInvalidValue;
  const int64_t nrecords = (int64_t)(w.marks - w.maps) / 16;  // maps and states, side by side
  const int64_t work = std::max(std::max<int64_t>(a.D, nrecords), packed ? a.L : 0);
  gs_prep_kernel<<<(unsigned)std::min<int64_t>(ceil_div(work, 256), 148 * 4), 256, 0, a.stream>>>(
      a.lam, a.c, a.D, const_cast<float *>(p.ncs), reinterpret_cast<uint4 *>(a.ws + w.maps),
      nrecords, p.ticket, a.cu, a.batch, a.L, const_cast<int *>(p.marks),
      const_cast<unsigned int *>(p.bad), p.h_out, a.states_in);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (packed) e = gated ? launch<T, true, true>(a, m, p) : launch<T, true, false>(a, m, p);
  else e = gated ? launch<T, false, true>(a, m, p) : launch<T, false, false>(a, m, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T> cudaError_t step(const GatedScanArgs &a) {
  const int64_t n2 = a.batch * (a.D / 2);
  gs_step_kernel<T><<<(unsigned)ceil_div(n2, 128), 128, 0, a.stream>>>(
      inputs<T>(a), a.lam, a.c, n2, a.D, a.h, static_cast<T *>(a.y));
  return cudaGetLastError();
}

// Offsets must start at 0, not decrease and end at the token count.
__global__ void gs_check_kernel(const int32_t *cu, int64_t batch, int64_t L, unsigned int *bad) {
  int wrong = 0;
  for (int64_t s = threadIdx.x; s < batch; s += blockDim.x) wrong |= cu[s + 1] < cu[s];
  if (threadIdx.x == 0) wrong |= cu[0] != 0 || cu[batch] != L;
  wrong = __syncthreads_or(wrong);
  if (threadIdx.x == 0) {
    *bad = wrong ? 1u : 0u;
    if (wrong) atomicOr(&g_gs_errors, kErrSeqlens);
  }
}

}  // namespace

void gated_scan_check(const int32_t *cu, int64_t batch, int64_t L, unsigned int *bad,
                      cudaStream_t stream) {
  gs_check_kernel<<<1, 1024, 0, stream>>>(cu, batch, L, bad);
}

bool gs_tensor_map(CUtensorMap *m, int io, const void *base, int64_t rows, int64_t L, int D,
                   int64_t ld) {
  using Encode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                              const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                              const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const Encode encode = []() -> Encode {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    return reinterpret_cast<Encode>(p);
  }();
  if (encode == nullptr) return false;
  const bool bf = io == MAMBA2_BF16;
  const uint64_t esz = bf ? 2 : 4;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)L, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(uint64_t)ld * esz, (uint64_t)ld * esz * (uint64_t)L};
  const cuuint32_t box[3] = {(cuuint32_t)kWidth,
                              (cuuint32_t)(bf ? kTile<__nv_bfloat16> : kTile<float>), 1};
  const cuuint32_t one[3] = {1, 1, 1};
  return encode(m, bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3,
                const_cast<void *>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t gated_scan_workspace(int64_t rows, int64_t L, int D, int io, bool packed) {
  return plan_of(rows, L, D, io, packed).total;
}

cudaError_t gated_scan_prefill(const GatedScanArgs &a) {
  return a.io == MAMBA2_BF16 ? prefill<__nv_bfloat16>(a) : prefill<float>(a);
}
cudaError_t gated_scan_step(const GatedScanArgs &a) {
  return a.io == MAMBA2_BF16 ? step<__nv_bfloat16>(a) : step<float>(a);
}

cudaError_t take_gated_scan_errors(unsigned int *out) {
  unsigned int v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_gs_errors, sizeof(v));
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_gs_errors, &zero, sizeof(zero));
  *out = v;
  return e;
}

cudaError_t set_gated_scan_stall(unsigned int v) {
  return cudaMemcpyToSymbol(g_gs_stall, &v, sizeof(v));
}

}  // namespace m2
