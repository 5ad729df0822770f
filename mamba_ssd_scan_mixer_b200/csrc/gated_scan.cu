// Prefill and decode step of the gated linear recurrence (gated_scan.cuh).
//
// Prefill reads every input once.  The tokens of a row are cut into chunks of 128
// and the channels into tiles of one 128-byte row; a tile is one chunk of one tile
// of channels.  Resident blocks take tiles in order, chunk by chunk, from a counter:
//   1. the tile's x, r and g arrive by TMA, two tiles ahead of the arithmetic;
//   2. each thread turns the 16 (fp32: 8) tokens of its two channels into
//      h_t = a_t h_{t-1} + b_t, keeps a and b in registers, and composes them; the
//      segments' maps are composed through shared memory to the tile's (A, H);
//   3. one warp publishes the tile's map and folds those of the chunks before it
//      onto the state that the chunk group before left: the state entering the tile;
//   4. each thread runs its tokens from that state and writes y.
// Every state is put together in an order fixed by the chunks' numbers alone, so that
// results do not depend on timing.  A block waits only for tiles of lower numbers,
// whose blocks are running: the tiles are handed out in order.
#include <algorithm>

#include "gated_scan.cuh"

namespace m2 {

static __device__ unsigned int g_gs_errors = 0;
static __device__ unsigned int g_gs_stall = 0;  // mamba2_debug_stall_waits

namespace {

constexpr int kThreads = 256;
constexpr int kStages = 2;
constexpr int kRowBytes = 128;  // of a tile's token
constexpr int kTensorBytes = kGsChunk * kRowBytes;
constexpr int kStageBytes = 3 * kTensorBytes;
// Chunks whose maps are folded one by one before a state is published again: more
// make a tile read more maps, fewer lengthen the chain of states.
constexpr int kGroup = 16;

// Bits of a token's mark in packed rows: (sequence << 2) | last << 1 | first.
constexpr int kFirst = 1, kLast = 2;

struct Scan {
  const float *ncs;  // [D] -c softplus(lam) log2(e)
  const void *z;
  int64_t ld_z, L;
  int D, nblk, nch, rows, tiles;
  const int *marks;         // packed rows: [L], else null
  const unsigned int *bad;  // packed rows: wrong offsets
  void *y;                  // or null: only the states entering the chunks are wanted
  const float *h_in;        // or null
  float *h_out, *ck;        // or null
  float4 *maps;             // [tiles][kLanes]
  float2 *states;           // [groups][rows][nblk][kLanes]
  unsigned int *flags, *ticket;
};

template <typename T> struct Layout {
  static constexpr int kWidth = kRowBytes / (int)sizeof(T);  // channels
  static constexpr int kLanes = kWidth / 2;                  // threads a token
  static constexpr int kSegs = kThreads / kLanes;
  static constexpr int kTokens = kGsChunk / kSegs;  // of a thread
};

struct Tile {
  int cb, row, chunk, left;
};

template <typename T> struct Shared {
  alignas(128) unsigned char in[kStages][kStageBytes];
  alignas(16) int marks[kStages][kGsChunk];
  float4 seg[Layout<T>::kSegs][Layout<T>::kLanes];
  float2 enter[Layout<T>::kLanes];
  uint64_t full[kStages];
  Tile tile[kStages];
};

// The counters reset, the decays' factor per channel, and for packed rows the
// offsets checked, the tokens marked and the states of empty sequences written.
__global__ void gs_prep_kernel(const float *lam, float c, int D, float *ncs, unsigned int *flags,
                               int tiles, unsigned int *ticket, const int32_t *cu, int64_t batch,
                               int64_t L, int *marks, unsigned int *bad, float *h_out,
                               int states_in) {
  launch_dependents();
  const int64_t at = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t all = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = at; i < D; i += all) ncs[i] = -c * softplus_f(lam[i]) * kLog2e;
  for (int64_t i = at; i < tiles; i += all) flags[i] = 0;
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

template <typename T> __device__ __forceinline__ F2 row_pair(const unsigned char *p);
template <> __device__ __forceinline__ F2 row_pair<float>(const unsigned char *p) {
  const float2 v = *reinterpret_cast<const float2 *>(p);
  return f2(v.x, v.y);
}
template <> __device__ __forceinline__ F2 row_pair<__nv_bfloat16>(const unsigned char *p) {
  const uint32_t w = *reinterpret_cast<const uint32_t *>(p);
  return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// Steps 2: a and b of the thread's tokens, and their composition.
template <typename T, bool FULL, bool PACKED>
__device__ __forceinline__ float4 make_maps(const unsigned char *in, const int *marks, F2 ncs, int n,
                                            const Scan &p, int d, F2 (&a)[Layout<T>::kTokens],
                                            F2 (&b)[Layout<T>::kTokens]) {
  F2 A = f2(1.0f), H = f2(0.0f);
  float4 map = make_float4(1.0f, 1.0f, 0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < Layout<T>::kTokens; ++i) {
    const unsigned char *row = in + i * kRowBytes;
    const F2 x = row_pair<T>(row), R = sigmoid2(row_pair<T>(row + kTensorBytes)),
             G = sigmoid2(row_pair<T>(row + 2 * kTensorBytes));
    F2 v;
    decay2(mul2(ncs, R), &a[i], &v);
    const float2 vv = unpack(v);
    b[i] = mul2(mul2(f2(sqrt_ap(vv.x), sqrt_ap(vv.y)), G), x);
    if (!FULL && i >= n) {
      a[i] = f2(1.0f);
      b[i] = f2(0.0f);
    }
    if (PACKED) {
      if ((FULL || i < n) && (marks[i] & kFirst)) {
        if (p.h_in != nullptr && d < p.D) {
          const float2 h = *reinterpret_cast<const float2 *>(p.h_in + (int64_t)(marks[i] >> 2) * p.D + d);
          b[i] = fma2(a[i], f2(h.x, h.y), b[i]);
        }
        a[i] = f2(-0.0f);
      }
      const float2 ai = unpack(a[i]), bi = unpack(b[i]);
      map = gs_then(map, make_float4(ai.x, ai.y, bi.x, bi.y));
    } else {
      A = mul2(A, a[i]);
      H = fma2(a[i], H, b[i]);
    }
  }
  if (PACKED) return map;
  const float2 x = unpack(A), y = unpack(H);
  return make_float4(x.x, x.y, y.x, y.y);
}

__device__ __forceinline__ void store_pair(float *p, float2 v) {
  *reinterpret_cast<float2 *>(p) = v;
}
__device__ __forceinline__ void store_pair(__nv_bfloat16 *p, float2 v) {
  *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(v.x, v.y);
}

template <typename T, bool PACKED, bool GATED>
__global__ void __launch_bounds__(kThreads, 2)
    gs_prefill_kernel(const __grid_constant__ CUtensorMap map_x,
                      const __grid_constant__ CUtensorMap map_r,
                      const __grid_constant__ CUtensorMap map_g, const Scan p) {
  using Lay = Layout<T>;
  constexpr int kLanes = Lay::kLanes, kTokens = Lay::kTokens;
  extern __shared__ __align__(128) unsigned char raw[];
  Shared<T> &sm = *reinterpret_cast<Shared<T> *>(raw);
  const int tid = threadIdx.x, lane = tid % kLanes, seg = tid / kLanes;
  if (test_stall(&g_gs_stall, &g_gs_errors)) return;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&sm.full[s], 1);
    fence_mbar_init();
  }
  __syncthreads();
  grid_dependency_wait();
  if (PACKED && *p.bad) return;

  // one thread: tile t's copies, into stage s
  auto fetch = [&](int s, int t) {
    Tile q;
    q.left = p.tiles - t;
    q.cb = t % p.nblk;
    q.row = t / p.nblk % p.rows;
    q.chunk = t / p.nblk / p.rows;
    sm.tile[s] = q;
    if (q.left <= 0) {
      mbar_arrive(&sm.full[s]);
      return;
    }
    const int t0 = q.chunk * kGsChunk, n = (int)min((int64_t)kGsChunk, p.L - t0);
    // (whole 16-byte groups of marks; the array is padded)
    const uint32_t mark_bytes = PACKED ? (n * 4 + 15) / 16 * 16 : 0;
    mbar_arrive_expect_tx(&sm.full[s], kStageBytes + mark_bytes);
    unsigned char *in = sm.in[s];
    tma_load_3d(in, &map_x, q.cb * Lay::kWidth, t0, q.row, &sm.full[s]);
    tma_load_3d(in + kTensorBytes, &map_r, q.cb * Lay::kWidth, t0, q.row, &sm.full[s]);
    tma_load_3d(in + 2 * kTensorBytes, &map_g, q.cb * Lay::kWidth, t0, q.row, &sm.full[s]);
    if (PACKED) bulk_g2s(sm.marks[s], p.marks + t0, mark_bytes, &sm.full[s]);
  };
  constexpr int kFetcher = 32;
  if (tid == kFetcher)
    for (int s = 0; s < kStages; ++s) fetch(s, (int)atomicAdd(p.ticket, 1u));

  for (int it = 0;; ++it) {
    const int s = it % kStages;
    const bool arrived = mbar_wait_bounded(&sm.full[s], (it / kStages) & 1, &g_gs_errors);
    // (also: the last tile's segments have been read)
    if (!__syncthreads_and(arrived)) {
      // a wait ran out: what this block has under way lands before it leaves
      if (tid == kFetcher)
        for (int i = it; i < it + kStages; ++i)
          mbar_wait_bounded(&sm.full[i % kStages], (i / kStages) & 1, &g_gs_errors);
      return;
    }
    const Tile q = sm.tile[s];
    if (q.left <= 0) return;  // so is every later tile's: no copy is under way
    int next = 0;
    if (tid == kFetcher) next = (int)atomicAdd(p.ticket, 1u);  // wanted after step 2
    const int t0 = q.chunk * kGsChunk, n = (int)min((int64_t)kGsChunk, p.L - t0);
    const int d = q.cb * Lay::kWidth + 2 * lane, first = seg * kTokens;
    const bool real = d < p.D;
    float2 ncs = make_float2(0.0f, 0.0f);
    if (real) ncs = *reinterpret_cast<const float2 *>(p.ncs + d);
    F2 a[kTokens], b[kTokens];
    const unsigned char *in = sm.in[s] + first * kRowBytes + lane * (2 * (int)sizeof(T));
    const int *marks = sm.marks[s] + first;
    sm.seg[seg][lane] =
        n == kGsChunk
            ? make_maps<T, true, PACKED>(in, marks, f2(ncs.x, ncs.y), n - first, p, d, a, b)
            : make_maps<T, false, PACKED>(in, marks, f2(ncs.x, ncs.y), n - first, p, d, a, b);
    int ends = 0;  // packed rows: which of the thread's tokens end a sequence
    if (PACKED && p.h_out != nullptr) {
#pragma unroll
      for (int i = 0; i < kTokens; ++i)
        if (i < n - first && (marks[i] & kLast)) ends |= 1 << i;
    }
    const int64_t token = (int64_t)q.row * p.L + t0 + first;
    __syncthreads();
    if (tid == kFetcher) fetch(s, next);
    typename Pair<T>::V gate[GATED ? kTokens : 1];  // under way while the states are looked up
    if (GATED) {
      const T *z = static_cast<const T *>(p.z) + token * p.ld_z + d;
#pragma unroll
      for (int i = 0; i < kTokens; ++i) {
        gate[i] = Pair<T>::put(0.0f, 0.0f);
        if (real && i < n - first)
          gate[i] = *reinterpret_cast<const typename Pair<T>::V *>(z + i * p.ld_z);
      }
    }

    const bool last_chunk = q.chunk == p.nch - 1;
    if (tid < 32) {
      float4 map = sm.seg[0][lane];
      for (int k = 1; k < Lay::kSegs; ++k) map = gs_then(map, sm.seg[k][lane]);
      float2 h = make_float2(0.0f, 0.0f);
      if (q.chunk == 0) {
        if (!PACKED && p.h_in != nullptr && real)
          h = *reinterpret_cast<const float2 *>(p.h_in + (int64_t)q.row * p.D + d);
        const float2 e = gs_through(map, h);  // known whole: nothing before it counts
        map = make_float4(-0.0f, -0.0f, e.x, e.y);
      }
      const int per_chunk = p.rows * p.nblk, mine = q.row * p.nblk + q.cb;
      const int tile = q.chunk * per_chunk + mine;
      const int group = q.chunk / kGroup, in_group = q.chunk % kGroup;
      if (!last_chunk && in_group != kGroup - 1) {
        if (tid < kLanes) __stcg(p.maps + (int64_t)tile * kLanes + lane, map);
        __syncwarp();
        if (tid == 0) flag_set(p.flags + tile);
      }
      if (q.chunk > 0) {
        // the chunks of the group before this one, and the last of the group before
        const int from = group > 0 ? group * kGroup - 1 : 0, need = q.chunk - from;
        const unsigned int *flag = p.flags + (int64_t)(from + tid) * per_chunk + mine;
        bool ready = tid >= need || flag_get(flag);
        if (!__all_sync(0xffffffffu, ready)) {
          const unsigned long long since = globaltimer_ns();
          for (;;) {
            ready = ready || flag_get(flag);
            if (__all_sync(0xffffffffu, ready)) break;
            const bool late = globaltimer_ns() - since > kWaitLimitNs;
            if (__any_sync(0xffffffffu, late)) {
              if (tid == 0) atomicOr(&g_gs_errors, kErrWaitTimeout);
              break;
            }
          }
        }
        __syncwarp();
        if (group > 0)
          h = __ldcg(p.states + ((int64_t)(group - 1) * per_chunk + mine) * kLanes + lane);
        for (int k0 = 0; k0 < in_group; k0 += 8) {
          float4 m[8];
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k0 + k < in_group)
              m[k] = __ldcg(p.maps + ((int64_t)(group * kGroup + k0 + k) * per_chunk + mine) * kLanes + lane);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k0 + k < in_group) h = gs_through(m[k], h);
        }
        if (!last_chunk && in_group == kGroup - 1) {
          if (tid < kLanes)
            __stcg(p.states + ((int64_t)group * per_chunk + mine) * kLanes + lane,
                   gs_through(map, h));
          __syncwarp();
          if (tid == 0) flag_set(p.flags + tile);
        }
      }
      if (tid < kLanes) {
        sm.enter[lane] = h;
        if (p.ck != nullptr && real)
          *reinterpret_cast<float2 *>(p.ck + ((int64_t)q.row * p.nch + q.chunk) * p.D + d) = h;
      }
    }
    __syncthreads();
    if (p.y == nullptr) continue;

    float2 h = sm.enter[lane];
    for (int k = 0; k < seg; ++k) h = gs_through(sm.seg[k][lane], h);
    F2 hh = f2(h.x, h.y);
    T *y = static_cast<T *>(p.y) + token * p.D + d;
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      if (PACKED) {
        const float2 ai = unpack(a[i]), bi = unpack(b[i]), hi = unpack(hh);
        const float2 e = gs_through(make_float4(ai.x, ai.y, bi.x, bi.y), hi);
        hh = f2(e.x, e.y);
      } else {
        hh = fma2(a[i], hh, b[i]);
      }
      if (real && i < n - first) {
        F2 o = hh;
        if (GATED) {
          const float2 z = Pair<T>::get(gate[i]);
          o = mul2(hh, mul2(f2(z.x, z.y), sigmoid2(f2(z.x, z.y))));
        }
        store_pair(y + (int64_t)i * p.D, unpack(o));
        if (PACKED && (ends >> i & 1))
          *reinterpret_cast<float2 *>(p.h_out + (int64_t)(p.marks[t0 + first + i] >> 2) * p.D +
                                      d) = unpack(hh);
      }
    }
    if (!PACKED && p.h_out != nullptr && last_chunk && real && first < n && n <= first + kTokens)
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
  int nblk, nch, lanes;
  int64_t tiles, groups;
  size_t ncs, flags, maps, states, marks, total;
};
Plan plan_of(int64_t rows, int64_t L, int D, int io, bool packed) {
  Plan p;
  const int width = gs_tile_width(io);
  p.lanes = width / 2;
  p.nblk = (int)ceil_div(D, width);
  p.nch = (int)ceil_div(L, kGsChunk);
  p.tiles = rows * p.nch * p.nblk;
  p.groups = p.nch / kGroup;
  p.ncs = 256;  // after the counter and the flag of wrong offsets
  p.flags = p.ncs + align_up((size_t)D * 4, 256);
  p.maps = p.flags + align_up((size_t)p.tiles * 4, 256);
  p.states = p.maps + (p.nch > 1 ? align_up((size_t)p.tiles * p.lanes * 16, 256) : 0);
  p.marks = p.states + align_up((size_t)p.groups * rows * p.nblk * p.lanes * 8, 256);
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
cudaError_t launch(const GatedScanArgs &a, const CUtensorMap (&m)[3], const Scan &p) {
  constexpr size_t smem = sizeof(Shared<T>);
  static_assert(2 * (smem + 2048) <= 227 * 1024, "two blocks to an SM");
  static ContextOnce once;
  if (!once.done()) {
    const cudaError_t e = cudaFuncSetAttribute(
        gs_prefill_kernel<T, PACKED, GATED>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    once.set();
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min(p.tiles, 2 * sm_count()), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, gs_prefill_kernel<T, PACKED, GATED>, m[0], m[1], m[2], p);
}

template <typename T> cudaError_t prefill(const GatedScanArgs &a) {
  const int64_t rows = a.rows();
  const bool packed = a.cu != nullptr;
  const Plan w = plan_of(rows, a.L, a.D, a.io, packed);
  Scan p;
  p.ncs = reinterpret_cast<float *>(a.ws + w.ncs);
  p.z = a.z;
  p.ld_z = a.ld_z;
  p.L = a.L;
  p.D = a.D;
  p.nblk = w.nblk;
  p.nch = w.nch;
  p.rows = (int)rows;
  p.tiles = (int)w.tiles;
  p.marks = packed ? reinterpret_cast<int *>(a.ws + w.marks) : nullptr;
  p.ticket = reinterpret_cast<unsigned int *>(a.ws);
  p.bad = p.ticket + 1;
  p.y = a.y;
  p.h_in = a.states_in ? a.h : nullptr;
  p.h_out = a.no_state_out ? nullptr : a.h;
  p.ck = a.ck;
  p.maps = reinterpret_cast<float4 *>(a.ws + w.maps);
  p.states = reinterpret_cast<float2 *>(a.ws + w.states);
  p.flags = reinterpret_cast<unsigned int *>(a.ws + w.flags);
  CUtensorMap m[3];
  if (!gs_tensor_map(&m[0], a.io, a.x, rows, a.L, a.D, a.ld_x) ||
      !gs_tensor_map(&m[1], a.io, a.r, rows, a.L, a.D, a.ld_r) ||
      !gs_tensor_map(&m[2], a.io, a.g, rows, a.L, a.D, a.ld_g))
    return cudaErrorInvalidValue;
  const int64_t work = std::max(std::max<int64_t>(a.D, w.tiles), packed ? a.L : 0);
  gs_prep_kernel<<<(unsigned)std::min<int64_t>(ceil_div(work, 256), 148), 256, 0, a.stream>>>(
      a.lam, a.c, a.D, const_cast<float *>(p.ncs), p.flags, p.tiles, p.ticket, a.cu, a.batch, a.L,
      const_cast<int *>(p.marks), const_cast<unsigned int *>(p.bad), p.h_out, a.states_in);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const bool gated = a.z != nullptr && a.y != nullptr;
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
  const cuuint32_t box[3] = {(cuuint32_t)gs_tile_width(io), (cuuint32_t)kGsChunk, 1};
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
