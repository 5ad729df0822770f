// Prefill and decode step of the gated linear recurrence (gated_scan.cuh).
//
// Prefill reads every input once.  A tile is 128 (fp32: 64) tokens of 32 channels of a
// row; resident blocks take tiles in order, all channels of a stretch of tokens before
// the next stretch, from a counter:
//   1. the tile's x, r and g (and z) arrive by TMA, two tiles ahead of the arithmetic;
//   2. each thread of the four computing warps turns the 16 (8) tokens of its two
//      channels into h_t = a_t h_{t-1} + b_t, keeps a and b in registers, and composes
//      them into the map of its segment, (A, H), in shared memory; the last of the
//      warps publishes the whole tile's map;
//   3. meanwhile a fifth warp looks up the state entering the tile: it folds the maps of
//      the tiles before it onto the state that one further back left.  When the
//      segments are there it fetches the tile after next;
//   4. each thread runs its tokens from that state and writes y; the last of the warps
//      has published the state that the tile leaves.
// Every state is put together in an order fixed by the tiles' numbers alone, so that
// results do not depend on timing.  A block waits only for tiles of lower numbers, whose
// blocks are running: the tiles are handed out in order.
//
// Bytes bound it where many rows or channels are under way (8 rows of 4096 tokens and 5120
// channels, bf16: 240 us, 85% of the copy rate; one row in fp32: 57 us, 89%).  In one bf16
// row the tiles under way reach over four steps of the row, and each waits about a
// microsecond a round for the map of the one before (43 us, 60%).  Next to that come the
// instructions: 71 a pair of channels and token with those of the waits, eight of them ex2,
// rcp or sqrt.
#include "gated_scan_tiles.cuh"

namespace m2 {
namespace {

// Blocks on an SM at once, and tokens of a tile: what registers and shared memory hold.
template <bool GATED> constexpr int kResident = GATED ? 3 : 4;
template <typename T, bool GATED>
using Tiles = Shared<T, GATED ? 4 : 3, sizeof(T) == 2 ? 128 : 64>;

// Step 2: a and b of the thread's tokens, and their composition.
template <typename S, bool FULL, bool NEAR>
__device__ __forceinline__ float4 make_maps(const unsigned char *in, F2 ncs, int n,
                                            F2 (&a)[S::kTokens], F2 (&b)[S::kTokens]) {
  using T = typename S::T;
  F2 A = f2(1.0f), H = f2(0.0f);
#pragma unroll
  for (int i = 0; i < S::kTokens; ++i) {
    const unsigned char *row = in + i * S::kRow;
    const Coeffs c =
        coefficients<NEAR>(gs_pair<T>(row), gs_clamped<T>(row + S::kTensor),
                           gs_clamped<T>(row + 2 * S::kTensor), ncs);
    a[i] = c.a;
    b[i] = c.b;
    if (!FULL && i >= n) {
      a[i] = f2(1.0f);
      b[i] = f2(0.0f);
    }
    A = mul2(A, a[i]);
    H = fma2(a[i], H, b[i]);
  }
  const float2 x = unpack(A), y = unpack(H);
  return make_float4(x.x, x.y, y.x, y.y);
}

// Packed rows: where a sequence begins (a bit of `begins`) its state comes in, and nothing
// from before.  Apart from the arithmetic above, so that this seldom used code is short:
// a second copy of all of it, fetched anew at each sequence, held the whole row up by 2 us.
template <typename S>
__device__ __forceinline__ float4 reset_maps(const int *marks, unsigned int begins, const Scan &p,
                                             int d, F2 (&a)[S::kTokens], F2 (&b)[S::kTokens]) {
  for (unsigned int left = begins; left != 0; left &= left - 1) {
    const int one = __ffs(left) - 1;
    float2 h = make_float2(0.0f, 0.0f);
    if (p.first != nullptr && d < p.D)
      h = *reinterpret_cast<const float2 *>(p.first + (int64_t)(marks[one] >> 2) * p.D + d);
#pragma unroll
    for (int i = 0; i < S::kTokens; ++i)
      if (i == one) {
        b[i] = fma2(a[i], f2(h.x, h.y), b[i]);
        a[i] = f2(-0.0f);
      }
  }
  float4 map = make_float4(1.0f, 1.0f, 0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < S::kTokens; ++i) {
    const float2 x = unpack(a[i]), y = unpack(b[i]);
    map = gs_then(map, make_float4(x.x, x.y, y.x, y.y));
  }
  return map;
}

template <typename T, bool PACKED, bool GATED>
__global__ void __launch_bounds__(kThreads, kResident<GATED>)
    gs_prefill_kernel(const __grid_constant__ Maps maps, const Scan p, T *y_out, float *h_out,
                      float *ck) {
  using S = Tiles<T, GATED>;
  extern __shared__ __align__(128) unsigned char raw[];
  S &sm = *reinterpret_cast<S *>(raw);
  const int warp = threadIdx.x >> 5;
  if (!begin<S, PACKED>(sm, p)) return;
  if (warp == kWarps) {
    look_up<S, PACKED, false>(sm, maps, p);
    return;
  }

  const int lane = threadIdx.x % kLanes, seg = threadIdx.x / kLanes;  // of a half warp
  const int first = seg * S::kTokens;
  for (int it = 0;; ++it) {
    const int s = it % S::kStages, half = it & 1;
    const bool there = mbar_wait_parked(&sm.full[s], (it / S::kStages) & 1, &g_gs_errors);
    if (!there) sm.dead = 1;  // (the error is raised: what comes of the old contents does not matter)
    const Tile q = sm.tile[s];
    if (q.left <= 0) return;
    const int t0 = q.step * S::kTile, n = (int)min((int64_t)S::kTile, p.L - t0);
    const int d = q.cb * kWidth + 2 * lane;
    const bool real = d < p.D;
    const float2 ncs = *reinterpret_cast<const float2 *>(&sm.ncs[s][2 * lane]);
    F2 a[S::kTokens], b[S::kTokens];
    const unsigned char *in = sm.in[s] + first * S::kRow + lane * (2 * (int)sizeof(T));
    const int *marks = sm.marks[s] + first;
    // packed rows: which of the warp's tokens begin and end a sequence
    unsigned int begins = 0, ends = 0;
    bool whole = true;  // (no sequence begins in either half)
    int owner = 0;      // of the first of the ends
    if (PACKED) {
      // (marks that did not come name no sequence)
      const int mark = there && lane < min(S::kTokens, n - first) ? marks[lane] : 0;
      const int up = threadIdx.x & 16;
      begins = __ballot_sync(0xffffffffu, mark & kFirst);
      ends = __ballot_sync(0xffffffffu, h_out != nullptr && (mark & kLast));
      whole = begins == 0;
      begins = begins >> up & 0xffff;
      ends = ends >> up & 0xffff;
      if (ends != 0) owner = marks[__ffs(ends) - 1] >> 2;
    }
    const F2 k = f2(ncs.x, ncs.y);
    float4 map;
    const bool close = __all_sync(0xffffffffu, near(ncs));
    if (close && n == S::kTile) map = make_maps<S, true, true>(in, k, n - first, a, b);
    else if (close) map = make_maps<S, false, true>(in, k, n - first, a, b);
    else map = make_maps<S, false, false>(in, k, n - first, a, b);
    if (PACKED && !whole) map = reset_maps<S>(marks, begins, p, d, a, b);
    sm.seg[half][seg][lane] = map;
    if (PACKED && threadIdx.x % 32 == 0) sm.resets[half][warp] = !whole;
    typename Pair<T>::V gate[GATED ? S::kTokens : 1];
    if (GATED) {
#pragma unroll
      for (int i = 0; i < S::kTokens; ++i)
        gate[i] = *reinterpret_cast<const typename Pair<T>::V *>(in + i * S::kRow + 3 * S::kTensor);
    }
    __syncwarp();
    if (threadIdx.x % 32 == 0) mbar_arrive(&sm.segs[half]);
    const int64_t token = (int64_t)q.row * p.L + t0 + first;
    float2 h;
    if (!exchange<PACKED>(sm, p, q, half, seg, lane, map, &h)) return;
    if (ck != nullptr && real && first % kGsChunk == 0 && first < n)
      *reinterpret_cast<float2 *>(
          ck + ((int64_t)q.row * ((p.L + kGsChunk - 1) / kGsChunk) + (t0 + first) / kGsChunk) * p.D +
          d) = h;
    F2 hh = f2(h.x, h.y);
    if (y_out != nullptr) {
      T *y = y_out + token * p.D + d;
      // all: every token of every lane is stored, and no sequence begins or ends
      auto run = [&](auto all) {
#pragma unroll
        for (int i = 0; i < S::kTokens; ++i) {
          if (PACKED && !decltype(all)::value && (begins >> i & 1)) hh = b[i];
          else hh = fma2(a[i], hh, b[i]);
          F2 o = hh;
          if (GATED) {
            const float2 z = Pair<T>::get(gate[i]);
            o = mul2(hh, mul2(f2(z.x, z.y), sigmoid2(f2(z.x, z.y))));
          }
          if (decltype(all)::value || (real && i < n - first)) {
            st2(y, unpack(o));
            if (PACKED && !decltype(all)::value && (ends >> i & 1)) {
              // (a short sequence's mark is read again: the stage may hold another tile)
              const int who = (ends & ((1u << i) - 1)) == 0 ? owner : p.marks[t0 + first + i] >> 2;
              *reinterpret_cast<float2 *>(h_out + (int64_t)who * p.D + d) = unpack(hh);
            }
          }
          y += p.D;
        }
      };
      if (__all_sync(0xffffffffu, real && n - first >= S::kTokens && (begins | ends) == 0))
        run(std::true_type());
      else
        run(std::false_type());
    }
    if (!PACKED && h_out != nullptr && q.step == p.steps - 1 && real && first < n &&
        n <= first + S::kTokens)
      // (tokens behind the last leave the state as it is)
      *reinterpret_cast<float2 *>(h_out + (int64_t)q.row * p.D + d) = unpack(hh);
  }
}

template <typename T> struct In {
  const T *x, *r, *g, *z;
  int64_t ld_x, ld_r, ld_g, ld_z;
};

// ---------------------------------------------------------------- short rows
// A thread runs the tokens of a row for two channels, four tokens' loads at a time: tiles
// would be mostly empty, and nothing has to be prepared.
constexpr int kShortBatch = 4;
template <typename T, bool GATED>
__global__ void __launch_bounds__(128, 5)
    gs_short_kernel(In<T> in, const float *lam, float c, int64_t pairs, int L, int D,
                    const float *h_in, float *h_out, float *ck, T *y) {
  grid_dependency_wait();
  using V = typename Pair<T>::V;
  const int64_t at = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (at >= pairs) return;
  const int64_t row = at / (D / 2), nch = (L + kGsChunk - 1) / kGsChunk;
  const int d = 2 * (int)(at % (D / 2));
  const T *x = in.x + row * L * in.ld_x + d, *r = in.r + row * L * in.ld_r + d,
          *g = in.g + row * L * in.ld_g + d, *z = in.z + (GATED ? row * L * in.ld_z + d : 0);
  T *out = y + row * L * D + d;
  F2 h = f2(0.0f);
  if (h_in != nullptr) {
    const float2 v = *reinterpret_cast<const float2 *>(h_in + row * D + d);
    h = f2(v.x, v.y);
  }
  const F2 ncs = f2(-c * softplus_f(lam[d]) * kLog2e, -c * softplus_f(lam[d + 1]) * kLog2e);
  auto run = [&](auto near) {
#pragma unroll 1
    for (int t0 = 0; t0 < L; t0 += kShortBatch) {
      const int n = min(kShortBatch, L - t0);
      V bx[kShortBatch], br[kShortBatch], bg[kShortBatch], bz[kShortBatch];
#pragma unroll
      for (int i = 0; i < kShortBatch; ++i)
        if (i < n) {
          bx[i] = *reinterpret_cast<const V *>(x + i * in.ld_x);
          br[i] = *reinterpret_cast<const V *>(r + i * in.ld_r);
          bg[i] = *reinterpret_cast<const V *>(g + i * in.ld_g);
          if (GATED) bz[i] = *reinterpret_cast<const V *>(z + i * in.ld_z);
        }
      if (ck != nullptr && t0 % kGsChunk == 0)
        *reinterpret_cast<float2 *>(ck + (row * nch + t0 / kGsChunk) * D + d) = unpack(h);
#pragma unroll
      for (int i = 0; i < kShortBatch; ++i)
        if (i < n) {
          const Coeffs k = coefficients<decltype(near)::value>(gs_pair<T>(&bx[i]), gs_clamped<T>(&br[i]),
                                               gs_clamped<T>(&bg[i]), ncs);
          h = fma2(k.a, h, k.b);
          if (y != nullptr) {
            F2 o = h;
            if (GATED) {
              const F2 zz = gs_pair<T>(&bz[i]);
              o = mul2(h, mul2(zz, sigmoid2(zz)));
            }
            st2(out + (int64_t)i * D, unpack(o));
          }
        }
      x += kShortBatch * in.ld_x;
      r += kShortBatch * in.ld_r;
      g += kShortBatch * in.ld_g;
      if (GATED) z += kShortBatch * in.ld_z;
      out += (int64_t)kShortBatch * D;
    }
  };
  if (__all_sync(__activemask(), near(unpack(ncs)))) run(std::true_type());
  else run(std::false_type());
  if (h_out != nullptr) *reinterpret_cast<float2 *>(h_out + row * D + d) = unpack(h);
}

// ---------------------------------------------------------------- decode

// 16 bytes of a row: V = 4 or 8 channels.
template <typename T> struct Lane {
  static constexpr int V = 16 / (int)sizeof(T);
  uint4 w;
  __device__ __forceinline__ void load(const T *p) { w = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ const void *pair(int k) const {
    return reinterpret_cast<const T *>(&w) + 2 * k;
  }
};

// One token of every sequence.  Bound by the state's and the rows' bytes (and, for few
// sequences, by the launch): a thread takes 16 bytes of each row, two rows one after the
// other; the decays' factors are made once for a block's rows.
constexpr int kStepGroups = 64, kStepRows = 4, kStepTurns = 2;
template <typename T, bool GATED>
__global__ void __launch_bounds__(kStepGroups *kStepRows)
    gs_step_kernel(In<T> in, const float *lam, float c, int64_t batch, int D,
                   float *h, T *y) {
  grid_dependency_wait();
  constexpr int V = Lane<T>::V;
  __shared__ float ncs[kStepGroups * V];
  const int group = threadIdx.x % kStepGroups, c0 = blockIdx.x * kStepGroups * V;
  const int d = c0 + group * V;
  const int64_t row = (int64_t)blockIdx.y * (kStepRows * kStepTurns) + threadIdx.x / kStepGroups;
  Lane<T> x[kStepTurns], r[kStepTurns], g[kStepTurns], z[kStepTurns];
  float4 s[kStepTurns][V / 4];
#pragma unroll
  for (int k = 0; k < kStepTurns; ++k) {
    const int64_t b = row + k * kStepRows;
    if (b < batch && d < D) {
      x[k].load(in.x + b * in.ld_x + d);
      r[k].load(in.r + b * in.ld_r + d);
      g[k].load(in.g + b * in.ld_g + d);
      if (GATED) z[k].load(in.z + b * in.ld_z + d);
#pragma unroll
      for (int j = 0; j < V / 4; ++j) s[k][j] = *reinterpret_cast<const float4 *>(h + b * D + d + 4 * j);
    }
  }
  for (int i = threadIdx.x; i < kStepGroups * V; i += kStepGroups * kStepRows)
    ncs[i] = c0 + i < D ? -c * softplus_f(lam[c0 + i]) * kLog2e : 0.0f;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kStepTurns; ++k) {
    const int64_t b = row + k * kStepRows;
    if (b >= batch || d >= D) continue;
    float *state = reinterpret_cast<float *>(s[k]);
    uint4 out;
#pragma unroll
    for (int j = 0; j < V / 2; ++j) {
      const float2 n = *reinterpret_cast<const float2 *>(&ncs[group * V + 2 * j]);
      const Coeffs q = coefficients<false>(gs_pair<T>(x[k].pair(j)), gs_clamped<T>(r[k].pair(j)),
                                           gs_clamped<T>(g[k].pair(j)), f2(n.x, n.y));
      F2 v = fma2(q.a, f2(state[2 * j], state[2 * j + 1]), q.b);
      const float2 w = unpack(v);
      state[2 * j] = w.x;
      state[2 * j + 1] = w.y;
      if (GATED) {
        const F2 zz = gs_pair<T>(z[k].pair(j));
        v = mul2(v, mul2(zz, sigmoid2(zz)));
      }
      st2(reinterpret_cast<T *>(&out) + 2 * j, unpack(v));
    }
    *reinterpret_cast<uint4 *>(y + b * D + d) = out;
#pragma unroll
    for (int j = 0; j < V / 4; ++j) *reinterpret_cast<float4 *>(h + b * D + d + 4 * j) = s[k][j];
  }
}

template <typename T> In<T> inputs(const GatedScanArgs &a) {
  return In<T>{static_cast<const T *>(a.x), static_cast<const T *>(a.r),
               static_cast<const T *>(a.g), static_cast<const T *>(a.z),
               a.ld_x,                      a.ld_r,
               a.ld_g,                      a.ld_z};
}

template <typename T, bool PACKED, bool GATED>
cudaError_t launch(const GatedScanArgs &a, const Maps &m, const Scan &p) {
  constexpr size_t smem = sizeof(Tiles<T, GATED>);
  static_assert(kResident<GATED> * (smem + 1024 + 256) <= 228 * 1024, "blocks to an SM");
  static ContextOnce once;
  return launch_dependent(gs_prefill_kernel<T, PACKED, GATED>, once,
                          std::min(p.tiles, kResident<GATED> * sm_count()), kThreads, smem,
                          a.stream, m, p, static_cast<T *>(a.y), a.no_state_out ? nullptr : a.h,
                          a.ck);
}

// Rows for gs_short_kernel.  It wins where tiles of 128 tokens are mostly empty: up to 16
// tokens always (one row of 16 tokens and 5120 channels 4.9 us against 7.0, 64 rows 15
// against 67), up to 64 where there are threads for the whole GPU (64 rows of 64 tokens 51
// against 67 us); one row of 64 tokens is slower by it (13.7 against 6.9 us), and 64 rows
// of 128 tokens too (96 against 64 us).
constexpr int64_t kShort = 16, kShortOfMany = 64, kMany = 65536;

template <typename T> cudaError_t prefill(const GatedScanArgs &a) {
  const int64_t rows = a.rows();
  const int64_t pairs = rows * (a.D / 2);
  if (a.cu == nullptr && (a.L <= kShort || (a.L <= kShortOfMany && pairs >= kMany))) {
    const auto kernel = a.z != nullptr && a.y != nullptr ? gs_short_kernel<T, true>
                                                         : gs_short_kernel<T, false>;
    return launch_dependent(kernel, (unsigned)ceil_div(pairs, 128), 128, 0, a.stream, inputs<T>(a), a.lam,
                            a.c, pairs, (int)a.L, a.D, a.states_in ? a.h : (float *)nullptr,
                            a.no_state_out ? (float *)nullptr : a.h, a.ck, static_cast<T *>(a.y));
  }
  const bool packed = a.cu != nullptr, gated = a.z != nullptr && a.y != nullptr;
  const Plan w = plan_of(rows, a.L, a.D, Tiles<T, false>::kTile, packed);
  Maps m = {};
  const void *in[4] = {a.x, a.r, a.g, a.z};
  const int64_t ld[4] = {a.ld_x, a.ld_r, a.ld_g, a.ld_z};
  for (int k = 0; k < (gated ? 4 : 3); ++k)
    if (!gs_tensor_map(&m.m[k], a.io, in[k], rows, a.L, a.D, ld[k], kWidth,
                       Tiles<T, false>::kTile))
      return cudaErrorInvalidValue;
  Scan p;
  // (a sequence without tokens keeps its state, or starts and ends at zero)
  cudaError_t e = prepare(a, w, a.ws, a.states_in ? a.h : nullptr, nullptr,
                          a.states_in || a.no_state_out ? nullptr : a.h, &p);
  if (e != cudaSuccess) return e;
  if (packed) e = gated ? launch<T, true, true>(a, m, p) : launch<T, true, false>(a, m, p);
  else e = gated ? launch<T, false, true>(a, m, p) : launch<T, false, false>(a, m, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T> cudaError_t step(const GatedScanArgs &a) {
  const dim3 grid((unsigned)ceil_div(a.D, kStepGroups * Lane<T>::V),
                  (unsigned)ceil_div(a.batch, kStepRows * kStepTurns));
  const auto kernel = a.z != nullptr ? gs_step_kernel<T, true> : gs_step_kernel<T, false>;
  return launch_dependent(kernel, grid, kStepGroups * kStepRows, 0, a.stream, inputs<T>(a), a.lam,
                          a.c, a.batch, a.D, a.h, static_cast<T *>(a.y));
}

}  // namespace

bool gs_tensor_map(CUtensorMap *m, int io, const void *base, int64_t rows, int64_t L, int D,
                   int64_t ld, int width, int tokens) {
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
  const cuuint32_t box[3] = {(cuuint32_t)width, (cuuint32_t)tokens, 1};
  const cuuint32_t one[3] = {1, 1, 1};
  return encode(m, bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3,
                const_cast<void *>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t gated_scan_workspace(int64_t rows, int64_t L, int D, int io, bool packed) {
  return plan_of(rows, L, D,
                 io == MAMBA2_BF16 ? Tiles<__nv_bfloat16, false>::kTile : Tiles<float, false>::kTile,
                 packed)
      .total;
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
