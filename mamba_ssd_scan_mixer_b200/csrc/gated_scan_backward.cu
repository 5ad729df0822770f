// Backward pass of the gated linear recurrence (gated_scan.cuh).
//
// With d_t the gradient of h_t (of a sequence's last: plus the final state's), and
// v = 1 - a^2,
//     d_t  = dy_t silu(z_t) + a_{t+1} d_{t+1}
//     dx   = d m G               dg = dx x (1 - G)           dz = dy h silu'(z)
//     dla  = d a (h_{t-1} - a b / v)                         (b = m G x; a^2 / m G x = a^2 b / v)
//     dr   = dla la (1 - R)      dlam = sum dla (-c R) sigmoid(lam)
// with 1 - R = e^-r R and 1 - G = e^-g G.
//
// What a token hands to the one before it, E_t = a_t d_t = a_t E_{t+1} + a_t dy_t silu(z_t),
// is the prefill's recurrence run from the last token to the first.  So:
//   1. gs_back_carry_kernel, built like the prefill's, runs it over r, dy and z, and
//      writes E only where 16 tokens end;
//   2. gs_back_apply_kernel then has, for each 16 tokens, the state that enters them (the
//      prefill's checkpoints) and the E that does: its warps depend on nobody.  Each runs
//      its 16 tokens forwards, keeping h, e^-r and e^-g, and backwards.
// The first pass costs 4 bytes an element beside the second's 14 (bf16).  (The second
// begins where the first ended, and finds 29 of 84 MB of r and dy in L2 at 4096 tokens of
// 5120 channels.)  Two passes, since the second then waits for nothing and the first, which
// waits, holds little.  (One pass whose sweep forwards runs while E is on its way would read
// r and dy once; it has not been built.)
//
// 4096 tokens of 5120 channels, bf16: the first 27 us (13 at the copy rate), the second
// 67 us (46).  The first waits for the maps of the tiles before, as the prefill does.  The
// second issues 119 instructions a pair of channels and token, 14 of them ex2, rcp or sqrt,
// at half of the issue rate with the 12 warps that its registers leave.  (With z, 8 warps: two
// stages leave room for two blocks.)
#include "gated_scan_tiles.cuh"

namespace m2 {
namespace {

static_assert(kGsChunk == 16, "tokens of a thread, between checkpoints");

// ---------------------------------------------------------------- E at the chunks' ends
// Nothing of a token is kept, so that a thread may take two chunks of 16: fewer, larger
// tiles to look up (27 against 30 us at 4096 tokens of 5120 channels).  With z a stage of
// such tiles would leave two blocks to an SM in place of four: there one chunk (78 against
// 86 us at 8 rows of 2048 tokens and 4096 channels).
template <typename T, bool GATED>
constexpr int kCarryTile = sizeof(T) == 2 && !GATED ? 256 : 128;
template <typename T, bool GATED>
using CarryTiles = Shared<T, GATED ? 3 : 2, kCarryTile<T, GATED>>;
template <typename T, bool GATED>
constexpr int kCarryResident = GATED ? (sizeof(T) == 2 ? 4 : 2) : 3;

__device__ __forceinline__ F2 silu2(F2 z) { return mul2(z, sigmoid2(z)); }

// The map of 16 tokens, last to first.  `lasts`: the tokens that end a sequence.
template <typename S, bool FULL, bool RESETS, bool NEAR, bool GATED>
__device__ __forceinline__ float4 back_map(const unsigned char *in, const int *marks,
                                           unsigned int lasts, F2 ncs, int n, const float *dh,
                                           int D, int d) {
  using T = typename S::T;
  F2 A = f2(1.0f), E = f2(0.0f);
  // the final gradient of the last sequence that ends here: under way early
  auto gradient_of = [&](int i) {
    float2 v = make_float2(0.0f, 0.0f);
    if (dh != nullptr && d < D)
      v = *reinterpret_cast<const float2 *>(dh + (int64_t)(marks[i] >> 2) * D + d);
    return f2(v.x, v.y);
  };
  const int one = RESETS ? 31 - __clz(lasts) : -1;
  F2 gradient = f2(0.0f);
  if (RESETS && one >= 0) gradient = gradient_of(one);
#pragma unroll
  for (int i = kGsChunk - 1; i >= 0; --i) {
    if (!FULL && i >= n) continue;
    const unsigned char *row = in + i * S::kRow;
    F2 a, less, dy = gs_pair<T>(row + S::kTensor);
    decay2<NEAR>(mul2(ncs, sigmoid2(gs_pair<T>(row))), &a, &less);
    if (GATED) dy = mul2(dy, silu2(gs_pair<T>(row + 2 * S::kTensor)));
    if (RESETS && (lasts >> i & 1)) {
      dy = add2(dy, i == one ? gradient : gradient_of(i));
      A = f2(-0.0f);
      E = mul2(a, dy);
    } else {
      A = mul2(A, a);
      E = mul2(a, add2(E, dy));
    }
  }
  const float2 x = unpack(A), y = unpack(E);
  return make_float4(x.x, x.y, y.x, y.y);
}

template <typename T, bool PACKED, bool GATED>
__global__ void __launch_bounds__(kThreads, (kCarryResident<T, GATED>))
    gs_back_carry_kernel(const __grid_constant__ Maps maps, const Scan p, const float *dh,
                         float *carry) {
  using S = CarryTiles<T, GATED>;
  extern __shared__ __align__(128) unsigned char raw[];
  S &sm = *reinterpret_cast<S *>(raw);
  if (!begin<S, PACKED>(sm, p)) return;
  launch_dependents();
  if (threadIdx.x >= 32 * kWarps) {
    look_up<S, PACKED, true>(sm, maps, p);
    return;
  }
  const int lane = threadIdx.x % kLanes, seg = threadIdx.x / kLanes;  // of a half warp
  const int first = (kSegs - 1 - seg) * S::kTokens;
  const int64_t nch = (p.L + kGsChunk - 1) / kGsChunk;
  for (int it = 0;; ++it) {
    const int s = it % S::kStages, half = it & 1;
    const bool there = mbar_wait_parked(&sm.full[s], (it / S::kStages) & 1, &g_gs_errors);
    if (!there) sm.dead = 1;  // (the error is raised: what comes of the old contents does not matter)
    const Tile q = sm.tile[s];
    if (q.left <= 0) return;
    const int t0 = (p.steps - 1 - q.step) * S::kTile, n = (int)min((int64_t)S::kTile, p.L - t0);
    const int d = q.cb * kWidth + 2 * lane;
    const float2 ncs = *reinterpret_cast<const float2 *>(&sm.ncs[s][2 * lane]);
    const F2 k = f2(ncs.x, ncs.y);
    constexpr int kChunks = S::kTokens / kGsChunk;  // of a thread
    float4 maps_of[kChunks], map;
    bool resets = false;
    const bool close = __all_sync(0xffffffffu, near(ncs));
#pragma unroll
    for (int c = kChunks - 1; c >= 0; --c) {
      const int at = first + c * kGsChunk;
      const unsigned char *in = sm.in[s] + at * S::kRow + lane * (2 * (int)sizeof(T));
      const int *marks = sm.marks[s] + at;
      unsigned int lasts = 0;
      if (PACKED)
        // (marks that did not come name no sequence)
        lasts = __ballot_sync(0xffffffffu,
                              there && lane < min(kGsChunk, n - at) && (marks[lane] & kLast));
      const bool whole = lasts == 0;  // (no sequence ends in either half)
      resets |= !whole;
      lasts = lasts >> (threadIdx.x & 16) & 0xffff;
      if (close && whole && n == S::kTile)
        maps_of[c] = back_map<S, true, false, true, GATED>(in, marks, 0, k, n - at, dh, p.D, d);
      else if (close)
        maps_of[c] = back_map<S, false, PACKED, true, GATED>(in, marks, lasts, k, n - at, dh, p.D, d);
      else
        maps_of[c] = back_map<S, false, PACKED, false, GATED>(in, marks, lasts, k, n - at, dh, p.D, d);
      map = c == kChunks - 1 ? maps_of[c] : gs_then(map, maps_of[c]);
    }
    sm.seg[half][seg][lane] = map;
    if (PACKED && threadIdx.x % 32 == 0) sm.resets[half][threadIdx.x / 32] = resets;
    __syncwarp();
    if (threadIdx.x % 32 == 0) mbar_arrive(&sm.segs[half]);
    float2 e;
    if (!exchange<PACKED>(sm, p, q, half, seg, lane, map, &e)) return;
#pragma unroll
    for (int c = kChunks - 1; c >= 0; --c) {
      const int at = first + c * kGsChunk;
      if (d < p.D && at < n)
        *reinterpret_cast<float2 *>(carry + ((int64_t)q.row * nch + (t0 + at) / kGsChunk) * p.D +
                                    d) = e;
      e = gs_through(maps_of[c], e);
    }
  }
}

// ---------------------------------------------------------------- the gradients
constexpr int kApplyTile = 64, kApplyWidth = 64;  // whole 128-byte lines of bf16

template <typename T, bool GATED> struct ApplyShared {
  static constexpr int kTensors = GATED ? 5 : 4;
  // one stage where two would leave too few blocks to an SM
  static constexpr int kStages = sizeof(T) == 2 ? 2 : 1;
  static constexpr int kRow = kApplyWidth * (int)sizeof(T), kTensor = kApplyTile * kRow;
  alignas(128) unsigned char in[kStages][kTensors * kTensor];
  alignas(16) float h[kStages][kWarps][kApplyWidth];  // the states entering the warps' tokens
  alignas(16) float e[kStages][kWarps][kApplyWidth];  // and the E
  alignas(16) int marks[kStages][kApplyTile];
  alignas(16) float ncs[kStages][kApplyWidth];
  float2 dl[2][kWarps][32];
  uint64_t full[kStages];
  int dead;  // a wait ran out: everybody leaves after the tile
};
// Three blocks of four warps: 168 registers a thread.
constexpr int kApplyThreads = 32 * kWarps;
template <typename T, bool GATED>
constexpr int kApplyResident = GATED ? 2 : 3;

// The tiles of a block, `stride` apart, without a division each.
struct Walk {
  int cb, row, step, dcb, drow, dstep;
  __device__ __forceinline__ Walk(int tile, int stride, const Scan &p)
      : cb(tile % p.nblk), row(tile / p.nblk % p.rows), step(tile / p.nblk / p.rows),
        dcb(stride % p.nblk), drow(stride / p.nblk % p.rows), dstep(stride / p.nblk / p.rows) {}
  __device__ __forceinline__ void next(const Scan &p) {
    cb += dcb;
    row += drow;
    step += dstep;
    if (cb >= p.nblk) {
      cb -= p.nblk;
      ++row;
    }
    if (row >= p.rows) {
      row -= p.rows;
      ++step;
    }
  }
};

template <typename T> struct Apply {
  Scan p;  // (steps, nblk and tiles: of kApplyTile tokens and kApplyWidth channels)
  const float *ck, *carry;  // [rows][chunks][D]
  const float *h_in, *dh;   // packed rows: the sequences' initial states and final gradients
  T *dx, *dr, *dg, *dz;
  float *dh_in, *dl;  // dl: [rows * steps][nblk * 64]
  unsigned long long zero;
};

// A state kept where a token's r and g were (each thread's own words).
template <typename T> __device__ __forceinline__ void put_state(unsigned char *r, unsigned char *g, F2 h);
template <> __device__ __forceinline__ void put_state<__nv_bfloat16>(unsigned char *r, unsigned char *g, F2 h) {
  const float2 v = unpack(h);
  *reinterpret_cast<float *>(r) = v.x;
  *reinterpret_cast<float *>(g) = v.y;
}
template <> __device__ __forceinline__ void put_state<float>(unsigned char *r, unsigned char *, F2 h) {
  *reinterpret_cast<float2 *>(r) = unpack(h);
}
template <typename T> __device__ __forceinline__ F2 get_state(const unsigned char *r, const unsigned char *g);
template <> __device__ __forceinline__ F2 get_state<__nv_bfloat16>(const unsigned char *r, const unsigned char *g) {
  return f2(*reinterpret_cast<const float *>(r), *reinterpret_cast<const float *>(g));
}
template <> __device__ __forceinline__ F2 get_state<float>(const unsigned char *r, const unsigned char *) {
  const float2 v = *reinterpret_cast<const float2 *>(r);
  return f2(v.x, v.y);
}

// One warp's 16 tokens.  FAST: all of them and of the channels there, no sequence begins or
// ends among them, and decays near one.
template <typename T, bool GATED, bool PACKED, bool FAST>
__device__ __forceinline__ F2 apply_tokens(ApplyShared<T, GATED> &sm, int s,
                                           const Apply<T> &q, int row, int64_t t0, int n, int first,
                                           int lane, int d) {
  using S = ApplyShared<T, GATED>;
  constexpr int K = kGsChunk, kTensor = S::kTensor;
  const Scan &p = q.p;
  const int warp = first / K;
  unsigned char *in = sm.in[s] + first * S::kRow + lane * (2 * (int)sizeof(T));
  const int *marks = sm.marks[s] + first;
  const float2 nn = *reinterpret_cast<const float2 *>(&sm.ncs[s][2 * lane]);
  const F2 ncs = f2(nn.x, nn.y);
  const float2 h0 = *reinterpret_cast<const float2 *>(&sm.h[s][warp][2 * lane]);
  const float2 e0 = *reinterpret_cast<const float2 *>(&sm.e[s][warp][2 * lane]);
  F2 h = f2(h0.x, h0.y), e = f2(e0.x, e0.y), dl = f2(0.0f);
  const bool real = FAST || d < p.D;
  const int count = FAST ? K : min(K, n - first);
  F2 er[K], eg[K];
#pragma unroll
  for (int i = 0; i < K; ++i) {
    er[i] = eg[i] = f2(1.0f);
    if (!FAST && i >= count) continue;
    if (!FAST && PACKED && (marks[i] & kFirst)) {
      h = f2(0.0f);
      if (q.h_in != nullptr && real) {
        const float2 v = *reinterpret_cast<const float2 *>(q.h_in + (int64_t)(marks[i] >> 2) * p.D + d);
        h = f2(v.x, v.y);
      }
    }
    unsigned char *at = in + i * S::kRow;
    const Coeffs c = coefficients<FAST>(gs_pair<T>(at), gs_clamped<T>(at + kTensor),
                                        gs_clamped<T>(at + 2 * kTensor), ncs);
    er[i] = c.er;
    eg[i] = c.eg;
    put_state<T>(at + kTensor, at + 2 * kTensor, h);
    h = fma2(c.a, h, c.b);
  }
  // e^-r and e^-g are kept in registers and h where r and g were: the rest is cheaper made
  // again than held.  (The compiler would hold it, in local memory; it does not know that
  // `zero` is zero.)  e^-r and not R: 1 - R = e^-r R is then as exact as R, where a difference
  // has no digit left from r = 17 on, nor its sign.  It costs a reciprocal more: training at
  // 4096 tokens of 5120 channels takes 137 us against 134, 8 rows of 2048 tokens and 4096
  // channels with z 452 against 431 (replayed from a graph).
  constexpr float kDown = 1.0f / kGateScale;
  const F2 ncs2 = F2{ncs.v ^ q.zero}, one = F2{f2(1.0f).v ^ q.zero}, down = F2{f2(kDown).v ^ q.zero};
  in += q.zero;
  const int64_t behind = ((int64_t)row * p.L + t0 + first + K) * p.D + d;
  T *dx_out = q.dx + behind, *dr_out = q.dr + behind, *dg_out = q.dg + behind,
    *dz_out = GATED ? q.dz + behind : nullptr;
  const int64_t stride = p.D;
  // (the gates of four tokens at once: one after the other the reciprocals are waited for, 464
  // against 452 us at 8 rows of 2048 tokens and 4096 channels with z)
  constexpr int kAtOnce = 4;
  Gates ks[kAtOnce];
#pragma unroll
  for (int i = K - 1; i >= 0; --i) {
    if (i % kAtOnce == kAtOnce - 1) {
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) ks[kAtOnce - 1 - j] = gates(er[i - j], eg[i - j], one, down);
    }
    dx_out -= stride;
    dr_out -= stride;
    dg_out -= stride;
    if (GATED) dz_out -= stride;
    if (!FAST && i >= count) continue;
    const unsigned char *at = in + i * S::kRow;
    const F2 x = gs_pair<T>(at);
    F2 dy = gs_pair<T>(at + 3 * kTensor), a, less;
    const Gates k = ks[i % kAtOnce];
    const F2 t = mul2(ncs2, k.R);
    decay2<FAST>(t, &a, &less);
    constexpr float down2 = kDown * kDown, up2 = kGateScale * kGateScale;
    // v = 1 - a^2, and enough to have a reciprocal: where it is next to nothing m, and b with
    // it, is taken for zero, and so is b / v
    const F2 vv = fma2(less, fma2(a, f2(-1.0f), f2(-1.0f)), f2(1e-30f));
    const float2 v = unpack(vv), w = unpack(mul2(vv, f2(down2)));
    const F2 before = get_state<T>(at + kTensor, at + 2 * kTensor);
    const F2 mG = mul2(f2(sqrt_ap(w.x), sqrt_ap(w.y)), k.G);
    const F2 b = mul2(mG, x);
    if (GATED) {
      const F2 z = gs_pair<T>(at + 4 * kTensor), sig = sigmoid2(z);
      const F2 ht = fma2(a, before, b);
      // silu' = sig (1 + z (1 - sig))
      const F2 slope = mul2(sig, fma2(z, fma2(sig, f2(-1.0f), f2(1.0f)), f2(1.0f)));
      if (real) st2(dz_out, unpack(mul2(mul2(dy, ht), slope)));
      dy = mul2(dy, mul2(z, sig));
    }
    if (!FAST && PACKED && (marks[i] & kLast)) {
      e = f2(0.0f);
      if (q.dh != nullptr && real) {
        const float2 g = *reinterpret_cast<const float2 *>(q.dh + (int64_t)(marks[i] >> 2) * p.D + d);
        e = f2(g.x, g.y);
      }
    }
    const F2 dd = add2(dy, e);
    const F2 dx = mul2(dd, mG);
    const F2 dg = mul2(mul2(dx, x), mul2(eg[i], mul2(k.G, down)));  // (1 - G = e^-g G)
    const F2 iv = f2(rcp(-v.x), rcp(-v.y));  // -1 / v
    e = mul2(a, dd);
    const F2 dla = mul2(e, fma2(mul2(a, b), iv, before));
    const F2 dlaR = mul2(dla, k.R);
    dl = add2(dl, dlaR);
    // dr = dla la (1 - R), with 1 - R = e^-r R.  (|la| < 2^-56 is flushed on the way: a gate so
    // shut, r = -inf, gets no gradient.)
    const F2 la = mul2(mul2_flush(t, f2(0.6931471805599453f * down2)), f2(up2));
    const F2 dr = mul2(dlaR, mul2(la, er[i]));
    if (real) {
      st2(dx_out, unpack(dx));
      st2(dr_out, unpack(dr));
      st2(dg_out, unpack(dg));
    }
    if (!FAST && PACKED && (marks[i] & kFirst) && q.dh_in != nullptr && real)
      *reinterpret_cast<float2 *>(q.dh_in + (int64_t)(marks[i] >> 2) * p.D + d) = unpack(e);
  }
  if (!PACKED && t0 + first == 0 && q.dh_in != nullptr && real)
    *reinterpret_cast<float2 *>(q.dh_in + (int64_t)row * p.D + d) = unpack(e);
  return dl;
}

template <typename T, bool PACKED, bool GATED>
__global__ void __launch_bounds__(kApplyThreads, (kApplyResident<T, GATED>))
    gs_back_apply_kernel(const __grid_constant__ Maps maps, const Apply<T> q) {
  using S = ApplyShared<T, GATED>;
  extern __shared__ __align__(128) unsigned char raw[];
  S &sm = *reinterpret_cast<S *>(raw);
  const Scan &p = q.p;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool stalled = test_stall(&g_gs_stall, &g_gs_errors);
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) mbar_init(&sm.full[s], 1);
    sm.dead = 0;
    fence_mbar_init();
  }
  __syncthreads();
  // (every block waits, so that what waits for this kernel has waited for the one before)
  grid_dependency_wait();
  launch_dependents();
  if (stalled || (PACKED && *p.bad)) return;
  const int64_t nch = (p.L + kGsChunk - 1) / kGsChunk;
  // one thread: a tile's copies, into stage s
  auto fetch = [&](int s, const Walk &w) {
    if (w.step >= p.steps) return;
    const int cb = w.cb, row = w.row, t0 = w.step * kApplyTile;
    const int n = (int)min((int64_t)kApplyTile, p.L - t0), chunks = (n + kGsChunk - 1) / kGsChunk;
    const uint32_t wide = (uint32_t)min(kApplyWidth, p.D - cb * kApplyWidth) * 4;
    const uint32_t mark_bytes = PACKED ? (n * 4 + 15) / 16 * 16 : 0;
    mbar_arrive_expect_tx(&sm.full[s], S::kTensors * S::kTensor + 2 * chunks * wide + kApplyWidth * 4 +
                                           mark_bytes);
#pragma unroll
    for (int k = 0; k < S::kTensors; ++k)
      tma_load_3d(sm.in[s] + k * S::kTensor, &maps.m[k], cb * kApplyWidth, t0, row, &sm.full[s]);
    const int64_t at = ((int64_t)row * nch + t0 / kGsChunk) * p.D + cb * kApplyWidth;
    for (int k = 0; k < chunks; ++k) {
      bulk_g2s(sm.h[s][k], q.ck + at + (int64_t)k * p.D, wide, &sm.full[s]);
      bulk_g2s(sm.e[s][k], q.carry + at + (int64_t)k * p.D, wide, &sm.full[s]);
    }
    bulk_g2s(sm.ncs[s], p.ncs + cb * kApplyWidth, kApplyWidth * 4, &sm.full[s]);
    if (PACKED) bulk_g2s(sm.marks[s], p.marks + t0, mark_bytes, &sm.full[s]);
  };
  constexpr int kFetcher = 32 * kWarps - 1;
  Walk at(blockIdx.x, gridDim.x, p), ahead = at;
  if (threadIdx.x == kFetcher)
    for (int s = 0; s < S::kStages; ++s, ahead.next(p)) fetch(s, ahead);
  const int first = warp * kGsChunk;
  for (int it = 0; at.step < p.steps; ++it, at.next(p)) {
    const int s = it % S::kStages, half = it & 1;
    const bool there = mbar_wait_parked(&sm.full[s], (it / S::kStages) & 1, &g_gs_errors);
    if (!there) sm.dead = 1;
    const int cb = at.cb, row = at.row, step = at.step;
    const int t0 = step * kApplyTile, n = (int)min((int64_t)kApplyTile, p.L - t0);
    const int d = cb * kApplyWidth + 2 * lane;
    F2 dl = f2(0.0f);
    if (there && first < n) {
      const float2 nn = *reinterpret_cast<const float2 *>(&sm.ncs[s][2 * lane]);
      bool fast = near(nn) && n - first >= kGsChunk && d < p.D;
      if (PACKED) fast = fast && !(lane < kGsChunk && (sm.marks[s][first + lane % kGsChunk] & 3));
      if (__all_sync(0xffffffffu, fast))
        dl = apply_tokens<T, GATED, PACKED, true>(sm, s, q, row, t0, n, first, lane, d);
      else
        dl = apply_tokens<T, GATED, PACKED, false>(sm, s, q, row, t0, n, first, lane, d);
    }
    sm.dl[half][warp][lane] = unpack(dl);
    fence_proxy_async_smem();  // the states written into the stage, before copies come there
    segments_done();  // every warp is done with the stage
    if (*reinterpret_cast<volatile int *>(&sm.dead)) {
      // what this block has under way lands before it leaves
      if (threadIdx.x == kFetcher)
        for (int i = it; i < it + S::kStages && at.step < p.steps; ++i, at.next(p))
          mbar_wait_parked(&sm.full[i % S::kStages], (i / S::kStages) & 1, &g_gs_errors);
      return;
    }
    if (threadIdx.x == kFetcher) {
      fetch(s, ahead);
      ahead.next(p);
    }
    if (warp == 0) {  // (the next tile's sums go to the other half)
      float2 v = sm.dl[half][0][lane];
#pragma unroll
      for (int k = 1; k < kWarps; ++k) {
        v.x += sm.dl[half][k][lane].x;
        v.y += sm.dl[half][k][lane].y;
      }
      *reinterpret_cast<float2 *>(
          q.dl + ((int64_t)row * p.steps + step) * (p.nblk * kApplyWidth) + d) = v;
    }
  }
}

// ---------------------------------------------------------------- dlam
// Sums of up to kSumRows rows of `in` [n][width] each, in a fixed order; the last round
// turns the sum into the gradient.
constexpr int kSumRows = 512, kSumGroups = 16;
__global__ void __launch_bounds__(32 * kSumGroups)
    gs_sum_kernel(const float *in, int64_t n, int width, float *out, const float *lam, float c, int D,
                  const unsigned int *bad) {
  grid_dependency_wait();
  launch_dependents();
  if (bad != nullptr && *bad) return;
  __shared__ float part[kSumGroups][33];
  const int lane = threadIdx.x & 31, group = threadIdx.x >> 5;
  const int d = blockIdx.y * 32 + lane;
  const int64_t r0 = (int64_t)blockIdx.x * kSumRows, r1 = min(n, r0 + kSumRows);
  float s = 0.0f;
  if (d < width) {
#pragma unroll 8
    for (int64_t r = r0 + group; r < r1; r += kSumGroups) s += in[r * width + d];
  }
  part[group][lane] = s;
  __syncthreads();
  if (group != 0 || d >= width) return;
  for (int k = 1; k < kSumGroups; ++k) s += part[k][lane];
  if (lam == nullptr) out[(int64_t)blockIdx.x * width + d] = s;
  else if (d < D) out[d] = -c * gs_sigmoid(lam[d]) * s;
}

// Where the parts of the backward pass's workspace are.
struct BackPlan {
  Plan scan;  // its own parts first
  size_t carry, ck, dl, sums, forward, total;
  int64_t partials;
};
BackPlan back_plan(int64_t rows, int64_t L, int D, int io, bool packed, int carry_tile) {
  BackPlan b;
  b.scan = plan_of(rows, L, D, carry_tile, packed);
  const size_t chunks = (size_t)(rows * ceil_div(L, kGsChunk)) * D * 4;
  const size_t width = (size_t)ceil_div(D, kApplyWidth) * kApplyWidth * 4;
  b.partials = rows * ceil_div(L, kApplyTile);
  b.carry = align_up(b.scan.total, 256);
  b.ck = b.carry + align_up(chunks, 256);
  b.dl = b.ck + align_up(chunks, 256);
  b.sums = b.dl + (size_t)b.partials * width;
  b.forward = b.sums + (b.partials > kSumRows ? 2 * (size_t)ceil_div(b.partials, kSumRows) * width : 0);
  b.total = b.forward + gated_scan_workspace(rows, L, D, io, packed);
  return b;
}

template <typename T, bool PACKED, bool GATED>
cudaError_t launch(const GatedScanBackwardArgs &b, const Scan &p, const float *ck, float *carry,
                   float *dl) {
  const GatedScanArgs &a = b.f;
  const int64_t rows = a.rows();
  const void *in[5] = {a.x, a.r, a.g, b.dy, a.z};
  const int64_t ld[5] = {a.ld_x, a.ld_r, a.ld_g, a.D, a.ld_z};
  Maps apply = {}, back = {};
  for (int k = 0; k < (GATED ? 5 : 4); ++k)
    if (!gs_tensor_map(&apply.m[k], a.io, in[k], rows, a.L, a.D, ld[k], kApplyWidth, kApplyTile))
      return cudaErrorInvalidValue;
  constexpr int kOf[3] = {1, 3, 4};  // r, dy, z
  for (int k = 0; k < (GATED ? 3 : 2); ++k)
    if (!gs_tensor_map(&back.m[k], a.io, in[kOf[k]], rows, a.L, a.D, ld[kOf[k]], kWidth,
                       kCarryTile<T, GATED>))
      return cudaErrorInvalidValue;
  {
    constexpr size_t smem = sizeof(CarryTiles<T, GATED>);
    static_assert((kCarryResident<T, GATED>)*(smem + 1024 + 256) <= 228 * 1024, "blocks to an SM");
    static ContextOnce once;
    const cudaError_t e = launch_dependent(
        gs_back_carry_kernel<T, PACKED, GATED>, once,
        std::min(p.tiles, kCarryResident<T, GATED> * sm_count()), kThreads, smem, a.stream, back, p,
        b.dh, carry);
    if (e != cudaSuccess) return e;
  }
  constexpr size_t smem = sizeof(ApplyShared<T, GATED>);
  static_assert((kApplyResident<T, GATED>)*(smem + 1024 + 256) <= 228 * 1024, "blocks to an SM");
  static ContextOnce once;
  Apply<T> q;
  q.p = p;
  q.p.steps = (int)ceil_div(a.L, kApplyTile);
  q.p.nblk = (int)ceil_div(a.D, kApplyWidth);
  q.p.tiles = (int)(rows * q.p.steps * q.p.nblk);
  q.ck = ck;
  q.carry = carry;
  q.h_in = b.h_in;
  q.dh = b.dh;
  q.dx = static_cast<T *>(b.dx);
  q.dr = static_cast<T *>(b.dr);
  q.dg = static_cast<T *>(b.dg);
  q.dz = static_cast<T *>(b.dz);
  q.dh_in = b.dh_in;
  q.dl = dl;
  q.zero = 0;
  return launch_dependent(gs_back_apply_kernel<T, PACKED, GATED>, once,
                          std::min(q.p.tiles, kApplyResident<T, GATED> * sm_count()), kApplyThreads, smem,
                          a.stream, apply, q);
}

template <typename T> cudaError_t backward(const GatedScanBackwardArgs &b) {
  const GatedScanArgs &a = b.f;
  const bool packed = a.cu != nullptr;
  const BackPlan w =
      back_plan(a.rows(), a.L, a.D, a.io, packed,
                a.z != nullptr ? kCarryTile<T, true> : kCarryTile<T, false>);
  const float *ck = b.ck;
  if (ck == nullptr) {  // the forward again, for the states that enter the chunks
    GatedScanArgs f = a;
    f.y = nullptr;
    f.h = const_cast<float *>(b.h_in);
    f.states_in = b.h_in != nullptr;
    f.no_state_out = true;
    f.ck = reinterpret_cast<float *>(a.ws + w.ck);
    f.ws = a.ws + w.forward;
    const cudaError_t e = gated_scan_prefill(f);
    if (e != cudaSuccess) return e;
    ck = f.ck;
  }
  Scan p;
  // (a sequence without tokens hands its state's gradient on)
  cudaError_t e = prepare(a, w.scan, a.ws, b.dh, b.dh, b.dh_in, &p);
  if (e != cudaSuccess) return e;
  float *carry = reinterpret_cast<float *>(a.ws + w.carry), *dl = reinterpret_cast<float *>(a.ws + w.dl);
  if (packed)
    e = a.z != nullptr ? launch<T, true, true>(b, p, ck, carry, dl)
                       : launch<T, true, false>(b, p, ck, carry, dl);
  else
    e = a.z != nullptr ? launch<T, false, true>(b, p, ck, carry, dl)
                       : launch<T, false, false>(b, p, ck, carry, dl);
  if (e != cudaSuccess) return e;
  const int width = (int)ceil_div(a.D, kApplyWidth) * kApplyWidth;
  const unsigned int *bad = packed ? p.bad : nullptr;
  const float *from = dl;
  float *to = reinterpret_cast<float *>(a.ws + w.sums);
  for (int64_t n = w.partials;;) {
    const int64_t m = ceil_div(n, kSumRows);
    const bool last = m == 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)m, (unsigned)ceil_div(width, 32), 1);
    cfg.blockDim = dim3(32 * kSumGroups, 1, 1);
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, gs_sum_kernel, from, n, width, last ? b.dlam : to,
                           last ? a.lam : (const float *)nullptr, a.c, a.D, bad);
    if (e != cudaSuccess || last) break;
    from = to;
    to += m * width;
    n = m;
  }
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

size_t gated_scan_backward_workspace(int64_t rows, int64_t L, int D, int io, bool packed) {
  return back_plan(rows, L, D, io, packed, 128).total;  // (the smaller of the tiles)
}

cudaError_t gated_scan_backward(const GatedScanBackwardArgs &b) {
  return b.f.io == MAMBA2_BF16 ? backward<__nv_bfloat16>(b) : backward<float>(b);
}

cudaError_t take_gated_scan_backward_errors(unsigned int *out) {
  unsigned int v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_gs_errors, sizeof(v));
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_gs_errors, &zero, sizeof(zero));
  *out = v;
  return e;
}

cudaError_t set_gated_scan_backward_stall(unsigned int v) {
  return cudaMemcpyToSymbol(g_gs_stall, &v, sizeof(v));
}

}  // namespace m2
