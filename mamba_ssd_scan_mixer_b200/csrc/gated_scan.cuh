// The gated linear recurrence: problem description and the per-token arithmetic
// shared by its prefill, step and backward kernels.
//
// With s = softplus(lam) per channel, R = sigmoid(r), G = sigmoid(g):
//     la = -c s R      a = exp(la)      m = sqrt(1 - a^2)
//     h_t = a h_{t-1} + m G x_t         y_t = h_t  [ * silu(z_t) ]
#pragma once

#include <cuda.h>

#include <atomic>

#include "common.cuh"

namespace m2 {

// Tokens of one checkpoint.
constexpr int kGsChunk = MAMBA2_GATED_SCAN_CHUNK;

struct GatedScanArgs {
  int64_t batch, L;  // packed rows: sequences, total tokens
  int D, io;
  float c;
  const float *lam;
  const void *x, *r, *g, *z;  // z may be null
  int64_t ld_x, ld_r, ld_g, ld_z;
  const int32_t *cu;  // packed rows: [batch + 1]; else null
  void *y;
  float *h;  // state in and out, or null
  int states_in;
  bool no_state_out = false;  // h is only read
  float *ck = nullptr;        // checkpoints, or null
  char *ws;
  cudaStream_t stream;
  int64_t rows() const { return cu != nullptr ? 1 : batch; }
  int64_t nchunks() const { return ceil_div(L, kGsChunk); }
};

struct GatedScanBackwardArgs {
  GatedScanArgs f;  // the forward's inputs (y, h and ck of the forward unused)
  const float *h_in;   // or null
  const void *dy;      // contiguous
  const float *dh;     // gradient of the final state, or null
  const float *ck;     // checkpoints of the forward, or null (recomputed)
  void *dx, *dr, *dg, *dz;
  float *dlam, *dh_in;  // dh_in may be null
};

cudaError_t gated_scan_prefill(const GatedScanArgs &a);
size_t gated_scan_workspace(int64_t rows, int64_t L, int D, int io, bool packed);
cudaError_t gated_scan_step(const GatedScanArgs &a);
cudaError_t gated_scan_backward(const GatedScanBackwardArgs &a);
size_t gated_scan_backward_workspace(int64_t rows, int64_t L, int D, int io, bool packed);
cudaError_t take_gated_scan_errors(unsigned int *out);
cudaError_t set_gated_scan_stall(unsigned int v);
cudaError_t take_gated_scan_backward_errors(unsigned int *out);
cudaError_t set_gated_scan_backward_stall(unsigned int v);
// Tiles of 64 tokens and 32 channels in a row: those of a call are counted in 32 bits.
inline int64_t gs_tiles(int64_t L, int64_t D) { return ceil_div(L, 64) * ceil_div(D, 32); }

// ---------------------------------------------------------------- arithmetic
__device__ __forceinline__ float gs_sigmoid(float v) { return 1.0f / (1.0f + expf(-v)); }

// Pairs of fp32 values in one 64-bit register: two multiply-adds an instruction.
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ F2 f2(float a) { return f2(a, a); }
__device__ __forceinline__ float2 unpack(F2 p) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 mul2_flush(F2 a, F2 b) {  // subnormal results become zero
  F2 r;
  asm("mul.rn.ftz.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float sqrt_ap(float x) {
  float r;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

constexpr float kLog2e = 1.4426950408889634f;

// sigmoid: the exponential overflows to infinity for very negative arguments, and its
// reciprocal is then zero; NaN stays NaN.
__device__ __forceinline__ F2 sigmoid2(F2 x) {
  const float2 t = unpack(mul2(x, f2(-kLog2e)));
  const float2 q = unpack(add2(f2(ex2(t.x), ex2(t.y)), f2(1.0f)));
  return f2(rcp(q.x), rcp(q.y));
}

// 2^f - 1 = f P(f) for |f| <= 1/2; P of degree 5, fitted here to 2.1e-8 of its value.
__device__ __forceinline__ F2 exp2m1(F2 f) {
  F2 q = fma2(f, f2(1.5403507859446108e-4f), f2(1.3390735257416964e-3f));
  q = fma2(f, q, f2(9.618237614631653e-3f));
  q = fma2(f, q, f2(5.550357326865196e-2f));
  q = fma2(f, q, f2(2.4022649228572845e-1f));
  return mul2(f, fma2(f, q, f2(6.931471824645996e-1f)));
}

// a = 2^t and less = a - 1 for t <= 0, both to a few half-steps relative to themselves.
// NEAR: t > -1/2 for every channel of the warp, so that a > 0.7; else t = k + f and
// a - 1 = 2^k (2^f - 1) + (2^k - 1), which cancels nowhere.  Where t > -1/2 the second way
// has k = 0 and rounds as the first does: a channel's numbers do not depend on its warp's
// others.  (near: of -c softplus(lam) log2(e), which times a gate of one or a step above is t.)
__device__ __forceinline__ bool near(float2 ncs) { return fminf(ncs.x, ncs.y) >= -0.4999995f; }
template <bool NEAR> __device__ __forceinline__ void decay2(F2 t, F2 *a, F2 *less) {
  if (NEAR) {
    *less = exp2m1(t);
    *a = add2(*less, f2(1.0f));
    return;
  }
  const float2 u = unpack(t);
  t = f2(max_nan(u.x, -125.0f), max_nan(u.y, -125.0f));  // 2^-125 is as good as zero
  const F2 kk = add2(t, f2(12582912.0f));  // 1.5 2^23: rounds, and leaves k in the low bits
  const F2 q = exp2m1(fma2(add2(kk, f2(-12582912.0f)), f2(-1.0f), t));
  const float2 ki = unpack(kk);
  const F2 s = f2(__int_as_float((__float_as_int(ki.x) << 23) + 0x3f800000),
                  __int_as_float((__float_as_int(ki.y) << 23) + 0x3f800000));
  *less = fma2(s, q, add2(s, f2(-1.0f)));
  *a = fma2(s, q, s);
}

// The recurrence's coefficients for two channels of a token: a and b = m G x.
//
// What bounds them is the unit of ex2, rcp and sqrt (16 lanes a clock and SM): R and G
// share a reciprocal, R = (1 + e^-g) / P and G = (1 + e^-r) / P with P their
// denominators' product.  r and g come cut off at -43 for that (gs_clamp), so that P
// stays finite; a gate below 2^-62 counts as 2^-62.  m is taken of v = 1 - a^2 times
// 2^-70, where the square root flushes v < 2^-56 to zero: r = -inf leaves the state
// exactly as it was (for c softplus(lam) < 32), and an increment lost is below 4e-9 of
// x.  The 2^35 that m then lacks is in G.
struct Coeffs {
  F2 a, b, t, less, m, er, eg;  // (m scaled by 2^-35); er, eg: e^-r, e^-g
};
constexpr float kGateScale = 34359738368.0f;  // 2^35
struct Gates {
  F2 R, G;  // (G scaled by 2^35)
};
// The gates of e^-r and e^-g; `one` and `down` are 1 and 2^-35.
__device__ __forceinline__ Gates gates(F2 er, F2 eg, F2 one, F2 down) {
  const F2 pr = add2(er, one), pg = fma2(eg, down, down);
  const float2 P = unpack(mul2(pr, pg));
  const F2 inv = f2(rcp(P.x), rcp(P.y));
  return Gates{mul2(pg, inv), mul2(pr, inv)};
}
template <bool NEAR>
__device__ __forceinline__ Coeffs coefficients(F2 x, F2 r, F2 g, F2 ncs) {
  constexpr float down = 1.0f / kGateScale, down2 = down * down;
  Coeffs c;
  const float2 er = unpack(mul2(r, f2(-kLog2e))), eg = unpack(mul2(g, f2(-kLog2e)));
  c.er = f2(ex2(er.x), ex2(er.y));
  c.eg = f2(ex2(eg.x), ex2(eg.y));
  const Gates k = gates(c.er, c.eg, f2(1.0f), f2(down));
  c.t = mul2(ncs, k.R);
  decay2<NEAR>(c.t, &c.a, &c.less);
  const float2 v = unpack(mul2(c.less, fma2(c.a, f2(-down2), f2(-down2))));
  c.m = f2(sqrt_ap(v.x), sqrt_ap(v.y));
  c.b = mul2(mul2(c.m, k.G), x);
  return c;
}

// Two channels of a row, and the same cut off for coefficients().
template <typename T> __device__ __forceinline__ F2 gs_pair(const void *p);
template <> __device__ __forceinline__ F2 gs_pair<float>(const void *p) {
  const float2 v = *reinterpret_cast<const float2 *>(p);
  return f2(v.x, v.y);
}
template <> __device__ __forceinline__ F2 gs_pair<__nv_bfloat16>(const void *p) {
  const uint32_t w = *reinterpret_cast<const uint32_t *>(p);
  return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <typename T> __device__ __forceinline__ F2 gs_clamped(const void *p);
template <> __device__ __forceinline__ F2 gs_clamped<float>(const void *p) {
  const float2 v = *reinterpret_cast<const float2 *>(p);
  return f2(max_nan(v.x, -43.0f), max_nan(v.y, -43.0f));
}
template <> __device__ __forceinline__ F2 gs_clamped<__nv_bfloat16>(const void *p) {
  uint32_t w;
  asm("max.NaN.bf16x2 %0, %1, %2;"
      : "=r"(w)
      : "r"(*reinterpret_cast<const uint32_t *>(p)), "r"(0xc22cc22cu));
  return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// Tensor maps and the copies they describe.
__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, int c0, int c1,
                                            int c2, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
      : "memory");
}
// Host: whether something that belongs to a context (a launch attribute) has been set in
// the current one.  Setting it twice is harmless, so that two threads may both do it.
struct ContextOnce {
  std::atomic<unsigned long long> seen[64] = {};
  bool done() {
    int d = 0;
    if (cudaGetDevice(&d) != cudaSuccess || d < 0 || d >= 64) return false;
    const unsigned long long id = current_context_id();
    return id != 0 && seen[d].load(std::memory_order_acquire) == id;
  }
  void set() {
    int d = 0;
    if (cudaGetDevice(&d) == cudaSuccess && d >= 0 && d < 64)
      seen[d].store(current_context_id(), std::memory_order_release);
  }
};

// [rows][L][D] with a token stride of ld elements, in boxes of `tokens` by `width`
// channels; false if it cannot be described.
bool gs_tensor_map(CUtensorMap *m, int io, const void *base, int64_t rows, int64_t L, int D,
                   int64_t ld, int width, int tokens);

// Records that blocks pass to one another.  A word that has not been written holds
// kUnset, a NaN that no arithmetic gives, so that each word tells by itself whether it is
// there: no flag, no fence, one trip to L2.
constexpr unsigned int kUnset = 0xffffffffu;
__device__ __forceinline__ void record_put(float4 *p, float4 v) {
  asm volatile("st.relaxed.gpu.global.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(v.x), "f"(v.y),
               "f"(v.z), "f"(v.w)
               : "memory");
}
__device__ __forceinline__ void record_put(float2 *p, float2 v) {
  asm volatile("st.relaxed.gpu.global.v2.f32 [%0], {%1, %2};" ::"l"(p), "f"(v.x), "f"(v.y)
               : "memory");
}
__device__ __forceinline__ float4 record_get(const float4 *p) {
  float4 v;
  asm volatile("ld.relaxed.gpu.global.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
__device__ __forceinline__ float2 record_get(const float2 *p) {
  float2 v;
  asm volatile("ld.relaxed.gpu.global.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ bool is_set(float2 v) {
  return max(__float_as_uint(v.x), __float_as_uint(v.y)) != kUnset;
}
__device__ __forceinline__ bool is_set(float4 v) {
  return max(max(__float_as_uint(v.x), __float_as_uint(v.y)),
             max(__float_as_uint(v.z), __float_as_uint(v.w))) != kUnset;
}
// Whether a phase is complete, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Waits for a phase, for at most kWaitLimitNs; false (and the flag) if it never came.  The
// hint lets the hardware park the warp instead of having it ask again and again, which
// took a third of all instructions issued.
__device__ __forceinline__ bool mbar_wait_parked(uint64_t *bar, uint32_t parity,
                                                 unsigned int *err) {
  unsigned long long since = 0;
  for (;;) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(1000000u)
        : "memory");
    if (ok) return true;
    const unsigned long long now = globaltimer_ns();
    if (since == 0) since = now;
    if (now - since > kWaitLimitNs) {
      atomicOr(err, kErrWaitTimeout);
      return false;
    }
  }
}

// The map of a state across a stretch of tokens, h_out = A h_in + H, for two channels:
// (A, A', H, H').  A sequence that begins inside the stretch leaves A = -0: what comes
// in is then not multiplied by zero but left out, so that a NaN of the sequence before
// stays there.  (A product of decays is never negative.)
__device__ __forceinline__ float2 gs_through(float4 m, float2 h) {
  h.x = __float_as_int(m.x) == (int)0x80000000 ? m.z : fmaf(m.x, h.x, m.z);
  h.y = __float_as_int(m.y) == (int)0x80000000 ? m.w : fmaf(m.y, h.y, m.w);
  return h;
}
// First one stretch, then another.
__device__ __forceinline__ float4 gs_then(float4 one, float4 two) {
  const float2 h = gs_through(two, make_float2(one.z, one.w));
  return make_float4(__float_as_int(two.x) == (int)0x80000000 ? two.x : one.x * two.x,
                     __float_as_int(two.y) == (int)0x80000000 ? two.y : one.y * two.y, h.x, h.y);
}

// Two neighbouring channels.
template <typename T> struct Pair;
template <> struct Pair<float> {
  using V = float2;
  static __device__ __forceinline__ float2 get(float2 v) { return v; }
  static __device__ __forceinline__ float2 put(float a, float b) { return make_float2(a, b); }
};
template <> struct Pair<__nv_bfloat16> {
  using V = __nv_bfloat162;
  static __device__ __forceinline__ float2 get(__nv_bfloat162 v) { return __bfloat1622float2(v); }
  static __device__ __forceinline__ __nv_bfloat162 put(float a, float b) {
    return __floats2bfloat162_rn(a, b);
  }
};
template <typename T> __device__ __forceinline__ void st2(T *p, float2 v) {
  *reinterpret_cast<typename Pair<T>::V *>(p) = Pair<T>::put(v.x, v.y);
}

}  // namespace m2
