// The gated linear recurrence: problem description and the per-token arithmetic
// shared by its prefill, step and backward kernels.
//
// With s = softplus(lam) per channel, R = sigmoid(r), G = sigmoid(g):
//     la = -c s R      a = exp(la)      m = sqrt(1 - a^2)
//     h_t = a h_{t-1} + m G x_t         y_t = h_t  [ * silu(z_t) ]
#pragma once

#include "common.cuh"

namespace m2 {

// Tokens of one tile of the scan, and of one checkpoint.
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
size_t gated_scan_workspace(int64_t rows, int64_t L, int D, int64_t batch, bool packed);
cudaError_t gated_scan_step(const GatedScanArgs &a);
cudaError_t gated_scan_backward(const GatedScanBackwardArgs &a);
size_t gated_scan_backward_workspace(int64_t rows, int64_t L, int D, int64_t batch, bool packed);
// Sets *bad to whether the offsets of packed rows are wrong (and raises the flag).
void gated_scan_check(const int32_t *cu, int64_t batch, int64_t L, unsigned int *bad,
                      cudaStream_t stream);
cudaError_t take_gated_scan_errors(unsigned int *out);

// ---------------------------------------------------------------- arithmetic
__device__ __forceinline__ float gs_sigmoid(float v) { return 1.0f / (1.0f + expf(-v)); }

struct Gate {
  float R, G, la, a, m;
};
// `ncs` = -c softplus(lam).  1 - a^2 comes from expm1, so that it keeps its
// relative accuracy where a is next to one.
__device__ __forceinline__ Gate gs_gate(float r, float g, float ncs) {
  Gate q;
  q.R = gs_sigmoid(r);
  q.G = gs_sigmoid(g);
  q.la = ncs * q.R;
  q.a = expf(q.la);
  q.m = sqrtf(-expm1f(2.0f * q.la));
  return q;
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
template <typename T> __device__ __forceinline__ float2 ld2(const T *p) {
  return Pair<T>::get(*reinterpret_cast<const typename Pair<T>::V *>(p));
}
template <typename T> __device__ __forceinline__ void st2(T *p, float a, float b) {
  *reinterpret_cast<typename Pair<T>::V *>(p) = Pair<T>::put(a, b);
}

// The sequences that begin or end inside tokens [t0, t0 + n) of packed rows:
// first[i] / last[i] = the sequence whose first / last token is t0 + i, else
// -1.  Called by the whole block; `n` <= kGsChunk.
__device__ __forceinline__ void gs_marks(const int32_t *cu, int64_t batch, int64_t t0, int n,
                                         int *first, int *last) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) first[i] = last[i] = -1;
  // the first sequence that ends after t0
  int64_t lo = 0, hi = batch;
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (cu[mid + 1] > t0) hi = mid;
    else lo = mid + 1;
  }
  __syncthreads();
  for (int64_t s = lo + threadIdx.x; s < batch; s += blockDim.x) {
    const int64_t b = cu[s], e = cu[s + 1];
    if (b >= t0 + n) break;
    if (e <= b) continue;
    if (b >= t0) first[b - t0] = (int)s;
    if (e - 1 >= t0 && e - 1 < t0 + n) last[e - 1 - t0] = (int)s;
  }
  __syncthreads();
}

}  // namespace m2
