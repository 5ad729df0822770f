// Prefill and decode step of the gated linear recurrence (gated_scan.cuh).
#include "gated_scan.cuh"

namespace m2 {
namespace {

static __device__ unsigned int g_gs_errors = 0;

constexpr int kThreads = 64;  // two channels each

template <typename T> struct In {
  const T *x, *r, *g, *z;
  int64_t ld_x, ld_r, ld_g, ld_z;
};

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

// One chunk as a map of the state that enters it: h_out = A h_in + H.
template <typename T, bool APPLY>
__global__ void gs_chunk_kernel(In<T> in, const float *lam, float c, int64_t L, int64_t nch, int D,
                                const int32_t *cu, int64_t batch, const unsigned int *bad,
                                const float *h0, float *h_out, const float *carry, float *A_out,
                                float *H_out, T *y) {
  __shared__ int first[kGsChunk], last[kGsChunk];
  if (cu != nullptr && *bad) return;
  const int64_t row = blockIdx.x / nch, ch = blockIdx.x % nch, t0 = ch * kGsChunk;
  const int n = (int)min((int64_t)kGsChunk, L - t0);
  if (cu != nullptr) gs_marks(cu, batch, t0, n, first, last);
  const int d = 2 * (blockIdx.y * kThreads + threadIdx.x);
  if (d >= D) return;
  const float ncs0 = -c * softplus_f(lam[d]), ncs1 = -c * softplus_f(lam[d + 1]);
  const int64_t rc = blockIdx.x;
  float2 A = make_float2(1.0f, 1.0f), h = make_float2(0.0f, 0.0f);
  if (APPLY) h = *reinterpret_cast<const float2 *>(carry + rc * D + d);
  for (int i = 0; i < n; ++i) {
    const int64_t t = row * L + t0 + i;
    const float2 x = ld2(in.x + t * in.ld_x + d), r = ld2(in.r + t * in.ld_r + d),
                 g = ld2(in.g + t * in.ld_g + d);
    const Gate p = gs_gate(r.x, g.x, ncs0), q = gs_gate(r.y, g.y, ncs1);
    if (cu != nullptr && first[i] >= 0) {
      A = make_float2(0.0f, 0.0f);
      h = h0 != nullptr ? *reinterpret_cast<const float2 *>(h0 + (int64_t)first[i] * D + d)
                        : make_float2(0.0f, 0.0f);
    }
    A.x *= p.a;
    A.y *= q.a;
    h.x = p.a * h.x + p.m * p.G * x.x;
    h.y = q.a * h.y + q.m * q.G * x.y;
    if (APPLY) {
      if (y != nullptr) {
        float2 o = h;
        if (in.z != nullptr) {
          const float2 z = ld2(in.z + t * in.ld_z + d);
          o.x *= z.x * gs_sigmoid(z.x);
          o.y *= z.y * gs_sigmoid(z.y);
        }
        st2(y + t * D + d, o.x, o.y);
      }
      if (cu != nullptr && h_out != nullptr && last[i] >= 0)
        *reinterpret_cast<float2 *>(h_out + (int64_t)last[i] * D + d) = h;
    }
  }
  if (!APPLY) {
    *reinterpret_cast<float2 *>(A_out + rc * D + d) = A;
    *reinterpret_cast<float2 *>(H_out + rc * D + d) = h;
  }
}

// The state entering each chunk of a row, in order.
__global__ void gs_carry_kernel(const float *A, const float *H, float *carry, int64_t nch, int D,
                                const float *h0, float *h_out, bool packed,
                                const unsigned int *bad) {
  if (packed && *bad) return;
  const int d = blockIdx.x * blockDim.x + threadIdx.x;
  if (d >= D) return;
  const int64_t row = blockIdx.y;
  float h = !packed && h0 != nullptr ? h0[row * D + d] : 0.0f;
  for (int64_t j = 0; j < nch; ++j) {
    const int64_t o = (row * nch + j) * D + d;
    carry[o] = h;
    const float a = A[o];
    h = a == 0.0f ? H[o] : a * h + H[o];
  }
  if (!packed && h_out != nullptr) h_out[row * D + d] = h;
}

// Packed rows: the initial states put aside (the final ones overwrite them), and
// the final state of a sequence without tokens.
__global__ void gs_copy_kernel(const float *h, float *h0, const int32_t *cu, int64_t n, int D,
                               int states_in, float *h_out, const unsigned int *bad) {
  if (*bad) return;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * blockDim.x) {
    if (states_in) h0[i] = h[i];
    else if (h_out != nullptr && cu[i / D + 1] <= cu[i / D]) h_out[i] = 0.0f;
  }
}

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

template <typename T> cudaError_t prefill(const GatedScanArgs &a) {
  const int64_t rows = a.rows(), nch = a.nchunks();
  const size_t n = (size_t)rows * nch * a.D;
  unsigned int *bad = reinterpret_cast<unsigned int *>(a.ws);
  float *A = reinterpret_cast<float *>(a.ws + 256), *H = A + n, *carry = H + n, *h0 = carry + n;
  if (a.ck != nullptr) carry = a.ck;
  float *h_out = a.no_state_out ? nullptr : a.h;
  const bool packed = a.cu != nullptr;
  const float *start = a.states_in ? a.h : nullptr;
  if (packed) {
    gated_scan_check(a.cu, a.batch, a.L, bad, a.stream);
    if (a.h != nullptr) {
      gs_copy_kernel<<<512, 256, 0, a.stream>>>(a.h, h0, a.cu, a.batch * a.D, a.D, a.states_in,
                                                h_out, bad);
      if (a.states_in) start = h0;
    }
  }
  const dim3 grid((unsigned)(rows * nch), (unsigned)ceil_div(a.D / 2, kThreads));
  gs_chunk_kernel<T, false><<<grid, kThreads, 0, a.stream>>>(inputs<T>(a), a.lam, a.c, a.L, nch,
                                                             a.D, a.cu, a.batch, bad, start, h_out,
                                                             nullptr, A, H, nullptr);
  gs_carry_kernel<<<dim3((unsigned)ceil_div(a.D, 128), (unsigned)rows), 128, 0, a.stream>>>(
      A, H, carry, nch, a.D, start, h_out, packed, bad);
  if (a.y != nullptr)
    gs_chunk_kernel<T, true><<<grid, kThreads, 0, a.stream>>>(
        inputs<T>(a), a.lam, a.c, a.L, nch, a.D, a.cu, a.batch, bad, start, h_out, carry, nullptr,
        nullptr, static_cast<T *>(a.y));
  return cudaGetLastError();
}

template <typename T> cudaError_t step(const GatedScanArgs &a) {
  const int64_t n2 = a.batch * (a.D / 2);
  gs_step_kernel<T><<<(unsigned)ceil_div(n2, 128), 128, 0, a.stream>>>(
      inputs<T>(a), a.lam, a.c, n2, a.D, a.h, static_cast<T *>(a.y));
  return cudaGetLastError();
}

}  // namespace

void gated_scan_check(const int32_t *cu, int64_t batch, int64_t L, unsigned int *bad,
                      cudaStream_t stream) {
  gs_check_kernel<<<1, 1024, 0, stream>>>(cu, batch, L, bad);
}

size_t gated_scan_workspace(int64_t rows, int64_t L, int D, int64_t batch, bool packed) {
  const size_t n = (size_t)rows * (size_t)ceil_div(L, kGsChunk) * (size_t)D;
  return 256 + align_up(3 * n * 4 + (packed ? (size_t)batch * D * 4 : 0), 256);
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

}  // namespace m2
