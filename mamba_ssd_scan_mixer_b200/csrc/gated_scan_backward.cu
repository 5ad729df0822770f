// Backward pass of the gated linear recurrence (gated_scan.cuh).
//
// With d_t the gradient of h_t (of the last token's: plus the final state's),
//     d_t  = dy_t silu(z_t) + a_{t+1} d_{t+1}
//     dx   = d m G               dg = d m x G (1 - G)        dz = dy h silu'(z)
//     dla  = d (a h_{t-1} - a^2 / m G x)
//     dr   = dla la (1 - R)      dlam = sum dla (-c R) sigmoid(lam)
#include "gated_scan.cuh"

namespace m2 {
namespace {

constexpr int kThreads = 64;  // two channels each
constexpr int kSub = 16;      // tokens whose states are held in registers

template <typename T> struct Bwd {
  const T *x, *r, *g, *z, *dy;
  int64_t ld_x, ld_r, ld_g, ld_z;
  const float *lam, *h_in, *dh, *ck;
  T *dx, *dr, *dg, *dz;
  float *dh_in;
  float c;
  int64_t L, nch, batch;
  int D;
  const int32_t *cu;
  float *P, *Q, *carry, *dlam_part;
  const unsigned int *bad;
};

__device__ __forceinline__ float2 silu2(float2 z) {
  return make_float2(z.x * gs_sigmoid(z.x), z.y * gs_sigmoid(z.y));
}

// What a chunk hands to the token before it (a d of its first token), as a map
// of what it is handed: out = P in + Q.
template <typename T> __global__ void gs_back_chunk_kernel(Bwd<T> p) {
  __shared__ int first[kGsChunk], last[kGsChunk];
  if (p.cu != nullptr && *p.bad) return;
  const int64_t rc = blockIdx.x, row = rc / p.nch, t0 = (rc % p.nch) * kGsChunk;
  const int n = (int)min((int64_t)kGsChunk, p.L - t0);
  if (p.cu != nullptr) gs_marks(p.cu, p.batch, t0, n, first, last);
  const int d = 2 * (blockIdx.y * kThreads + threadIdx.x);
  if (d >= p.D) return;
  const float ncs0 = -p.c * softplus_f(p.lam[d]), ncs1 = -p.c * softplus_f(p.lam[d + 1]);
  float2 P = make_float2(1.0f, 1.0f), e = make_float2(0.0f, 0.0f);
  for (int i = n - 1; i >= 0; --i) {
    const int64_t t = row * p.L + t0 + i;
    const float2 r = ld2(p.r + t * p.ld_r + d);
    float2 dy = ld2(p.dy + t * p.D + d);
    if (p.z != nullptr) {
      const float2 s = silu2(ld2(p.z + t * p.ld_z + d));
      dy.x *= s.x;
      dy.y *= s.y;
    }
    if (p.cu != nullptr && last[i] >= 0 && p.dh != nullptr) {
      const float2 f = *reinterpret_cast<const float2 *>(p.dh + (int64_t)last[i] * p.D + d);
      dy.x += f.x;
      dy.y += f.y;
    }
    const float a0 = expf(ncs0 * gs_sigmoid(r.x)), a1 = expf(ncs1 * gs_sigmoid(r.y));
    e.x = a0 * (dy.x + e.x);
    e.y = a1 * (dy.y + e.y);
    P.x *= a0;
    P.y *= a1;
    if (p.cu != nullptr && first[i] >= 0) P = e = make_float2(0.0f, 0.0f);
  }
  *reinterpret_cast<float2 *>(p.P + rc * p.D + d) = P;
  *reinterpret_cast<float2 *>(p.Q + rc * p.D + d) = e;
}

template <typename T> __global__ void gs_back_carry_kernel(Bwd<T> p) {
  if (p.cu != nullptr && *p.bad) return;
  const int d = blockIdx.x * blockDim.x + threadIdx.x;
  if (d >= p.D) return;
  const int64_t row = blockIdx.y;
  float e = p.cu == nullptr && p.dh != nullptr ? p.dh[row * p.D + d] : 0.0f;
  for (int64_t j = p.nch - 1; j >= 0; --j) {
    const int64_t o = (row * p.nch + j) * p.D + d;
    p.carry[o] = e;
    e = p.P[o] == 0.0f ? p.Q[o] : p.P[o] * e + p.Q[o];
  }
  if (p.cu == nullptr && p.dh_in != nullptr) p.dh_in[row * p.D + d] = e;
}

template <typename T> __global__ void gs_back_apply_kernel(Bwd<T> p) {
  __shared__ int first[kGsChunk], last[kGsChunk];
  if (p.cu != nullptr && *p.bad) return;
  const int64_t rc = blockIdx.x, row = rc / p.nch, t0 = (rc % p.nch) * kGsChunk;
  const int n = (int)min((int64_t)kGsChunk, p.L - t0);
  if (p.cu != nullptr) gs_marks(p.cu, p.batch, t0, n, first, last);
  const int d = 2 * (blockIdx.y * kThreads + threadIdx.x);
  if (d >= p.D) return;
  const float ncs[2] = {-p.c * softplus_f(p.lam[d]), -p.c * softplus_f(p.lam[d + 1])};
  const float2 c0 = *reinterpret_cast<const float2 *>(p.ck + rc * p.D + d);
  const float2 e0 = *reinterpret_cast<const float2 *>(p.carry + rc * p.D + d);
  float start[kGsChunk / kSub][2], h[2] = {c0.x, c0.y}, e[2] = {e0.x, e0.y};
  float dl[2] = {0.0f, 0.0f};
  auto state_before = [&](int i) {  // a sequence's first token starts from its own state
    if (p.cu == nullptr || first[i] < 0) return;
    const float2 v = p.h_in != nullptr ? *reinterpret_cast<const float2 *>(
                                             p.h_in + (int64_t)first[i] * p.D + d)
                                       : make_float2(0.0f, 0.0f);
    h[0] = v.x;
    h[1] = v.y;
  };
  for (int i = 0; i < n; ++i) {
    const int64_t t = row * p.L + t0 + i;
    if (i % kSub == 0) {
      start[i / kSub][0] = h[0];
      start[i / kSub][1] = h[1];
    }
    state_before(i);
    const float2 x = ld2(p.x + t * p.ld_x + d), r = ld2(p.r + t * p.ld_r + d),
                 g = ld2(p.g + t * p.ld_g + d);
    const Gate u = gs_gate(r.x, g.x, ncs[0]), v = gs_gate(r.y, g.y, ncs[1]);
    h[0] = u.a * h[0] + u.m * u.G * x.x;
    h[1] = v.a * h[1] + v.m * v.G * x.y;
  }
  for (int b = (n - 1) / kSub; b >= 0; --b) {
    float before[kSub][2];
    const int i1 = min(n, (b + 1) * kSub);
    h[0] = start[b][0];
    h[1] = start[b][1];
    for (int i = b * kSub; i < i1; ++i) {
      const int64_t t = row * p.L + t0 + i;
      state_before(i);
      before[i - b * kSub][0] = h[0];
      before[i - b * kSub][1] = h[1];
      const float2 x = ld2(p.x + t * p.ld_x + d), r = ld2(p.r + t * p.ld_r + d),
                   g = ld2(p.g + t * p.ld_g + d);
      const Gate u = gs_gate(r.x, g.x, ncs[0]), v = gs_gate(r.y, g.y, ncs[1]);
      h[0] = u.a * h[0] + u.m * u.G * x.x;
      h[1] = v.a * h[1] + v.m * v.G * x.y;
    }
    for (int i = i1 - 1; i >= b * kSub; --i) {
      const int64_t t = row * p.L + t0 + i;
      const float2 x2 = ld2(p.x + t * p.ld_x + d), r2 = ld2(p.r + t * p.ld_r + d),
                   g2 = ld2(p.g + t * p.ld_g + d), dy2 = ld2(p.dy + t * p.D + d);
      const float x[2] = {x2.x, x2.y}, r[2] = {r2.x, r2.y}, g[2] = {g2.x, g2.y},
                  dy[2] = {dy2.x, dy2.y};
      float z[2] = {0.0f, 0.0f}, dx[2], dr[2], dg[2], dz[2];
      if (p.z != nullptr) {
        const float2 z2 = ld2(p.z + t * p.ld_z + d);
        z[0] = z2.x;
        z[1] = z2.y;
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const Gate q = gs_gate(r[k], g[k], ncs[k]);
        const float hp = before[i - b * kSub][k], ht = q.a * hp + q.m * q.G * x[k];
        float dh = dy[k];
        if (p.z != nullptr) {
          const float s = gs_sigmoid(z[k]);
          dz[k] = dy[k] * ht * s * (1.0f + z[k] * (1.0f - s));
          dh *= z[k] * s;
        }
        if (p.cu != nullptr && last[i] >= 0 && p.dh != nullptr)
          dh += p.dh[(int64_t)last[i] * p.D + d + k];
        const float dt = dh + e[k];
        dx[k] = dt * q.m * q.G;
        dg[k] = dx[k] * x[k] * (1.0f - q.G);
        // as la -> 0 both la / m and R / m go to zero with m
        const float per_m = q.m > 0.0f ? 1.0f / q.m : 0.0f;
        const float dla = dt * (q.a * hp - q.a * q.a * per_m * q.G * x[k]);
        dr[k] = dla * q.la * (1.0f - q.R);
        dl[k] += dla * q.R;
        e[k] = q.a * dt;
      }
      st2(p.dx + t * p.D + d, dx[0], dx[1]);
      st2(p.dr + t * p.D + d, dr[0], dr[1]);
      st2(p.dg + t * p.D + d, dg[0], dg[1]);
      if (p.z != nullptr) st2(p.dz + t * p.D + d, dz[0], dz[1]);
      if (p.cu != nullptr && first[i] >= 0) {
        if (p.dh_in != nullptr)
          *reinterpret_cast<float2 *>(p.dh_in + (int64_t)first[i] * p.D + d) =
              make_float2(e[0], e[1]);
        e[0] = e[1] = 0.0f;
      }
    }
  }
  *reinterpret_cast<float2 *>(p.dlam_part + rc * p.D + d) = make_float2(dl[0], dl[1]);
}

// Packed rows: a sequence without tokens hands its state's gradient on.
__global__ void gs_back_empty_kernel(const int32_t *cu, const float *dh, float *dh_in, int64_t n,
                                     int D, const unsigned int *bad) {
  if (*bad) return;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * blockDim.x)
    if (cu[i / D + 1] <= cu[i / D]) dh_in[i] = dh != nullptr ? dh[i] : 0.0f;
}

__global__ void gs_dlam_kernel(const float *part, int64_t n, int D, const float *lam, float c,
                               float *dlam, const unsigned int *bad) {
  if (bad != nullptr && *bad) return;
  const int d = blockIdx.x * blockDim.x + threadIdx.x;
  if (d >= D) return;
  float s = 0.0f;
  for (int64_t i = 0; i < n; ++i) s += part[i * D + d];
  dlam[d] = -c * gs_sigmoid(lam[d]) * s;
}

template <typename T> cudaError_t backward(const GatedScanBackwardArgs &b) {
  const GatedScanArgs &a = b.f;
  const int64_t rows = a.rows(), nch = a.nchunks();
  const size_t n = (size_t)rows * nch * a.D;
  unsigned int *bad = reinterpret_cast<unsigned int *>(a.ws);
  if (a.cu != nullptr) gated_scan_check(a.cu, a.batch, a.L, bad, a.stream);
  float *P = reinterpret_cast<float *>(a.ws + 256), *Q = P + n, *carry = Q + n, *part = carry + n,
        *own_ck = part + n;
  const float *ck = b.ck;
  if (ck == nullptr) {  // the forward again, for the states that enter the chunks
    GatedScanArgs f = a;
    f.y = nullptr;
    f.h = const_cast<float *>(b.h_in);
    f.states_in = b.h_in != nullptr;
    f.ck = own_ck;
    f.ws = a.ws + 256 + align_up(5 * n * 4, 256);
    f.no_state_out = true;
    const cudaError_t e = gated_scan_prefill(f);
    if (e != cudaSuccess) return e;
    ck = own_ck;
  }
  Bwd<T> p;
  p.x = static_cast<const T *>(a.x);
  p.r = static_cast<const T *>(a.r);
  p.g = static_cast<const T *>(a.g);
  p.z = static_cast<const T *>(a.z);
  p.dy = static_cast<const T *>(b.dy);
  p.ld_x = a.ld_x;
  p.ld_r = a.ld_r;
  p.ld_g = a.ld_g;
  p.ld_z = a.ld_z;
  p.lam = a.lam;
  p.h_in = b.h_in;
  p.dh = b.dh;
  p.ck = ck;
  p.dx = static_cast<T *>(b.dx);
  p.dr = static_cast<T *>(b.dr);
  p.dg = static_cast<T *>(b.dg);
  p.dz = static_cast<T *>(b.dz);
  p.dh_in = b.dh_in;
  p.c = a.c;
  p.L = a.L;
  p.nch = nch;
  p.batch = a.batch;
  p.D = a.D;
  p.cu = a.cu;
  p.P = P;
  p.Q = Q;
  p.carry = carry;
  p.dlam_part = part;
  p.bad = bad;
  const dim3 grid((unsigned)(rows * nch), (unsigned)ceil_div(a.D / 2, kThreads));
  gs_back_chunk_kernel<T><<<grid, kThreads, 0, a.stream>>>(p);
  gs_back_carry_kernel<T>
      <<<dim3((unsigned)ceil_div(a.D, 128), (unsigned)rows), 128, 0, a.stream>>>(p);
  gs_back_apply_kernel<T><<<grid, kThreads, 0, a.stream>>>(p);
  if (a.cu != nullptr && b.dh_in != nullptr)
    gs_back_empty_kernel<<<512, 256, 0, a.stream>>>(a.cu, b.dh, b.dh_in, a.batch * a.D, a.D, bad);
  gs_dlam_kernel<<<(unsigned)ceil_div(a.D, 128), 128, 0, a.stream>>>(part, rows * nch, a.D, a.lam,
                                                                    a.c, b.dlam, a.cu != nullptr ? bad : nullptr);
  return cudaGetLastError();
}

}  // namespace

size_t gated_scan_backward_workspace(int64_t rows, int64_t L, int D, int io, bool packed) {
  const size_t n = (size_t)rows * (size_t)ceil_div(L, kGsChunk) * (size_t)D;
  return 256 + align_up(5 * n * 4, 256) + gated_scan_workspace(rows, L, D, io, packed);
}

cudaError_t gated_scan_backward(const GatedScanBackwardArgs &b) {
  return b.f.io == MAMBA2_BF16 ? backward<__nv_bfloat16>(b) : backward<float>(b);
}

}  // namespace m2
