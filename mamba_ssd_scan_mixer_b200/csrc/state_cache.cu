// The 8-bit state cache: recurrent states written into slots as codes of 8 bits
// with a power-of-two scale for each block of consecutive values, and read back.
//
// The scale 2^e of a block is the least power of two with amax <= qmax 2^e
// (qmax = 127 for int8, 448 for e4m3), kept as the biased exponent byte e + 127.
// A power of two makes v 2^-e exact, so the only rounding is the code's own (to
// nearest, ties to even), and a state that was read back and is written again
// gives the same values.
//
// Bytes bound both ways.  256 SSM states of 80 x 64 x 64 in fp32 (336 MB) into int8: 73 us,
// 5.7 TB/s; back: 67 us, 6.3 TB/s.  bf16: 46 and 41 us.  What a store lacks to the copy rate
// is the maximum that each block's values wait for, and the search for a later row of the
// same slot.  (2 us of each less than with launches that begin where the kernel before ends.)
#include <cuda_fp8.h>

#include "state_cache.cuh"

namespace m2 {
namespace {

static __device__ unsigned int g_sc_errors = 0;
constexpr unsigned int kErrSlots = 8u;  // bit 3 of mamba2_device_errors

// 2^(byte - 127); byte 0 is the subnormal 2^-127
__device__ __forceinline__ float pow2_of(int byte) {
  return __int_as_float(byte == 0 ? 0x00400000 : byte << 23);
}
// The biased exponent for a block of largest magnitude amax (255: not finite).
template <bool INT8> __device__ __forceinline__ int scale_byte(float amax) {
  const int bits = __float_as_int(amax);
  if (bits >= 0x7f800000) return 255;
  // amax = 1.f 2^E: qmax is 1.984375 2^6 or 1.75 2^8
  const int over = (bits & 0x7fffff) > (INT8 ? 0x7e0000 : 0x600000);
  return max(0, (bits >> 23) - (INT8 ? 6 : 8) + over);
}
// 2^(127 - byte), byte <= 249
__device__ __forceinline__ float inverse_of(int byte) {
  return __int_as_float((254 - byte) << 23);
}

// Four values times 2^-e (exact) as four codes, the first in the low byte.
template <bool INT8> __device__ __forceinline__ uint32_t encode4(const float *v, float inv) {
  if (INT8) {
    // adding 1.5 2^23 rounds to an integer (to nearest, ties to even) and leaves it
    // in the low bits
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = __float_as_uint(fmaf(v[i], inv, 12582912.0f));
    return __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
  }
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[0] * inv, v[1] * inv),
                                               __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[2] * inv, v[3] * inv),
                                               __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}
template <bool INT8> __device__ __forceinline__ uint32_t encode1(float v, float inv) {
  if (INT8) return __float_as_uint(fmaf(v, inv, 12582912.0f)) & 0xffu;
  return __nv_cvt_float_to_fp8(v * inv, __NV_SATFINITE, __NV_E4M3);
}
template <bool INT8>
__device__ __forceinline__ void decode4(uint32_t q, float scale, float *v) {
  if (INT8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (float)(int8_t)(q >> (8 * i)) * scale;
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 f = __half22float2(
          __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(q >> (16 * i)), __NV_E4M3)));
      v[2 * i] = f.x * scale;
      v[2 * i + 1] = f.y * scale;
    }
  }
}
template <bool INT8> __device__ __forceinline__ float decode1(uint32_t q, float scale) {
  if (INT8) return (float)(int8_t)q * scale;
  return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)q, __NV_E4M3))) * scale;
}
// The scale to decode with; NaN for a block that held something not finite.
__device__ __forceinline__ float scale_of(int byte) {
  return byte == 255 ? __int_as_float(0x7fffffff) : pow2_of(byte);
}

// The slot of batch row b, or -1 if nothing is to be done for it: a negative
// slot, or one out of range (flagged).
__device__ __forceinline__ int64_t slot_of(const int32_t *slots, int64_t b, int64_t nslots) {
  const int64_t s = slots[b];
  if (s >= nslots) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&g_sc_errors, kErrSlots);
    return -1;
  }
  return s < 0 ? -1 : s;
}
// Whether a later row names slot s too (then this row is not written).  Each block
// reads the rest of the slots: 4 bytes a row, small beside a state of thousands of
// values for batches of hundreds (4096 rows of 8192 values: 39 us, 26 at the copy rate; 65535
// rows of 512: 840 us, 26).
__device__ __forceinline__ bool named_later(const int32_t *slots, int64_t b, int64_t batch,
                                            int64_t s) {
  int later = 0;
  for (int64_t i = b + 1 + threadIdx.x; i < batch; i += blockDim.x) later |= slots[i] == s;
  return __syncthreads_or(later) != 0;
}

constexpr int kThreads = 256;

// 16 bytes of a state: V = 4 or 8 values.
template <typename T> struct Vec;
template <> struct Vec<float> {
  static constexpr int V = 4;
  static __device__ __forceinline__ void get(uint4 u, float *v) {
    v[0] = __uint_as_float(u.x), v[1] = __uint_as_float(u.y);
    v[2] = __uint_as_float(u.z), v[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 put(const float *v) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                      __float_as_uint(v[3]));
  }
};
template <> struct Vec<__nv_bfloat16> {
  static constexpr int V = 8;
  static __device__ __forceinline__ void get(uint4 u, float *v) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 put(const float *v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 q = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&q);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// Rows on 16-byte boundaries: a lane takes 16 bytes of the state, LANES lanes a
// block of LANES * V values; a warp has kU such pieces of 32 * V values under way.
constexpr int kU = 4;
// (No pointer is __restrict__: what nobody else changes may be read before the wait for
// the kernel that makes it.)
template <typename T, bool INT8, int LANES>
__global__ void __launch_bounds__(kThreads)
    store_vec_kernel(const T *state, int64_t ld, int64_t n, int64_t nb,
                     const int32_t *slots, int64_t batch, int64_t nslots,
                     uint8_t *codes, uint8_t *scales) {
  grid_dependency_wait();
  constexpr int V = Vec<T>::V;
  const int64_t b = blockIdx.y;
  const int lane = threadIdx.x & 31;
  const int64_t c0 = ((int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32) * kU;
  uint4 raw[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) {  // under way before the slots are looked at
    const int64_t i = (c0 + u) * (32 * V) + lane * V;
    raw[u] = i < n ? __ldcs(reinterpret_cast<const uint4 *>(state + b * ld + i))
                   : make_uint4(0, 0, 0, 0);
  }
  const int64_t s = slot_of(slots, b, nslots);
  if (s < 0 || named_later(slots, b, batch, s)) return;
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int64_t i = (c0 + u) * (32 * V) + lane * V;
    float v[V];
    Vec<T>::get(raw[u], v);
    int m = 0;  // the largest magnitude as bits: an order that keeps NaN
#pragma unroll
    for (int k = 0; k < V; ++k) m = max(m, __float_as_int(v[k]) & 0x7fffffff);
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    const int e = scale_byte<INT8>(__int_as_float(m));
    const float inv = inverse_of(min(e, 249));
    if (i >= n) continue;
    uint32_t q[V / 4];
#pragma unroll
    for (int k = 0; k < V / 4; ++k) q[k] = e == 255 ? 0u : encode4<INT8>(v + 4 * k, inv);
    if (V == 4) *reinterpret_cast<uint32_t *>(codes + s * n + i) = q[0];
    else *reinterpret_cast<uint2 *>(codes + s * n + i) = make_uint2(q[0], q[V / 4 - 1]);
    if (lane % LANES == 0) scales[s * nb + i / (LANES * V)] = (uint8_t)e;
  }
}

template <typename T, bool INT8>
__global__ void __launch_bounds__(kThreads)
    load_vec_kernel(T *state, int64_t ld, int64_t n, int shift, int64_t nb,
                    const int32_t *slots, int64_t nslots,
                    const uint8_t *codes, const uint8_t *scales) {
  grid_dependency_wait();
  constexpr int V = Vec<T>::V;
  const int64_t b = blockIdx.y;
  const int64_t s = slot_of(slots, b, nslots);
  if (s < 0) return;
  const int64_t c0 = ((int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32) * kU;
  const int lane = threadIdx.x & 31;
  uint32_t q[kU][V / 4];
  int e[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int64_t i = (c0 + u) * (32 * V) + lane * V;
    if (i < n) {
      if (V == 4) {
        q[u][0] = *reinterpret_cast<const uint32_t *>(codes + s * n + i);
      } else {
        const uint2 w = *reinterpret_cast<const uint2 *>(codes + s * n + i);
        q[u][0] = w.x;
        q[u][V / 4 - 1] = w.y;
      }
      e[u] = scales[s * nb + (i >> shift)];
    }
  }
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int64_t i = (c0 + u) * (32 * V) + lane * V;
    if (i >= n) continue;
    float v[V];
#pragma unroll
    for (int k = 0; k < V / 4; ++k) decode4<INT8>(q[u][k], scale_of(e[u]), v + 4 * k);
    __stcs(reinterpret_cast<uint4 *>(state + b * ld + i), Vec<T>::put(v));
  }
}

// Rows anywhere (a row of 327679 values: stores 107 us fp32, 110 us bf16, loads 100 us, with
// the 16-byte lanes of the same sizes at 73, 46 and 67): a lane takes single values, 32 apart, so that a warp's loads and
// stores are of neighbouring ones; a warp has kPer * 32 values (whole blocks) under
// way.
constexpr int kPer = 8;

template <typename T, bool INT8, int PER>  // PER: a block's values in a lane
__global__ void __launch_bounds__(kThreads)
    store_any_kernel(const T *state, int64_t ld, int64_t n, int64_t nb,
                     const int32_t *slots, int64_t batch, int64_t nslots,
                     uint8_t *codes, uint8_t *scales) {
  grid_dependency_wait();
  const int64_t b = blockIdx.y;
  const int lane = threadIdx.x & 31;
  const int64_t i0 =
      ((int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32) * (32 * kPer) + lane;
  const int left = (int)max((int64_t)0, min(n - i0, (int64_t)32 * kPer));  // values from i0 on
  const T *in = state + b * ld + i0;
  float v[kPer];
#pragma unroll
  for (int u = 0; u < kPer; ++u) v[u] = 32 * u < left ? to_f(in[32 * u]) : 0.0f;
  const int64_t s = slot_of(slots, b, nslots);
  if (s < 0 || named_later(slots, b, batch, s)) return;
  uint8_t *out = codes + s * n + i0;
  uint8_t *sc = scales + s * nb + i0 / (32 * PER);
#pragma unroll
  for (int k = 0; k < kPer; k += PER) {
    int m = 0;
#pragma unroll
    for (int u = k; u < k + PER; ++u) m = max(m, __float_as_int(v[u]) & 0x7fffffff);
    const int e = scale_byte<INT8>(__int_as_float(__reduce_max_sync(0xffffffffu, m)));
    const float inv = inverse_of(min(e, 249));
#pragma unroll
    for (int u = k; u < k + PER; ++u)
      if (32 * u < left) out[32 * u] = e == 255 ? 0 : (uint8_t)encode1<INT8>(v[u], inv);
    if (lane == 0 && 32 * k < left) sc[k / PER] = (uint8_t)e;
  }
}

template <typename T, bool INT8>
__global__ void __launch_bounds__(kThreads)
    load_any_kernel(T *state, int64_t ld, int64_t n, int shift, int64_t nb,
                    const int32_t *slots, int64_t nslots,
                    const uint8_t *codes, const uint8_t *scales) {
  grid_dependency_wait();
  const int64_t b = blockIdx.y;
  const int64_t s = slot_of(slots, b, nslots);
  if (s < 0) return;
  const int64_t i0 = ((int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32) * (32 * kPer) +
                     (threadIdx.x & 31);
  const int left = (int)max((int64_t)0, min(n - i0, (int64_t)32 * kPer));
  const uint8_t *in = codes + s * n + i0, *sc = scales + s * nb + (i0 >> shift);
  const int k0 = (int)(i0 & ((1 << shift) - 1));  // i0's place in its block
  T *out = state + b * ld + i0;
  uint8_t q[kPer], e[kPer];
#pragma unroll
  for (int u = 0; u < kPer; ++u)
    if (32 * u < left) {
      q[u] = in[32 * u];
      e[u] = sc[(k0 + 32 * u) >> shift];
    }
#pragma unroll
  for (int u = 0; u < kPer; ++u)
    if (32 * u < left) out[32 * u] = from_f<T>(decode1<INT8>(q[u], scale_of(e[u])));
}

// A launch that is made ready while the kernel before it ends (it waits for that one).
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Whether every row of the state is on a 16-byte boundary and its codes can be
// moved V at a time.
template <typename T> bool on_boundaries(const StateCacheArgs &a) {
  constexpr int V = Vec<T>::V;
  return a.n % V == 0 && (a.batch == 1 || a.ld % V == 0) && aligned(a.state, 16) &&
         aligned(a.codes, V);
}
int log2_of(int v) { return v == 32 ? 5 : v == 64 ? 6 : 7; }

template <typename T, bool INT8> cudaError_t store(const StateCacheArgs &a) {
  constexpr int V = Vec<T>::V;
  const int64_t nb = ceil_div(a.n, a.block);
  const T *state = static_cast<const T *>(a.state);
  uint8_t *codes = static_cast<uint8_t *>(a.codes);
  if (on_boundaries<T>(a)) {
    const dim3 grid((unsigned)ceil_div(a.n, (int64_t)kThreads * V * kU), (unsigned)a.batch);
    const auto kernel = a.block == 32   ? store_vec_kernel<T, INT8, 32 / V>
                        : a.block == 64 ? store_vec_kernel<T, INT8, 64 / V>
                                        : store_vec_kernel<T, INT8, 128 / V>;
    return launch(kernel, grid, a.stream, state, a.ld, a.n, nb, a.slots, a.batch, a.nslots, codes,
                  a.scales);
  } else {
    const dim3 grid((unsigned)ceil_div(a.n, kThreads * kPer), (unsigned)a.batch);
    const auto kernel = a.block == 32   ? store_any_kernel<T, INT8, 1>
                        : a.block == 64 ? store_any_kernel<T, INT8, 2>
                                        : store_any_kernel<T, INT8, 4>;
    return launch(kernel, grid, a.stream, state, a.ld, a.n, nb, a.slots, a.batch, a.nslots, codes,
                  a.scales);
  }
}
template <typename T, bool INT8> cudaError_t load(const StateCacheArgs &a) {
  constexpr int V = Vec<T>::V;
  const int64_t nb = ceil_div(a.n, a.block);
  T *state = static_cast<T *>(a.state);
  const uint8_t *codes = static_cast<const uint8_t *>(a.codes);
  if (on_boundaries<T>(a))
    return launch(load_vec_kernel<T, INT8>,
                  dim3((unsigned)ceil_div(a.n, (int64_t)kThreads * V * kU), (unsigned)a.batch),
                  a.stream, state, a.ld, a.n, log2_of(a.block), nb, a.slots, a.nslots, codes,
                  static_cast<const uint8_t *>(a.scales));
  return launch(load_any_kernel<T, INT8>,
                dim3((unsigned)ceil_div(a.n, kThreads * kPer), (unsigned)a.batch), a.stream, state,
                a.ld, a.n, log2_of(a.block), nb, a.slots, a.nslots, codes,
                static_cast<const uint8_t *>(a.scales));
}

}  // namespace

cudaError_t state_cache_store(const StateCacheArgs &a) {
  if (a.state_dtype == MAMBA2_BF16)
    return a.format == MAMBA2_CODES_INT8 ? store<__nv_bfloat16, true>(a)
                                         : store<__nv_bfloat16, false>(a);
  return a.format == MAMBA2_CODES_INT8 ? store<float, true>(a) : store<float, false>(a);
}
cudaError_t state_cache_load(const StateCacheArgs &a) {
  if (a.state_dtype == MAMBA2_BF16)
    return a.format == MAMBA2_CODES_INT8 ? load<__nv_bfloat16, true>(a)
                                         : load<__nv_bfloat16, false>(a);
  return a.format == MAMBA2_CODES_INT8 ? load<float, true>(a) : load<float, false>(a);
}

cudaError_t take_state_cache_errors(unsigned int *out) {
  unsigned int v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_sc_errors, sizeof(v));
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_sc_errors, &zero, sizeof(zero));
  *out = v;
  return e;
}

}  // namespace m2
