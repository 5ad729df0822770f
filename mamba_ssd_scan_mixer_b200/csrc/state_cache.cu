// The 8-bit state cache: recurrent states written into slots as codes of 8 bits
// with a power-of-two scale for each block of consecutive values, and read back.
//
// The scale 2^e of a block is the least power of two with amax <= qmax 2^e
// (qmax = 127 for int8, 448 for e4m3), kept as the biased exponent byte e + 127.
// A power of two makes v 2^-e exact, so the only rounding is the code's own (to
// nearest, ties to even), and a state that was read back and is written again
// gives the same values.
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
template <bool INT8> __device__ __forceinline__ uint8_t encode(float v) {
  if (INT8) return (uint8_t)(int8_t)__float2int_rn(v);
  return (uint8_t)__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
}
template <bool INT8> __device__ __forceinline__ float decode(uint8_t q) {
  if (INT8) return (float)(int8_t)q;
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(q, __NV_E4M3)));
}

// The slot of batch row b, or -1 if nothing is to be done for it: a negative
// slot, one out of range (flagged), or (store) one that a later row names too.
__device__ __forceinline__ int64_t slot_of(const int32_t *slots, int64_t b, int64_t nslots) {
  const int64_t s = slots[b];
  if (s >= nslots) {
    atomicOr(&g_sc_errors, kErrSlots);
    return -1;
  }
  return s < 0 ? -1 : s;
}

template <typename T, bool INT8>
__global__ void store_kernel(const T *state, int64_t ld, int64_t n, int block, int64_t nb,
                             const int32_t *slots, int64_t batch, int64_t nslots, uint8_t *codes,
                             uint8_t *scales) {
  const int64_t b = blockIdx.y;
  const int64_t s = slot_of(slots, b, nslots);
  if (s < 0) return;
  int later = 0;
  for (int64_t i = b + 1 + threadIdx.x; i < batch; i += blockDim.x) later |= slots[i] == s;
  if (__syncthreads_or(later)) return;
  const int64_t k = (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;
  const int lane = threadIdx.x & 31;
  if (k >= nb) return;
  const int64_t i0 = k * block, i1 = min(n, i0 + block);
  int m = 0;  // the largest magnitude as bits: an order that keeps NaN
  for (int64_t i = i0 + lane; i < i1; i += 32)
    m = max(m, __float_as_int(to_f(state[b * ld + i])) & 0x7fffffff);
  m = __reduce_max_sync(0xffffffffu, m);
  const int e = scale_byte<INT8>(__int_as_float(m));
  for (int64_t i = i0 + lane; i < i1; i += 32)
    codes[s * n + i] = e == 255 ? 0 : encode<INT8>(to_f(state[b * ld + i]) * inverse_of(e));
  if (lane == 0) scales[s * nb + k] = (uint8_t)e;
}

template <typename T, bool INT8>
__global__ void load_kernel(T *state, int64_t ld, int64_t n, int block, int64_t nb,
                            const int32_t *slots, int64_t nslots, const uint8_t *codes,
                            const uint8_t *scales) {
  const int64_t b = blockIdx.y;
  const int64_t s = slot_of(slots, b, nslots);
  if (s < 0) return;
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= n) return;
  const int e = scales[s * nb + i / block];
  const float v = e == 255 ? __int_as_float(0x7fffffff) : decode<INT8>(codes[s * n + i]) * pow2_of(e);
  state[b * ld + i] = from_f<T>(v);
}

template <typename T, bool INT8> cudaError_t store(const StateCacheArgs &a) {
  const int64_t nb = ceil_div(a.n, a.block);
  store_kernel<T, INT8><<<dim3((unsigned)ceil_div(nb, 8), (unsigned)a.batch), 256, 0, a.stream>>>(
      static_cast<const T *>(a.state), a.ld, a.n, a.block, nb, a.slots, a.batch, a.nslots,
      static_cast<uint8_t *>(a.codes), a.scales);
  return cudaGetLastError();
}
template <typename T, bool INT8> cudaError_t load(const StateCacheArgs &a) {
  const int64_t nb = ceil_div(a.n, a.block);
  load_kernel<T, INT8><<<dim3((unsigned)ceil_div(a.n, 256), (unsigned)a.batch), 256, 0, a.stream>>>(
      static_cast<T *>(a.state), a.ld, a.n, a.block, nb, a.slots, a.nslots,
      static_cast<const uint8_t *>(a.codes), a.scales);
  return cudaGetLastError();
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
