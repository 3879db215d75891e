// Eight consecutive elements (bf16: 16 bytes, fp32: 32 bytes) as floats.
#pragma once

#include "armt_internal.cuh"

namespace armt {

template <typename T>
struct Vec8;

template <>
struct Vec8<bf16> {
  uint4 a;
  __device__ __forceinline__ void load(const bf16* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float* v) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void set(const float* v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b2 = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b2);
    }
    a = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void store(bf16* p) const { *reinterpret_cast<uint4*>(p) = a; }
};

template <>
struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float* v) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  __device__ __forceinline__ void set(const float* v) {
    a = make_float4(v[0], v[1], v[2], v[3]);
    b = make_float4(v[4], v[5], v[6], v[7]);
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
};

// Token id i of an int32 or int64 array.
__device__ __forceinline__ long long load_id(const void* p, int bytes, long long i) {
  return bytes == 8 ? reinterpret_cast<const long long*>(p)[i] : (long long)reinterpret_cast<const int*>(p)[i];
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
// On a multiple of its elements' size (ids; single numbers a row).
inline bool aligned_to(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// Sizes and types that the operators at the ends of the model share.
inline armt_status check_sizes(armt_dtype dtype, int n, int v, int d) {
  if (n < 1 || v < 1 || d < 1) return ARMT_ERR_INVALID_ARG;
  if (dtype != ARMT_BF16 && dtype != ARMT_FP32) return ARMT_ERR_INVALID_ARG;
  // 32-bit row and entry numbers with room for a grid's step
  if (n > (1 << 30) || v > (1 << 30) || d > (1 << 20)) return ARMT_ERR_UNSUPPORTED;
  return d % 8 ? ARMT_ERR_UNSUPPORTED : ARMT_OK;
}

inline armt_status cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return ARMT_OK;
  cudaGetLastError();
  return e == cudaErrorMemoryAllocation ? ARMT_ERR_OOM : ARMT_ERR_CUDA;
}

}  // namespace armt
