// RMSNorm with a gain and its gradient (the norm in front of the head).
//
//   r = (mean x^2 + eps)^-1/2      y = x r g
//   u = dy g      dx = r (u - x r^2 mean(u x))      dg = sum over rows of dy x r
//
// Bound by memory traffic: every element is read once and written once.  W
// warps hold a row in registers (a lane VPL groups of 8 columns, at a stride
// of 256 W columns so that a warp's access is contiguous).  The gradient's
// blocks walk over the rows with the gain's sums in registers, one partial sum
// per block, joined in order by a second kernel.
#include <cmath>

#include "armt_internal.cuh"
#include "vec8.cuh"

namespace armt {

namespace {

constexpr int NORM_WARPS = 8;

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Sum over the row's W warps (all of the block's when W > 1).
template <int W>
__device__ __forceinline__ float row_sum(float x, float* s) {
  x = warp_sum(x);
  if constexpr (W > 1) {
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = x;
    __syncthreads();
    x = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) x += s[w];
  }
  return x;
}

template <typename T, int VPL, int W>
__global__ void __launch_bounds__(32 * NORM_WARPS) rms_norm_kernel(const T* x, const T* gain, T* y, float* rstd, int n,
                                                                   int d, float eps) {
  __shared__ float s[NORM_WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = W == 1 ? blockIdx.x * NORM_WARPS + warp : blockIdx.x;
  const int c0 = ((W == 1 ? 0 : warp * 32) + lane) * 8;
  const bool in = row < n;
  Vec8<T> v[VPL];
  float ss = 0.f;
#pragma unroll
  for (int k = 0; k < VPL; ++k) {
    const int c = c0 + k * 256 * W;
    v[k].zero();
    if (in && c < d) v[k].load(x + (long long)row * d + c);
  }
#pragma unroll
  for (int k = 0; k < VPL; ++k) {
    float f[8];
    v[k].get(f);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
  }
  const float r = rsqrtf(row_sum<W>(ss, s) / (float)d + eps);
  if (!in) return;
  if (rstd && c0 == 0) rstd[row] = r;
#pragma unroll
  for (int k = 0; k < VPL; ++k) {
    const int c = c0 + k * 256 * W;
    if (c < d) {
      Vec8<T> gv;
      gv.load(gain + c);
      float f[8], g[8];
      v[k].get(f);
      gv.get(g);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = f[i] * r * g[i];
      v[k].set(f);
      v[k].store(y + (long long)row * d + c);
    }
  }
}

// part[block][d]: sums of dy x r over the block's rows.
template <typename T, int VPL, int W>
__global__ void __launch_bounds__(32 * NORM_WARPS) rms_norm_grad_kernel(const T* x, const T* gain, const float* rstd,
                                                                        const T* dy, T* dx, float* part, int n,
                                                                        int d) {
  extern __shared__ float sums[];   // W == 1: [d], the warps' sums joined one warp after another
  __shared__ float s[NORM_WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c0 = ((W == 1 ? 0 : warp * 32) + lane) * 8;
  float acc[VPL][8];
#pragma unroll
  for (int k = 0; k < VPL; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[k][i] = 0.f;
  const int step = W == 1 ? gridDim.x * NORM_WARPS : gridDim.x;
  for (int row = W == 1 ? blockIdx.x * NORM_WARPS + warp : blockIdx.x; row < n; row += step) {
    Vec8<T> xv[VPL], dv[VPL];
#pragma unroll
    for (int k = 0; k < VPL; ++k) {
      const int c = c0 + k * 256 * W;
      xv[k].zero();
      dv[k].zero();
      if (c < d) {
        xv[k].load(x + (long long)row * d + c);
        dv[k].load(dy + (long long)row * d + c);
      }
    }
    const float r = rstd[row];
    float ux = 0.f;
#pragma unroll
    for (int k = 0; k < VPL; ++k) {
      const int c = c0 + k * 256 * W;
      if (c < d) {
        Vec8<T> gv;
        gv.load(gain + c);
        float a[8], b[8], g[8];
        xv[k].get(a);
        dv[k].get(b);
        gv.get(g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ux = fmaf(b[i] * g[i], a[i], ux);
          acc[k][i] = fmaf(b[i] * a[i], r, acc[k][i]);
        }
      }
    }
    const float m = row_sum<W>(ux, s) / (float)d * r * r;
#pragma unroll
    for (int k = 0; k < VPL; ++k) {
      const int c = c0 + k * 256 * W;
      if (c < d) {
        Vec8<T> gv;
        gv.load(gain + c);
        float a[8], b[8], g[8];
        xv[k].get(a);
        dv[k].get(b);
        gv.get(g);
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = r * (b[i] * g[i] - a[i] * m);
        xv[k].set(a);
        xv[k].store(dx + (long long)row * d + c);
      }
    }
  }
  float* out = part + (long long)blockIdx.x * d;
  if constexpr (W == 1) {
    for (int w = 0; w < NORM_WARPS; ++w) {
      if (warp == w) {
#pragma unroll
        for (int k = 0; k < VPL; ++k) {
          const int c = c0 + k * 256;
          if (c < d) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int at = i * (d / 8) + c / 8;   // lanes on consecutive words
              sums[at] = (w ? sums[at] : 0.f) + acc[k][i];
            }
          }
        }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < d; c += 32 * NORM_WARPS) out[c] = sums[(c & 7) * (d / 8) + c / 8];
  } else {
#pragma unroll
    for (int k = 0; k < VPL; ++k) {
      const int c = c0 + k * 256 * W;
      if (c < d) {
#pragma unroll
        for (int i = 0; i < 8; ++i) out[c + i] = acc[k][i];
      }
    }
  }
}

// d_gain: 32 columns a block, 32 groups of partial sums side by side.
template <typename T>
__global__ void __launch_bounds__(1024) rms_norm_gain_kernel(const float* part, int parts, int d, T* d_gain) {
  __shared__ float s[32][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5, c = blockIdx.x * 32 + x;
  const int per = (parts + 31) / 32;
  float acc = 0.f;
  if (c < d) {
#pragma unroll 4
    for (int k = y * per; k < min(parts, (y + 1) * per); ++k) acc += part[(long long)k * d + c];
  }
  s[y][x] = acc;
  __syncthreads();
  if (y == 0 && c < d) {
    for (int g = 1; g < 32; ++g) acc += s[g][x];
    d_gain[c] = (T)acc;
  }
}

constexpr int NORM_WARP_D = 2048;                  // widest row of one warp
constexpr int NORM_MAX_D = 256 * 8 * NORM_WARPS;   // 8 groups a lane, 8 warps a row

int grad_blocks(int n, int d) {
  const int rows = d <= NORM_WARP_D ? NORM_WARPS : 1;   // per block and step
  const int want = (n + rows - 1) / rows;
  return want < 2 * 148 ? want : 2 * 148;
}

// W = 1 up to 2048 columns: no block-wide sums; above, the block holds a row
// (16 groups a lane would spill the gradient's registers).
#define ARMT_NORM_CASES(F) \
  if (d <= 256) { F(1, 1) } else if (d <= 512) { F(2, 1) } else if (d <= 1024) { F(4, 1) } \
  else if (d <= NORM_WARP_D) { F(8, 1) } else if (d <= 4096) { F(2, NORM_WARPS) } \
  else if (d <= 8192) { F(4, NORM_WARPS) } else { F(8, NORM_WARPS) }

template <typename T>
cudaError_t norm(const T* x, const T* gain, T* y, float* rstd, int n, int d, float eps, cudaStream_t st) {
  const int grid = d <= NORM_WARP_D ? (n + NORM_WARPS - 1) / NORM_WARPS : n;
#define ARMT_F(V, W) rms_norm_kernel<T, V, W><<<grid, 32 * NORM_WARPS, 0, st>>>(x, gain, y, rstd, n, d, eps);
  ARMT_NORM_CASES(ARMT_F)
#undef ARMT_F
  return cudaGetLastError();
}

template <typename T>
cudaError_t norm_grad(const T* x, const T* gain, const float* rstd, const T* dy, T* dx, T* d_gain, float* part, int n,
                      int d, cudaStream_t st) {
  const int grid = grad_blocks(n, d);
  const size_t smem = d <= NORM_WARP_D ? (size_t)d * 4 : 0;
#define ARMT_F(V, W) \
  rms_norm_grad_kernel<T, V, W><<<grid, 32 * NORM_WARPS, smem, st>>>(x, gain, rstd, dy, dx, part, n, d);
  ARMT_NORM_CASES(ARMT_F)
#undef ARMT_F
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  rms_norm_gain_kernel<T><<<(d + 31) / 32, 1024, 0, st>>>(part, grid, d, d_gain);
  return cudaGetLastError();
}

armt_status check_norm(armt_dtype dtype, int n, int d) {
  const armt_status s = check_sizes(dtype, n, 1, d);
  if (s != ARMT_OK) return s;
  return d > NORM_MAX_D ? ARMT_ERR_UNSUPPORTED : ARMT_OK;
}

}  // namespace

}  // namespace armt

using namespace armt;

extern "C" armt_status armt_rms_norm(armt_dtype dtype, int n, int d, const void* x, const void* gain, float eps,
                                     void* y, float* rstd, void* stream) {
  const armt_status s = check_norm(dtype, n, d);
  if (s != ARMT_OK) return s;
  if (!x || !gain || !y || !(eps >= 0.f) || !std::isfinite(eps) || !aligned16(x) || !aligned16(gain) || !aligned16(y))
    return ARMT_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == ARMT_BF16) return cuda_status(norm<bf16>((const bf16*)x, (const bf16*)gain, (bf16*)y, rstd, n, d, eps, st));
  return cuda_status(norm<float>((const float*)x, (const float*)gain, (float*)y, rstd, n, d, eps, st));
}

extern "C" armt_status armt_rms_norm_grad_workspace(armt_dtype dtype, int n, int d, size_t* bytes) {
  if (!bytes) return ARMT_ERR_INVALID_ARG;
  *bytes = 0;
  const armt_status s = check_norm(dtype, n, d);
  if (s != ARMT_OK) return s;
  *bytes = (size_t)grad_blocks(n, d) * d * 4;
  return ARMT_OK;
}

extern "C" armt_status armt_rms_norm_grad(armt_dtype dtype, int n, int d, const void* x, const void* gain,
                                          const float* rstd, const void* dy, void* dx, void* d_gain, void* workspace,
                                          size_t workspace_bytes, void* stream) {
  size_t need = 0;
  const armt_status s = armt_rms_norm_grad_workspace(dtype, n, d, &need);
  if (s != ARMT_OK) return s;
  if (!x || !gain || !rstd || !dy || !dx || !d_gain || !workspace || workspace_bytes < need || !aligned16(x) ||
      !aligned16(gain) || !aligned16(dy) || !aligned16(dx) || !aligned16(workspace))
    return ARMT_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == ARMT_BF16)
    return cuda_status(norm_grad<bf16>((const bf16*)x, (const bf16*)gain, rstd, (const bf16*)dy, (bf16*)dx,
                                       (bf16*)d_gain, (float*)workspace, n, d, st));
  return cuda_status(norm_grad<float>((const float*)x, (const float*)gain, rstd, (const float*)dy, (float*)dx,
                                      (float*)d_gain, (float*)workspace, n, d, st));
}
