// RMSNorm with a gain and its gradient (the norm in front of the head).
//
//   r = (mean x^2 + eps)^-1/2      y = x r g
//   u = dy g      dx = r (u - x r^2 mean(u x))      dg = sum over rows of dy x r
//
// Bound by memory traffic: every element is read once and written once.  W
// warps hold a row in registers (a lane VPL groups of 8 columns, at a stride
// of 256 W columns, so that a warp's access is contiguous).  The gradient's
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

// The gradient's block is one row's W warps.  Few columns a lane (two groups of
// 8 up to 4096 columns) leave room for many blocks, which hide each other's
// latencies; more warps to a row would spend more instructions on the row's
// sums than on its elements.  At 32771 x 2048: one warp to a row 104 us, eight
// 117, four 73 (5.5 TB/s).  Wider rows take four groups a lane and spill 144 to
// 212 bytes a thread; with 2^26 elements, gain included: bf16 81 us up to 4096
// columns, 95 at 8192, 98 at 16384 (4.2 TB/s); fp32 131, 158, 190.
template <typename T, int VPL, int W>
struct NormGrad {
  static constexpr int WARPS_PER_SM = VPL * sizeof(T) <= 4 ? 24 : 16;
  static constexpr int BLOCKS = WARPS_PER_SM / W;
  static constexpr bool AHEAD = VPL * sizeof(T) <= 8;   // the next row is loaded before this one is worked on
};

// part[block][d]: sums of dy x r over the block's rows.
template <typename T, int VPL, int W>
__global__ void __launch_bounds__(32 * W, NormGrad<T, VPL, W>::BLOCKS)
    rms_norm_grad_kernel(const T* x, const T* gain, const float* rstd, const T* dy, T* dx, float* part, int n, int d) {
  constexpr bool AHEAD = NormGrad<T, VPL, W>::AHEAD;
  __shared__ float s[2][W];   // alternating, so that one barrier a row is enough
  const int c0 = threadIdx.x * 8;
  Vec8<T> gv[VPL], xv[VPL], dv[VPL], xn[AHEAD ? VPL : 1], dn[AHEAD ? VPL : 1];
  float2 acc[VPL][4];
  float r = 0.f, rn = 0.f;
#pragma unroll
  for (int k = 0; k < VPL; ++k) {
    const int c = c0 + k * 256 * W;
    gv[k].zero();
    if (c < d) gv[k].load(gain + c);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[k][i] = make_float2(0.f, 0.f);
  }
  auto fetch = [&](int row, Vec8<T>* a, Vec8<T>* b, float& rs) {
#pragma unroll
    for (int k = 0; k < VPL; ++k) {
      const int c = c0 + k * 256 * W;
      a[k].zero();
      b[k].zero();
      if (row < n && c < d) {
        a[k].load(x + (long long)row * d + c);
        b[k].load(dy + (long long)row * d + c);
      }
    }
    rs = row < n ? rstd[row] : 0.f;
  };
  int row = blockIdx.x, turn = 0;
  if constexpr (AHEAD) fetch(row, xn, dn, rn);
  for (; row < n; row += gridDim.x, turn ^= 1) {
    if constexpr (AHEAD) {
#pragma unroll
      for (int k = 0; k < VPL; ++k) {
        xv[k] = xn[k];
        dv[k] = dn[k];
      }
      r = rn;
      fetch(row + (int)gridDim.x, xn, dn, rn);
    } else {
      fetch(row, xv, dv, r);
    }
    float2 ux = make_float2(0.f, 0.f);
    const float2 r2 = make_float2(r, r);
#pragma unroll
    for (int k = 0; k < VPL; ++k) {
      float2 a[4], b[4], g[4];
      xv[k].get(&a[0].x);
      dv[k].get(&b[0].x);
      gv[k].get(&g[0].x);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ux = __ffma2_rn(__fmul2_rn(b[i], g[i]), a[i], ux);
        acc[k][i] = __ffma2_rn(__fmul2_rn(b[i], a[i]), r2, acc[k][i]);
      }
    }
    const float m = -row_sum<W>(ux.x + ux.y, s[turn]) / (float)d * r * r;
    const float2 m2 = make_float2(m, m);
#pragma unroll
    for (int k = 0; k < VPL; ++k) {
      const int c = c0 + k * 256 * W;
      if (c < d) {
        float2 a[4], b[4], g[4];
        xv[k].get(&a[0].x);
        dv[k].get(&b[0].x);
        gv[k].get(&g[0].x);
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = __fmul2_rn(__ffma2_rn(a[i], m2, __fmul2_rn(b[i], g[i])), r2);
        xv[k].set(&a[0].x);
        xv[k].store(dx + (long long)row * d + c);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < VPL; ++k) {
    const int c = c0 + k * 256 * W;
    if (c < d) {
      float4* out = reinterpret_cast<float4*>(part + (long long)blockIdx.x * d + c);
      out[0] = make_float4(acc[k][0].x, acc[k][0].y, acc[k][1].x, acc[k][1].y);
      out[1] = make_float4(acc[k][2].x, acc[k][2].y, acc[k][3].x, acc[k][3].y);
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
#pragma unroll 8
    for (int k = y * per; k < min(parts, (y + 1) * per); ++k) acc += part[(long long)k * d + c];
  }
  s[y][x] = acc;
  __syncthreads();
  if (y == 0 && c < d) {
    for (int g = 1; g < 32; ++g) acc += s[g][x];
    d_gain[c] = (T)acc;
  }
}

constexpr int NORM_WARP_D = 2048;                  // widest row that one warp normalises
constexpr int NORM_MAX_D = 256 * 8 * NORM_WARPS;   // 8 groups a lane, 8 warps a row

// Blocks of the gradient: what one wave of the B200's 148 SMs holds.
template <typename T, int VPL, int W>
int grad_blocks(int n) {
  constexpr int most = 148 * NormGrad<T, VPL, W>::BLOCKS;
  return n < most ? n : most;
}

// By the row's length: two groups of 8 a lane as far as 8 warps reach.
#define ARMT_NORM_GRAD_CASES(F) \
  if (d <= 256) { F(1, 1) } else if (d <= 512) { F(2, 1) } else if (d <= 1024) { F(2, 2) } \
  else if (d <= 2048) { F(2, 4) } else if (d <= 4096) { F(2, 8) } else if (d <= 8192) { F(4, 8) } else { F(4, 16) }

template <typename T>
int grad_parts(int n, int d) {
#define ARMT_F(V, W) return grad_blocks<T, V, W>(n);
  ARMT_NORM_GRAD_CASES(ARMT_F)
#undef ARMT_F
}

template <typename T>
cudaError_t norm(const T* x, const T* gain, T* y, float* rstd, int n, int d, float eps, cudaStream_t st) {
  // one warp to a row: no block-wide sums; above, the block holds a row
  const int grid = d <= NORM_WARP_D ? (n + NORM_WARPS - 1) / NORM_WARPS : n;
#define ARMT_F(V, W) rms_norm_kernel<T, V, W><<<grid, 32 * NORM_WARPS, 0, st>>>(x, gain, y, rstd, n, d, eps);
  if (d <= 256) { ARMT_F(1, 1) }
  else if (d <= 512) { ARMT_F(2, 1) }
  else if (d <= 1024) { ARMT_F(4, 1) }
  else if (d <= NORM_WARP_D) { ARMT_F(8, 1) }
  else if (d <= 4096) { ARMT_F(2, NORM_WARPS) }
  else if (d <= 8192) { ARMT_F(4, NORM_WARPS) }
  else { ARMT_F(8, NORM_WARPS) }
#undef ARMT_F
  return cudaGetLastError();
}

template <typename T>
cudaError_t norm_grad(const T* x, const T* gain, const float* rstd, const T* dy, T* dx, T* d_gain, float* part, int n,
                      int d, cudaStream_t st) {
  const int grid = grad_parts<T>(n, d);
#define ARMT_F(V, W) rms_norm_grad_kernel<T, V, W><<<grid, 32 * W, 0, st>>>(x, gain, rstd, dy, dx, part, n, d);
  ARMT_NORM_GRAD_CASES(ARMT_F)
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
  if (!x || !gain || !y || !(eps >= 0.f) || !std::isfinite(eps) || !aligned16(x) || !aligned16(gain) ||
      !aligned16(y) || !aligned_to(rstd, 4))
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
  *bytes = (size_t)(dtype == ARMT_BF16 ? grad_parts<bf16>(n, d) : grad_parts<float>(n, d)) * d * 4;
  return ARMT_OK;
}

extern "C" armt_status armt_rms_norm_grad(armt_dtype dtype, int n, int d, const void* x, const void* gain,
                                          const float* rstd, const void* dy, void* dx, void* d_gain, void* workspace,
                                          size_t workspace_bytes, void* stream) {
  size_t need = 0;
  const armt_status s = armt_rms_norm_grad_workspace(dtype, n, d, &need);
  if (s != ARMT_OK) return s;
  if (!x || !gain || !rstd || !dy || !dx || !d_gain || !workspace || workspace_bytes < need || !aligned16(x) ||
      !aligned16(gain) || !aligned16(dy) || !aligned16(dx) || !aligned16(workspace) || !aligned_to(rstd, 4) ||
      !aligned_to(d_gain, dtype == ARMT_BF16 ? 2 : 4))
    return ARMT_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == ARMT_BF16)
    return cuda_status(norm_grad<bf16>((const bf16*)x, (const bf16*)gain, rstd, (const bf16*)dy, (bf16*)dx,
                                       (bf16*)d_gain, (float*)workspace, n, d, st));
  return cuda_status(norm_grad<float>((const float*)x, (const float*)gain, rstd, (const float*)dy, (float*)dx,
                                      (float*)d_gain, (float*)workspace, n, d, st));
}
