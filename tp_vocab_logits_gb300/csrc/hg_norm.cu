// Root-mean-square norm of rows with the residual's addition, and its gradient.
//
// One CTA per row, which it reads as often as it needs to (once for the squares,
// once more for the output); a warp takes 128 columns at a time, so that it holds
// the block of an 8-bit scale by itself. Memory bounds both directions.

#include <cuda_fp8.h>

#include "hg_norm.cuh"

namespace hg {
namespace norm {
namespace {

using vocab::Elem;
using vocab::div_up;
using vocab::launch_dependent;
using vocab::let_successor_start;
using vocab::wait_for_predecessor;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr float kE4m3Most = 448.f;
constexpr float kLeastScale = 1.17549435e-38f;  // 2^-126: its reciprocal is finite

template <bool MAX>
__device__ __forceinline__ float combine(float a, float b) {
  return MAX ? fmaxf(a, b) : a + b;
}

// Over the CTA's threads, the same value in each; `red` is free again afterwards.
template <bool MAX>
__device__ float block_all(float v, float* red) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v = combine<MAX>(v, __shfl_xor_sync(0xffffffffu, v, m));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) v = combine<MAX>(v, red[w]);
  __syncthreads();
  return v;
}

__device__ __forceinline__ uint8_t to_e4m3(float v) {
  return (uint8_t)__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
}

// The scale of values up to `most` in magnitude.
__device__ __forceinline__ float scale_of(float most) {
  return most == 0.f ? 1.f : fmaxf(most / kE4m3Most, kLeastScale);
}

struct RowsArgs {
  NormCall c;
  int K;
};

template <typename T>
__global__ void __launch_bounds__(kThreads) rows_kernel(const __grid_constant__ RowsArgs a) {
  __shared__ float red[kWarps];
  wait_for_predecessor();
  let_successor_start();
  const NormCall& c = a.c;
  const size_t n = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const T* x = static_cast<const T*>(c.x.p) + n * c.x.ld;
  const T* res = c.residual.p ? static_cast<const T*>(c.residual.p) + n * c.residual.ld : nullptr;
  T* sum = c.sum.p ? static_cast<T*>(c.sum.p) + n * c.sum.ld : nullptr;
  const T* gain = static_cast<const T*>(c.gain);
  auto added = [&](int k) {
    const float v = Elem<T>::up(x[k]);
    return res ? Elem<T>::down(v + Elem<T>::up(res[k])) : x[k];
  };
  float squares = 0.f;
  for (int b = warp * 128; b < a.K; b += kWarps * 128)
    for (int k = b + lane; k < b + 128 && k < a.K; k += 32) {
      const T s = added(k);
      if (sum) sum[k] = s;
      squares += Elem<T>::up(s) * Elem<T>::up(s);
    }
  const float rstd = rsqrtf(block_all<false>(squares, red) / (float)a.K + c.eps);
  if (c.rstd && threadIdx.x == 0) c.rstd[n] = rstd;
  auto normed = [&](int k) {
    const T s = sum ? sum[k] : added(k);  // this thread's own, where it was written
    return Elem<T>::up(s) * rstd * Elem<T>::up(gain[k]);
  };
  if (!c.e4m3) {
    T* out = static_cast<T*>(c.out.p) + n * c.out.ld;
    for (int b = warp * 128; b < a.K; b += kWarps * 128)
      for (int k = b + lane; k < b + 128 && k < a.K; k += 32) out[k] = Elem<T>::down(normed(k));
    return;
  }
  uint8_t* out = static_cast<uint8_t*>(c.out.p) + n * c.out.ld;
  float scale = 1.f;
  if (c.scale_block == 0) {
    float most = 0.f;
    for (int b = warp * 128; b < a.K; b += kWarps * 128)
      for (int k = b + lane; k < b + 128 && k < a.K; k += 32) most = fmaxf(most, fabsf(normed(k)));
    scale = scale_of(block_all<true>(most, red));
    if (threadIdx.x == 0) c.scales[n] = scale;
  }
  for (int b = warp * 128; b < a.K; b += kWarps * 128) {
    if (c.scale_block != 0) {
      float most = 0.f;
      for (int k = b + lane; k < b + 128 && k < a.K; k += 32) most = fmaxf(most, fabsf(normed(k)));
#pragma unroll
      for (int m = 16; m > 0; m >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, m));
      scale = scale_of(most);
      if (lane == 0) c.scales[n * (size_t)((a.K + 127) / 128) + b / 128] = scale;
    }
    const float inverse = 1.f / scale;
    for (int k = b + lane; k < b + 128 && k < a.K; k += 32) out[k] = to_e4m3(normed(k) * inverse);
  }
}

struct GradArgs {
  GradCall c;
  int K;
  int parts;
  float* partial;
};

// grad_x, a row per CTA.
template <typename T>
__global__ void __launch_bounds__(kThreads) grad_x_kernel(const __grid_constant__ GradArgs a) {
  __shared__ float red[kWarps];
  wait_for_predecessor();
  let_successor_start();
  const GradCall& c = a.c;
  const size_t n = blockIdx.x;
  const T* s = static_cast<const T*>(c.s.p) + n * c.s.ld;
  const T* up = static_cast<const T*>(c.grad_out.p) + n * c.grad_out.ld;
  const T* more = c.grad_sum.p ? static_cast<const T*>(c.grad_sum.p) + n * c.grad_sum.ld : nullptr;
  T* out = static_cast<T*>(c.grad_x.p) + n * c.grad_x.ld;
  const T* gain = static_cast<const T*>(c.gain);
  const float rstd = c.rstd[n];
  float inner = 0.f;
  for (int k = threadIdx.x; k < a.K; k += kThreads)
    inner += Elem<T>::up(up[k]) * Elem<T>::up(gain[k]) * Elem<T>::up(s[k]);
  inner = block_all<false>(inner, red) / (float)a.K * (rstd * rstd * rstd);
  for (int k = threadIdx.x; k < a.K; k += kThreads) {
    float v = rstd * (Elem<T>::up(up[k]) * Elem<T>::up(gain[k])) - Elem<T>::up(s[k]) * inner;
    if (more) v += Elem<T>::up(more[k]);
    out[k] = Elem<T>::down(v);
  }
}

constexpr int kColumns = 32;
constexpr int kSubRows = kThreads / kColumns;

// Sums of grad_gain over every parts-th row from part on, 32 columns per CTA.
template <typename T>
__global__ void __launch_bounds__(kThreads) gain_parts_kernel(const __grid_constant__ GradArgs a) {
  __shared__ float sums[kSubRows][kColumns];
  wait_for_predecessor();
  let_successor_start();
  const GradCall& c = a.c;
  const int columns = (a.K + kColumns - 1) / kColumns;
  const int part = blockIdx.x / columns;
  const int k = (blockIdx.x - part * columns) * kColumns + (threadIdx.x & 31);
  const int sub = threadIdx.x >> 5;
  float v = 0.f;
  if (k < a.K)
    for (size_t n = (size_t)part * kSubRows + sub; n < (size_t)c.N;
         n += (size_t)a.parts * kSubRows)
      v += Elem<T>::up(static_cast<const T*>(c.grad_out.p)[n * c.grad_out.ld + k]) *
           Elem<T>::up(static_cast<const T*>(c.s.p)[n * c.s.ld + k]) * c.rstd[n];
  sums[sub][threadIdx.x & 31] = v;
  __syncthreads();
  if (sub != 0 || k >= a.K) return;
  for (int i = 1; i < kSubRows; ++i) v += sums[i][threadIdx.x];
  a.partial[(size_t)part * a.K + k] = v;
}

// The parts' sums in their order.
template <typename T>
__global__ void __launch_bounds__(kThreads) gain_join_kernel(const __grid_constant__ GradArgs a) {
  wait_for_predecessor();
  let_successor_start();
  const int k = blockIdx.x * kThreads + threadIdx.x;
  if (k >= a.K) return;
  float v = 0.f;
  for (int p = 0; p < a.parts; ++p) v += a.partial[(size_t)p * a.K + k];
  T* out = static_cast<T*>(a.c.grad_gain) + k;
  if (a.c.accumulate) v += Elem<T>::up(*out);
  *out = Elem<T>::down(v);
}

template <typename T>
cudaError_t rows_as(const RowsArgs& a, cudaStream_t stream) {
  return launch_dependent(rows_kernel<T>, a, (unsigned)a.c.N, kThreads, 0, 1, stream);
}

template <typename T>
cudaError_t grad_as(const GradArgs& a, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  if (a.c.grad_gain) {  // first: grad_x may be written over grad_out
    const long long blocks = div_up(a.K, kColumns) * a.parts;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    e = launch_dependent(gain_parts_kernel<T>, a, (unsigned)blocks, kThreads, 0, 1, stream);
    if (e == cudaSuccess)
      e = launch_dependent(gain_join_kernel<T>, a, (unsigned)div_up(a.K, kThreads), kThreads, 0, 1,
                           stream);
  }
  if (e != cudaSuccess || !a.c.grad_x.p || a.c.N == 0) return e;
  return launch_dependent(grad_x_kernel<T>, a, (unsigned)a.c.N, kThreads, 0, 1, stream);
}

}  // namespace

int grad_parts(const hg_norm& h, int N) {
  const long long parts = div_up(N, kSubRows);
  return parts < 1 ? 1 : parts < 2 * h.sms ? (int)parts : 2 * h.sms;
}

cudaError_t rows(const hg_norm& h, const NormCall& c, cudaStream_t stream) {
  RowsArgs a = {c, h.K};
  switch (h.dtype) {
    case HG_BF16:
      return rows_as<__nv_bfloat16>(a, stream);
    case HG_FP16:
      return rows_as<__half>(a, stream);
    default:
      return rows_as<float>(a, stream);
  }
}

cudaError_t rows_grad(const hg_norm& h, const GradCall& c, cudaStream_t stream) {
  GradArgs a = {c, h.K, grad_parts(h, c.N), h.partial};
  switch (h.dtype) {
    case HG_BF16:
      return grad_as<__nv_bfloat16>(a, stream);
    case HG_FP16:
      return grad_as<__half>(a, stream);
    default:
      return grad_as<float>(a, stream);
  }
}

}  // namespace norm
}  // namespace hg
