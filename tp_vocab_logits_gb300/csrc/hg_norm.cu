// Root-mean-square norm of rows with the residual's addition, and its gradient.
//
// Memory bounds both directions, so a row is read once: its threads hold it in
// registers, packed as it came, between the sum over the row and the output. A CTA takes
// one row, or several where they are short, with A accesses of E elements a thread.
// Rows that are longer than a CTA's registers hold are read twice.

#include <cuda_fp8.h>

#include "hg_norm.cuh"

namespace hg {
namespace norm {
namespace {

using vocab::Elem;
using vocab::Pack;
using vocab::div_up;
using vocab::launch_dependent;
using vocab::let_successor_start;
using vocab::round_up;
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

// How a launch lays rows on threads.
struct Shape {
  int threads;  // of a row: whole warps
  int rows;     // of a CTA
};

// Over a row's threads, the same value in each. `red` holds a word per warp of the CTA, and is
// free again after the next barrier of it.
template <bool MAX>
__device__ __forceinline__ float row_all(float v, float* red, int warps) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v = combine<MAX>(v, __shfl_xor_sync(0xffffffffu, v, m));
  if (warps == 1) return v;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) red[warp] = v;
  __syncthreads();
  v = lane < warps ? red[warp - warp % warps + lane] : 0.f;
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v = combine<MAX>(v, __shfl_xor_sync(0xffffffffu, v, m));
  return v;
}

template <typename T, int E, int A>
__device__ __forceinline__ void load_row(Pack<T, E> (&to)[A], const Rows& m, size_t n, int first,
                                         int step, int accesses) {
  const Pack<T, E>* p = reinterpret_cast<const Pack<T, E>*>(static_cast<const T*>(m.p) + n * m.ld);
#pragma unroll
  for (int j = 0; j < A; ++j)
    if (first + j * step < accesses) to[j] = p[first + j * step];
}

template <typename T, int E, int A>
__device__ __forceinline__ void clear_row(Pack<T, E> (&to)[A]) {
#pragma unroll
  for (int j = 0; j < A; ++j)
#pragma unroll
    for (int e = 0; e < E; ++e) to[j].v[e] = Elem<T>::down(0.f);
}

template <typename T, int E, int A>
__device__ __forceinline__ void store_row(const Pack<T, E> (&from)[A], const RowsOut& m, size_t n,
                                          int first, int step, int accesses) {
  Pack<T, E>* p = reinterpret_cast<Pack<T, E>*>(static_cast<T*>(m.p) + n * m.ld);
#pragma unroll
  for (int j = 0; j < A; ++j)
    if (first + j * step < accesses) p[first + j * step] = from[j];
}

struct RowsArgs {
  NormCall c;
  int K;
  Shape shape;
};

// Most threads of a row: what leaves the widest accesses' registers unspilled.
template <int A, int BYTES>
constexpr int most_threads() {
  return A * BYTES >= 64 ? 512 : 1024;
}

// 8-bit output of a row whose elements are y(j, e).
template <int E, int A, typename Y>
__device__ __forceinline__ void store_e4m3(const RowsArgs& a, size_t n, bool there, int first,
                                           float* red, Y y) {
  const NormCall& c = a.c;
  const int step = a.shape.threads, accesses = a.K / E;
  uint8_t* out = static_cast<uint8_t*>(c.out.p) + n * c.out.ld;
  float most[A];
#pragma unroll
  for (int j = 0; j < A; ++j) {
    most[j] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) most[j] = fmaxf(most[j], fabsf(y(j, e)));
  }
  if (c.scale_block == 0) {
#pragma unroll
    for (int j = 1; j < A; ++j) most[0] = fmaxf(most[0], most[j]);
    const float scale = scale_of(row_all<true>(most[0], red, step / 32));
    if (there && first == 0) c.scales[n] = scale;
#pragma unroll
    for (int j = 0; j < A; ++j) most[j] = scale;
  } else {
    // The lanes that hold a block of 128 columns: 128 / E neighbours, or whole warps.
    constexpr int kLanes = 128 / E < 32 ? 128 / E : 32;
    const size_t blocks = (size_t)((a.K + 127) / 128);
#pragma unroll
    for (int j = 0; j < A; ++j)
#pragma unroll
      for (int m = kLanes / 2; m > 0; m >>= 1)
        most[j] = fmaxf(most[j], __shfl_xor_sync(0xffffffffu, most[j], m));
    if constexpr (128 / E > 32) {
      __shared__ unsigned joined[1024 * A * E / 128];  // magnitudes order as their bits do
      for (int b = threadIdx.x; b < a.shape.rows * (int)blocks; b += blockDim.x) joined[b] = 0;
      __syncthreads();
      const int block0 = threadIdx.x / step * (int)blocks;
#pragma unroll
      for (int j = 0; j < A; ++j)
        if ((threadIdx.x & 31) == 0 && first + j * step < accesses)
          atomicMax(&joined[block0 + (first + j * step) / (128 / E)], __float_as_uint(most[j]));
      __syncthreads();
#pragma unroll
      for (int j = 0; j < A; ++j)
        if (first + j * step < accesses)
          most[j] = __uint_as_float(joined[block0 + (first + j * step) / (128 / E)]);
    }
#pragma unroll
    for (int j = 0; j < A; ++j) {
      const int i = first + j * step;
      most[j] = scale_of(most[j]);
      if (there && i < accesses && i % (128 / E) == 0) c.scales[n * blocks + i / (128 / E)] = most[j];
    }
  }
  if (!there) return;
#pragma unroll
  for (int j = 0; j < A; ++j) {
    const float inverse = 1.f / most[j];
    Pack<uint8_t, E> q;
#pragma unroll
    for (int e = 0; e < E; ++e) q.v[e] = to_e4m3(y(j, e) * inverse);
    if (first + j * step < accesses) reinterpret_cast<Pack<uint8_t, E>*>(out)[first + j * step] = q;
  }
}

template <typename T, int E, int A, bool QUANT>
__global__ void __launch_bounds__((most_threads<A, E * (int)sizeof(T)>()))
    rows_kernel(const __grid_constant__ RowsArgs a) {
  __shared__ float red[2][32];
  wait_for_predecessor();
  let_successor_start();
  const NormCall& c = a.c;
  const int step = a.shape.threads, sub = threadIdx.x / step, first = threadIdx.x - sub * step;
  const int accesses = a.K / E;
  const size_t n = (size_t)blockIdx.x * a.shape.rows + sub;
  const bool there = n < (size_t)c.N;
  Pack<T, E> s[A], g[A];
  clear_row(s);
  clear_row(g);
  if (there) {
    load_row(s, c.x, n, first, step, accesses);
    if (c.residual.p) {
      load_row(g, c.residual, n, first, step, accesses);
#pragma unroll
      for (int j = 0; j < A; ++j)
#pragma unroll
        for (int e = 0; e < E; ++e)
          s[j].v[e] = Elem<T>::down(Elem<T>::up(s[j].v[e]) + Elem<T>::up(g[j].v[e]));
    }
    load_row(g, Rows{c.gain, 0}, 0, first, step, accesses);
    if (c.sum.p) store_row(s, c.sum, n, first, step, accesses);
  }
  float squares = 0.f;
#pragma unroll
  for (int j = 0; j < A; ++j)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float v = Elem<T>::up(s[j].v[e]);
      squares += v * v;
    }
  const float rstd =
      rsqrtf(row_all<false>(squares, red[0], step / 32) / (float)a.K + c.eps);
  if (there && c.rstd && first == 0) c.rstd[n] = rstd;
  auto y = [&](int j, int e) {
    return Elem<T>::up(s[j].v[e]) * rstd * Elem<T>::up(g[j].v[e]);
  };
  if constexpr (QUANT) {
    store_e4m3<E, A>(a, n, there, first, red[1], y);
  } else if (there) {
#pragma unroll
    for (int j = 0; j < A; ++j)
#pragma unroll
      for (int e = 0; e < E; ++e) s[j].v[e] = Elem<T>::down(y(j, e));
    store_row(s, c.out, n, first, step, accesses);
  }
}

// Rows of any length: read again for the output (and once more for a row's scale), a warp
// taking 128 columns at a time, so that it holds the block of a scale by itself.
template <typename T>
__global__ void __launch_bounds__(kThreads) long_rows_kernel(const __grid_constant__ RowsArgs a) {
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
  Shape shape;
  int parts;
  float* partial;
};

// Both gradients in one pass: a CTA takes every parts-th row (or group of short rows),
// holds it in registers between the inner sum and grad_x, and adds what its columns give
// to grad_gain up in registers over all its rows.
template <typename T, int E, int A, int THREADS, bool GAIN>
__global__ void __launch_bounds__(THREADS)
    grad_kernel(const __grid_constant__ GradArgs a) {
  __shared__ float red[2][32];
  wait_for_predecessor();
  let_successor_start();
  const GradCall& c = a.c;
  const int step = a.shape.threads, sub = threadIdx.x / step, first = threadIdx.x - sub * step;
  const int accesses = a.K / E;
  Pack<T, E> g[A], s[A], up[A], more[A];
  clear_row(g);
  clear_row(s);
  clear_row(up);
  clear_row(more);
  load_row(g, Rows{c.gain, 0}, 0, first, step, accesses);
  float acc[A][E] = {};
  int turn = 0;
  for (size_t n0 = (size_t)blockIdx.x * a.shape.rows; n0 < (size_t)c.N;
       n0 += (size_t)a.parts * a.shape.rows) {
    const size_t n = n0 + sub;
    const bool there = n < (size_t)c.N;
    float rstd = 0.f;
    if (there) {
      load_row(s, c.s, n, first, step, accesses);
      load_row(up, c.grad_out, n, first, step, accesses);
      if (c.grad_sum.p) load_row(more, c.grad_sum, n, first, step, accesses);
      rstd = c.rstd[n];
    }
    if (c.grad_x.p) {
      float inner = 0.f;
#pragma unroll
      for (int j = 0; j < A; ++j)
#pragma unroll
        for (int e = 0; e < E; ++e)
          inner += Elem<T>::up(up[j].v[e]) * Elem<T>::up(g[j].v[e]) * Elem<T>::up(s[j].v[e]);
      inner = row_all<false>(inner, red[turn], step / 32) / (float)a.K * (rstd * rstd * rstd);
      turn ^= 1;
#pragma unroll
      for (int j = 0; j < A; ++j)
#pragma unroll
        for (int e = 0; e < E; ++e)
          more[j].v[e] = Elem<T>::down(rstd * (Elem<T>::up(up[j].v[e]) * Elem<T>::up(g[j].v[e])) -
                                       Elem<T>::up(s[j].v[e]) * inner + Elem<T>::up(more[j].v[e]));
      if (there) store_row(more, c.grad_x, n, first, step, accesses);
      if (!c.grad_sum.p) clear_row(more);
    }
    if (GAIN && there) {
#pragma unroll
      for (int j = 0; j < A; ++j)
#pragma unroll
        for (int e = 0; e < E; ++e)
          acc[j][e] += Elem<T>::up(up[j].v[e]) * Elem<T>::up(s[j].v[e]) * rstd;
    }
  }
  if (!GAIN) return;
  float* partial = a.partial + (size_t)blockIdx.x * a.K;
  if (a.shape.rows == 1) {
#pragma unroll
    for (int j = 0; j < A; ++j)
      if (first + j * step < accesses) {
        float* to = partial + (size_t)(first + j * step) * E;
#pragma unroll
        for (int e = 0; e < E; e += 4)
          if constexpr (E >= 4)
            *reinterpret_cast<float4*>(to + e) =
                make_float4(acc[j][e], acc[j][e + 1], acc[j][e + 2], acc[j][e + 3]);
          else if constexpr (E == 2)
            *reinterpret_cast<float2*>(to) = make_float2(acc[j][0], acc[j][1]);
          else
            *to = acc[j][0];
      }
    return;
  }
  // Short rows: the CTA's groups in their order. Fewer than 128 threads hold a row.
  __shared__ float sums[128 * A * E];
#pragma unroll
  for (int j = 0; j < A; ++j)
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (first + j * step < accesses) sums[sub * a.K + (first + j * step) * E + e] = acc[j][e];
  __syncthreads();
  for (int k = threadIdx.x; k < a.K; k += blockDim.x) {
    float v = sums[k];
    for (int r = 1; r < a.shape.rows; ++r) v += sums[r * a.K + k];
    partial[k] = v;
  }
}

// Rows of any length, read twice for grad_x and once more for the sums of grad_gain.

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

constexpr int kJoinSubs = 32;

// The parts' sums: each of 32 warps adds up every 32nd part, in order, and one thread a
// column the warps' sums.
template <typename T>
__global__ void __launch_bounds__(32 * kJoinSubs)
    gain_join_kernel(const __grid_constant__ GradArgs a) {
  __shared__ float sums[kJoinSubs][33];
  wait_for_predecessor();
  let_successor_start();
  const int lane = threadIdx.x & 31, sub = threadIdx.x >> 5;
  const int k = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (k < a.K)
#pragma unroll 4
    for (int p = sub; p < a.parts; p += kJoinSubs) v += a.partial[(size_t)p * a.K + k];
  sums[lane][sub] = v;
  __syncthreads();
  v = sums[sub][lane];  // column sub, warp lane
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  const int column = blockIdx.x * 32 + sub;
  if (lane != 0 || column >= a.K) return;
  T* out = static_cast<T*>(a.c.grad_gain) + column;
  if (a.c.accumulate) v += Elem<T>::up(*out);
  *out = Elem<T>::down(v);
}

template <typename T, int E, int A>
cudaError_t rows_as(const hg_norm& h, RowsArgs& a, cudaStream_t stream) {
  a.shape.threads = (int)round_up(div_up(a.K / E, A), 32);
  a.shape.rows = a.shape.threads < 128 ? 128 / a.shape.threads : 1;
  const unsigned grid = (unsigned)div_up(a.c.N, a.shape.rows);
  const unsigned block = (unsigned)(a.shape.threads * a.shape.rows);
  return a.c.e4m3 ? launch_dependent(rows_kernel<T, E, A, true>, a, grid, block, 0, 1, stream)
                  : launch_dependent(rows_kernel<T, E, A, false>, a, grid, block, 0, 1, stream);
}

// A accesses a thread: as few as the row allows where rows are few and their latency
// counts, else LONG of them, so that several rows' loads are under way on an SM.
template <typename T, int E, int LONG>
cudaError_t rows_by(const hg_norm& h, RowsArgs& a, cudaStream_t stream) {
  const int accesses = a.K / E;
  if (accesses > LONG * most_threads<LONG, E * (int)sizeof(T)>())
    return launch_dependent(long_rows_kernel<T>, a, (unsigned)a.c.N, kThreads, 0, 1, stream);
  if (a.c.N <= h.sms && accesses <= 1024) return rows_as<T, E, 1>(h, a, stream);
  return rows_as<T, E, LONG>(h, a, stream);
}

template <typename T>
cudaError_t join_gain(const GradArgs& a, cudaStream_t stream) {
  return launch_dependent(gain_join_kernel<T>, a, (unsigned)div_up(a.K, 32), 32 * kJoinSubs, 0, 1,
                          stream);
}

template <typename T>
cudaError_t grad_of_long_rows(GradArgs& a, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  if (a.c.grad_gain) {  // first: grad_x may be written over grad_out
    const long long blocks = div_up(a.K, kColumns) * a.parts;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    e = launch_dependent(gain_parts_kernel<T>, a, (unsigned)blocks, kThreads, 0, 1, stream);
    if (e == cudaSuccess) e = join_gain<T>(a, stream);
  }
  if (e != cudaSuccess || !a.c.grad_x.p || a.c.N == 0) return e;
  return launch_dependent(grad_x_kernel<T>, a, (unsigned)a.c.N, kThreads, 0, 1, stream);
}

template <typename T, int E, int A, int THREADS>
cudaError_t grad_as(const hg_norm& h, GradArgs& a, cudaStream_t stream) {
  a.shape.threads = (int)round_up(div_up(a.K / E, A), 32);
  a.shape.rows = a.shape.threads < 128 ? 128 / a.shape.threads : 1;
  const unsigned block = (unsigned)(a.shape.threads * a.shape.rows);
  const long long groups = div_up(a.c.N, a.shape.rows);
  const int most = grad_parts(h);
  a.parts = groups < 1 ? 1 : groups < most ? (int)groups : most;
  const unsigned grid = (unsigned)a.parts;
  if (!a.c.grad_gain)
    return launch_dependent(grad_kernel<T, E, A, THREADS, false>, a, grid, block, 0, 1, stream);
  const cudaError_t e =
      launch_dependent(grad_kernel<T, E, A, THREADS, true>, a, grid, block, 0, 1, stream);
  return e == cudaSuccess ? join_gain<T>(a, stream) : e;
}

// As few accesses a thread as the row allows where rows are few, else A of them, or
// twice that, whichever THREADS hold the row.
template <typename T, int E, int A, int THREADS>
cudaError_t grad_by(const hg_norm& h, GradArgs& a, cudaStream_t stream) {
  const int accesses = a.K / E;
  if (a.c.N <= h.sms && accesses <= 1024) return grad_as<T, E, 1, 1024>(h, a, stream);
  if (accesses <= A * THREADS) return grad_as<T, E, A, THREADS>(h, a, stream);
  if (accesses <= 2 * A * THREADS) return grad_as<T, E, 2 * A, THREADS>(h, a, stream);
  const long long parts = div_up(a.c.N, kSubRows);
  const int most = grad_parts(h);
  a.parts = parts < 1 ? 1 : parts < most ? (int)parts : most;
  return grad_of_long_rows<T>(a, stream);
}

}  // namespace

int grad_parts(const hg_norm& h) {
  const long long most = (long long)h.sms * (h.K <= 2048 ? 8 : h.K <= 4096 ? 4 : 2);
  return h.max_rows < most ? h.max_rows : (int)most;
}

template <typename T>
cudaError_t rows_of(const hg_norm& h, RowsArgs& a, cudaStream_t stream) {
  const NormCall& c = a.c;
  Access access;
  access.rows(c.x.p, c.x.ld, c.N, sizeof(T));
  access.rows(c.residual.p, c.residual.ld, c.N, sizeof(T));
  access.rows(c.sum.p, c.sum.ld, c.N, sizeof(T));
  access.rows(c.gain, 0, 1, sizeof(T));
  // An 8-bit output's accesses are narrower by the same factor.
  access.bits |= reinterpret_cast<uintptr_t>(c.out.p) * (c.e4m3 ? sizeof(T) : 1);
  if (c.N > 1) access.bits |= c.out.ld * sizeof(T);
  access.bits |= (size_t)a.K * sizeof(T);
  switch (access.bytes(sizeof(T))) {
    case 16:
      return rows_by<T, 16 / sizeof(T), 2>(h, a, stream);
    case 4:
      return rows_by<T, 4 / sizeof(T), 8>(h, a, stream);
    default:
      return rows_by<T, 1, 8>(h, a, stream);
  }
}

cudaError_t rows(const hg_norm& h, const NormCall& c, cudaStream_t stream) {
  RowsArgs a = {c, h.K, {}};
  switch (h.dtype) {
    case HG_BF16:
      return rows_of<__nv_bfloat16>(h, a, stream);
    case HG_FP16:
      return rows_of<__half>(h, a, stream);
    default:
      return rows_of<float>(h, a, stream);
  }
}

template <typename T>
cudaError_t grad_of(const hg_norm& h, GradArgs& a, cudaStream_t stream) {
  const GradCall& c = a.c;
  Access access;
  access.rows(c.s.p, c.s.ld, c.N, sizeof(T));
  access.rows(c.grad_out.p, c.grad_out.ld, c.N, sizeof(T));
  access.rows(c.grad_sum.p, c.grad_sum.ld, c.N, sizeof(T));
  access.rows(c.grad_x.p, c.grad_x.ld, c.N, sizeof(T));
  access.rows(c.gain, 0, 1, sizeof(T));
  access.bits |= (size_t)a.K * sizeof(T);
  switch (access.bytes(sizeof(T))) {
    case 16:
      return grad_by<T, 16 / sizeof(T), 2, 512>(h, a, stream);
    case 4:
      return grad_by<T, 4 / sizeof(T), 2, 1024>(h, a, stream);
    default:
      return grad_by<T, 1, 4, 1024>(h, a, stream);
  }
}

cudaError_t rows_grad(const hg_norm& h, const GradCall& c, cudaStream_t stream) {
  GradArgs a = {c, h.K, {}, 1, h.partial};
  switch (h.dtype) {
    case HG_BF16:
      return grad_of<__nv_bfloat16>(h, a, stream);
    case HG_FP16:
      return grad_of<__half>(h, a, stream);
    default:
      return grad_of<float>(h, a, stream);
  }
}

}  // namespace norm
}  // namespace hg
