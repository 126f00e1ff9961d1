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
__device__ __forceinline__ uint16_t to_e4m3x2(float lo, float hi) {
  uint16_t w;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(w) : "f"(hi), "f"(lo));
  return w;
}

// The scale of values up to `most` in magnitude, and its reciprocal (to two units of its
// last place: what it multiplies is rounded to four bits).
__device__ __forceinline__ float scale_of(float most) {
  return most == 0.f ? 1.f : fmaxf(most * (1.f / kE4m3Most), kLeastScale);
}
__device__ __forceinline__ float inverse_of(float scale) { return __fdividef(1.f, scale); }

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


// 8-bit output of a row.
template <int E, int A>
__device__ __forceinline__ void store_e4m3(const RowsArgs& a, size_t n, bool there, int first,
                                           float* red, const float (&y)[A][E]) {
  const NormCall& c = a.c;
  const int step = a.shape.threads, accesses = a.K / E;
  uint8_t* out = static_cast<uint8_t*>(c.out.p) + n * c.out.ld;
  float most[A];
#pragma unroll
  for (int j = 0; j < A; ++j) {
    most[j] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) most[j] = fmaxf(most[j], fabsf(y[j][e]));
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
    const float inverse = inverse_of(most[j]);
    Pack<uint8_t, E> q;
    if constexpr (E == 1) {
      q.v[0] = to_e4m3(y[j][0] * inverse);
    } else {
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const uint16_t w = to_e4m3x2(y[j][e] * inverse, y[j][e + 1] * inverse);
        q.v[e] = (uint8_t)w;
        q.v[e + 1] = (uint8_t)(w >> 8);
      }
    }
    if (first + j * step < accesses) reinterpret_cast<Pack<uint8_t, E>*>(out)[first + j * step] = q;
  }
}

template <typename T, int E, int A, bool QUANT>
__global__ void __launch_bounds__(1024) rows_kernel(const __grid_constant__ RowsArgs a) {
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
    float v[A][E];
#pragma unroll
    for (int j = 0; j < A; ++j)
#pragma unroll
      for (int e = 0; e < E; ++e) v[j][e] = y(j, e);
    store_e4m3<E, A>(a, n, there, first, red[1], v);
  } else if (there) {
#pragma unroll
    for (int j = 0; j < A; ++j)
#pragma unroll
      for (int e = 0; e < E; ++e) s[j].v[e] = Elem<T>::down(y(j, e));
    store_row(s, c.out, n, first, step, accesses);
  }
}

// Copies of a thread's own 16 bytes into shared memory, which only that thread reads: they
// run ahead of it over several rows without holding registers, and need no barrier.
__device__ __forceinline__ void copy_ahead(uint4* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(to)),
               "l"(from)
               : "memory");
}
__device__ __forceinline__ void close_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits for all but the last S - 1 groups of this thread's copies.
template <int S>
__device__ __forceinline__ void wait_copies() {
  asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
}

template <typename T, int A>
__device__ __forceinline__ void fetch_row(uint4* to, int pitch, const Rows& m, size_t n, int first,
                                          int step, int accesses) {
  const uint4* p = reinterpret_cast<const uint4*>(static_cast<const T*>(m.p) + n * m.ld);
#pragma unroll
  for (int j = 0; j < A; ++j)
    if (first + j * step < accesses) copy_ahead(to + j * pitch, p + first + j * step);
}

// The same for many rows in 16-byte accesses: a CTA takes every grid-th group of rows, and has
// the next ones' loads, S rows a thread with this one's, under way.
template <typename T, int A, int S, bool QUANT>
__global__ void __launch_bounds__(1024) rows_stream_kernel(const __grid_constant__ RowsArgs a) {
  constexpr int E = 16 / sizeof(T);
  extern __shared__ uint4 ring[];  // [stage][x, residual][A][threads]
  __shared__ float red[2][2][32];
  wait_for_predecessor();
  let_successor_start();
  const NormCall& c = a.c;
  const int step = a.shape.threads, sub = threadIdx.x / step, first = threadIdx.x - sub * step;
  const int accesses = a.K / E, pitch = blockDim.x;
  const size_t stride = (size_t)gridDim.x * a.shape.rows;
  size_t n = (size_t)blockIdx.x * a.shape.rows + sub;
  auto fetch = [&](size_t row, int stage) {
    uint4* to = ring + stage * 2 * A * pitch + threadIdx.x;
    if (row < (size_t)c.N) {
      fetch_row<T, A>(to, pitch, c.x, row, first, step, accesses);
      if (c.residual.p) fetch_row<T, A>(to + A * pitch, pitch, c.residual, row, first, step, accesses);
    }
    close_copies();
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) fetch(n + i * stride, i);
  Pack<T, E> g[A], s[A];
  clear_row(g);
  load_row(g, Rows{c.gain, 0}, 0, first, step, accesses);
  int stage = 0, turn = 0;
  for (size_t n0 = (size_t)blockIdx.x * a.shape.rows; n0 < (size_t)c.N; n0 += stride, n += stride) {
    const bool there = n < (size_t)c.N;
    fetch(n + (S - 1) * stride, stage == 0 ? S - 1 : stage - 1);
    wait_copies<S>();
    const uint4* from = ring + stage * 2 * A * pitch + threadIdx.x;
    float squares = 0.f;
#pragma unroll
    for (int j = 0; j < A; ++j) {
      const bool in = there && first + j * step < accesses;
      if (in) {
        *reinterpret_cast<uint4*>(&s[j]) = from[j * pitch];
        if (c.residual.p) {
          Pack<T, E> r;
          *reinterpret_cast<uint4*>(&r) = from[(A + j) * pitch];
#pragma unroll
          for (int e = 0; e < E; ++e)
            s[j].v[e] = Elem<T>::down(Elem<T>::up(s[j].v[e]) + Elem<T>::up(r.v[e]));
        }
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) s[j].v[e] = Elem<T>::down(0.f);
      }
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float v = Elem<T>::up(s[j].v[e]);
        squares += v * v;
      }
    }
    if (there && c.sum.p) store_row(s, c.sum, n, first, step, accesses);
    const float rstd =
        rsqrtf(row_all<false>(squares, red[turn][0], step / 32) / (float)a.K + c.eps);
    if (there && c.rstd && first == 0) c.rstd[n] = rstd;
    auto y = [&](int j, int e) {
      return Elem<T>::up(s[j].v[e]) * rstd * Elem<T>::up(g[j].v[e]);
    };
    if constexpr (QUANT) {
      float v[A][E];
#pragma unroll
      for (int j = 0; j < A; ++j)
#pragma unroll
        for (int e = 0; e < E; ++e) v[j][e] = y(j, e);
      store_e4m3<E, A>(a, n, there, first, red[turn][1], v);
    } else if (there) {
#pragma unroll
      for (int j = 0; j < A; ++j)
#pragma unroll
        for (int e = 0; e < E; ++e) s[j].v[e] = Elem<T>::down(y(j, e));
      store_row(s, c.out, n, first, step, accesses);
    }
    turn ^= 1;
    if (++stage == S) stage = 0;
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
    const float inverse = inverse_of(scale);
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

// What a CTA's rows give to grad_gain.
template <int E, int A>
__device__ __forceinline__ void store_partial(const GradArgs& a, const float (&acc)[A][E], int sub,
                                              int first) {
  const int step = a.shape.threads, accesses = a.K / E;
  float* partial = a.partial + (size_t)blockIdx.x * a.K;
  // Several rows a CTA: the threads that hold a column add up in the rows' order.
  if (a.shape.rows > 1) {
    extern __shared__ float sums[];  // [rows][K], where the rows' copies were
    __syncthreads();
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
    return;
  }
#pragma unroll
  for (int j = 0; j < A; ++j) {
    if (first + j * step >= accesses) continue;
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
}

// Both gradients in one pass: a CTA takes every parts-th row (or group of short rows),
// holds it in registers between the inner sum and grad_x, and adds what its columns give
// to grad_gain up in registers over all its rows.
template <typename T, int E, int A, bool GAIN>
__global__ void __launch_bounds__(1024)
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
  if (GAIN) store_partial<E, A>(a, acc, sub, first);
}

// The same for many rows in 16-byte accesses, streamed as rows_stream_kernel does. A row is
// read twice, from shared memory, so that the registers are left to the sums of grad_gain.
template <typename T, int A, int S>
__global__ void __launch_bounds__(1024) grad_stream_kernel(const __grid_constant__ GradArgs a) {
  constexpr int E = 16 / sizeof(T);
  extern __shared__ uint4 ring[];  // [stage][s, grad_out, grad_sum][A][threads]
  __shared__ float red[2][32];
  wait_for_predecessor();
  let_successor_start();
  const GradCall& c = a.c;
  const int step = a.shape.threads, sub = threadIdx.x / step, first = threadIdx.x - sub * step;
  const int accesses = a.K / E, pitch = blockDim.x;
  const size_t stride = (size_t)gridDim.x * a.shape.rows;
  size_t n = (size_t)blockIdx.x * a.shape.rows + sub;
  auto fetch = [&](size_t row, int stage) {
    uint4* to = ring + stage * 3 * A * pitch + threadIdx.x;
    if (row < (size_t)c.N) {
      fetch_row<T, A>(to, pitch, c.s, row, first, step, accesses);
      fetch_row<T, A>(to + A * pitch, pitch, c.grad_out, row, first, step, accesses);
      if (c.grad_sum.p && c.grad_x.p)
        fetch_row<T, A>(to + 2 * A * pitch, pitch, c.grad_sum, row, first, step, accesses);
    }
    close_copies();
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) fetch(n + i * stride, i);
  Pack<T, E> g[A];
  clear_row(g);
  load_row(g, Rows{c.gain, 0}, 0, first, step, accesses);
  float acc[A][E] = {};
  int stage = 0, turn = 0;
  for (size_t n0 = (size_t)blockIdx.x * a.shape.rows; n0 < (size_t)c.N; n0 += stride, n += stride) {
    const bool there = n < (size_t)c.N;
    fetch(n + (S - 1) * stride, stage == 0 ? S - 1 : stage - 1);
    const float rstd = there ? c.rstd[n] : 0.f;
    wait_copies<S>();
    const uint4* from = ring + stage * 3 * A * pitch + threadIdx.x;
    Pack<T, E> s, up, more;
    float inner = 0.f;
#pragma unroll
    for (int j = 0; j < A; ++j) {
      if (!there || first + j * step >= accesses) continue;
      *reinterpret_cast<uint4*>(&s) = from[j * pitch];
      *reinterpret_cast<uint4*>(&up) = from[(A + j) * pitch];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float t = Elem<T>::up(up.v[e]) * Elem<T>::up(s.v[e]);
        inner += t * Elem<T>::up(g[j].v[e]);
        acc[j][e] += t * rstd;
      }
    }
    if (c.grad_x.p) {
      inner = row_all<false>(inner, red[turn], step / 32) / (float)a.K * (rstd * rstd * rstd);
      turn ^= 1;
      Pack<T, E>* out =
          reinterpret_cast<Pack<T, E>*>(static_cast<T*>(c.grad_x.p) + n * c.grad_x.ld);
#pragma unroll
      for (int j = 0; j < A; ++j) {
        if (!there || first + j * step >= accesses) continue;
        *reinterpret_cast<uint4*>(&s) = from[j * pitch];
        *reinterpret_cast<uint4*>(&up) = from[(A + j) * pitch];
        if (c.grad_sum.p)
          *reinterpret_cast<uint4*>(&more) = from[(2 * A + j) * pitch];
        else
          *reinterpret_cast<uint4*>(&more) = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < E; ++e)
          more.v[e] = Elem<T>::down(rstd * (Elem<T>::up(up.v[e]) * Elem<T>::up(g[j].v[e])) -
                                    Elem<T>::up(s.v[e]) * inner + Elem<T>::up(more.v[e]));
        out[first + j * step] = more;
      }
    }
    if (++stage == S) stage = 0;
  }
  if (c.grad_gain) store_partial<E, A>(a, acc, sub, first);
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

constexpr int kStages = 3, kStagesQuant = 2;
constexpr size_t kRingMost = 220 * 1024;  // beside the kernels' static shared memory

// Lays rows on threads for a kernel that streams them, `target` threads an SM, and returns the
// CTAs of its grid.
template <int A>
unsigned stream_shape(Shape& shape, int accesses, int N, int sms, int target) {
  shape.threads = (int)round_up(div_up(accesses, A), 32);
  const int block = shape.threads < 128 ? 128 : 512;
  shape.rows = shape.threads < block ? block / shape.threads : 1;
  if (shape.rows > N / sms) shape.rows = N / sms > 1 ? N / sms : 1;  // a CTA for every SM first
  const int per_sm = target / (shape.threads * shape.rows);
  const long long full = (long long)(per_sm > 1 ? per_sm : 1) * sms;
  const long long groups = div_up(N, shape.rows);
  return (unsigned)(groups < full ? groups : full);
}

template <typename T, int S, bool QUANT>
cudaError_t rows_stream(const hg_norm& h, RowsArgs& a, cudaStream_t stream) {
  // The 8-bit output's second round of maxima wants more rows at a time (2048 rows of 7168:
  // 26 us with 512 threads an SM, 21.5 with 1024; plain, 8192 rows, 70 and 82).
  const unsigned grid = stream_shape<2>(a.shape, a.K / (16 / (int)sizeof(T)), a.c.N, h.sms,
                                        QUANT ? 1024 : 512);
  const unsigned block = (unsigned)(a.shape.threads * a.shape.rows);
  return launch_dependent(rows_stream_kernel<T, 2, S, QUANT>, a, grid, block,
                          (size_t)S * 2 * 2 * block * 16, 1, stream);
}

// Few accesses a thread where rows are few and their latency counts; many rows in 16-byte
// accesses are streamed; others take LONG accesses a thread, so that several rows'
// loads are under way on an SM.
template <typename T, int E, int LONG>
cudaError_t rows_by(const hg_norm& h, RowsArgs& a, cudaStream_t stream) {
  constexpr bool kWide = E * sizeof(T) == 16;
  const int accesses = a.K / E;
  if (accesses > LONG * 1024)
    return launch_dependent(long_rows_kernel<T>, a, (unsigned)a.c.N, kThreads, 0, 1, stream);
  if (a.c.N <= h.sms && accesses <= 1024) return rows_as<T, E, 1>(h, a, stream);
  if constexpr (kWide)
    return a.c.e4m3 ? rows_stream<T, kStagesQuant, true>(h, a, stream)
                    : rows_stream<T, kStages, false>(h, a, stream);
  else
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

template <typename T, int E, int A>
cudaError_t grad_as(const hg_norm& h, GradArgs& a, cudaStream_t stream) {
  a.shape.threads = (int)round_up(div_up(a.K / E, A), 32);
  a.shape.rows = a.shape.threads < 128 ? 128 / a.shape.threads : 1;
  const unsigned block = (unsigned)(a.shape.threads * a.shape.rows);
  const long long groups = div_up(a.c.N, a.shape.rows);
  const int most = grad_parts(h);
  a.parts = groups < 1 ? 1 : groups < most ? (int)groups : most;
  const unsigned grid = (unsigned)a.parts;
  const size_t smem = a.shape.rows > 1 ? (size_t)a.shape.rows * a.K * sizeof(float) : 0;
  if (!a.c.grad_gain)
    return launch_dependent(grad_kernel<T, E, A, false>, a, grid, block, 0, 1, stream);
  const cudaError_t e =
      launch_dependent(grad_kernel<T, E, A, true>, a, grid, block, smem, 1, stream);
  return e == cudaSuccess ? join_gain<T>(a, stream) : e;
}

template <typename T>
cudaError_t grad_stream(const hg_norm& h, GradArgs& a, cudaStream_t stream) {
  const unsigned grid =
      stream_shape<2>(a.shape, a.K / (16 / (int)sizeof(T)), a.c.N, h.sms, 512);
  a.parts = (int)grid;
  const unsigned block = (unsigned)(a.shape.threads * a.shape.rows);
  const size_t stage = (size_t)3 * 2 * block * 16;
  const cudaError_t e =
      3 * stage <= kRingMost
          ? launch_dependent(grad_stream_kernel<T, 2, 3>, a, grid, block, 3 * stage, 1, stream)
          : launch_dependent(grad_stream_kernel<T, 2, 2>, a, grid, block, 2 * stage, 1, stream);
  return e == cudaSuccess && a.c.grad_gain ? join_gain<T>(a, stream) : e;
}

template <typename T>
cudaError_t grad_of_rows_beyond(const hg_norm& h, GradArgs& a, cudaStream_t stream) {
  const long long parts = div_up(a.c.N, kSubRows);
  const int most = grad_parts(h);
  a.parts = parts < 1 ? 1 : parts < most ? (int)parts : most;
  return grad_of_long_rows<T>(a, stream);
}

// Few accesses a thread where rows are few and their latency counts; many rows in 16-byte
// accesses are streamed; others take A or twice as many accesses a thread.
template <typename T, int E, int A>
cudaError_t grad_by(const hg_norm& h, GradArgs& a, cudaStream_t stream) {
  const int accesses = a.K / E;
  if (a.c.N <= h.sms && accesses <= 1024) return grad_as<T, E, 1>(h, a, stream);
  if constexpr (E * sizeof(T) == 16) {
    if (accesses <= 2 * 1024) return grad_stream<T>(h, a, stream);
  } else {
    if (accesses <= A * 1024) return grad_as<T, E, A>(h, a, stream);
    if (accesses <= 2 * A * 1024) return grad_as<T, E, 2 * A>(h, a, stream);
  }
  return grad_of_rows_beyond<T>(h, a, stream);
}

}  // namespace

template <typename T>
cudaError_t prepare_as() {
  cudaError_t e = cudaSuccess;
  for (void (*kernel)(RowsArgs) : {rows_stream_kernel<T, 2, kStagesQuant, true>,
                                   rows_stream_kernel<T, 2, kStages, false>})
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRingMost);
  for (void (*kernel)(GradArgs) : {grad_stream_kernel<T, 2, 2>, grad_stream_kernel<T, 2, 3>})
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRingMost);
  return e;
}

cudaError_t prepare(const hg_norm& h) {
  return h.dtype == HG_BF16   ? prepare_as<__nv_bfloat16>()
         : h.dtype == HG_FP16 ? prepare_as<__half>()
                              : prepare_as<float>();
}

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
      return grad_by<T, 16 / sizeof(T), 2>(h, a, stream);
    case 4:
      return grad_by<T, 4 / sizeof(T), 2>(h, a, stream);
    default:
      return grad_by<T, 1, 4>(h, a, stream);
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
