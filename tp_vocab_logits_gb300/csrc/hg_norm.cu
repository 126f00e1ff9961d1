// Root-mean-square norm of rows with the residual's addition, and its gradient.
//
// Memory bounds both directions, so a row is read once: a group of threads, whole warps,
// holds it (in registers, packed as it came, or in shared memory) between the sum over
// the row and the output. A CTA has one group, or several that work on rows of their own.
// Rows in 16-byte accesses, if there are many of them, are streamed: each thread copies
// the 16 bytes that it will itself read into a ring in shared memory (cp.async), a few rows
// ahead, which takes no registers and no barrier. Longer rows than the kernels hold are read
// again, element by element: more than 2048 accesses of 16 bytes, 8192 shorter ones (the
// gradient: 4096 of 4 bytes, 8192 of 2).

#include <cuda_fp8.h>

#include <cstring>

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

constexpr int kThreads = 256;  // of the kernels for long rows
constexpr int kWarps = kThreads / 32;
constexpr int kMostThreads = 1024;
constexpr float kE4m3Most = 448.f;
constexpr float kLeastScale = 1.17549435e-38f;  // 2^-126: its reciprocal is finite

template <bool MAX>
__device__ __forceinline__ float combine(float a, float b) {
  return MAX ? fmaxf(a, b) : a + b;
}

// Over a warp, the same value in each lane. Maxima are of magnitudes, ordered as their bits.
template <bool MAX>
__device__ __forceinline__ float warp_all(float v) {
  if constexpr (MAX) {
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
  } else {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
  }
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
// last place: what it multiplies is rounded to four bits, so that only values in the middle
// between two, within 2^-20, may go to the other one; their error is half a step either way.
// Of 2048 rows of 7168 bf16, 865 values differ from a division's, all of them exact ties).
__device__ __forceinline__ float scale_of(float most) {
  return most == 0.f ? 1.f : fmaxf(most * (1.f / kE4m3Most), kLeastScale);
}
__device__ __forceinline__ float inverse_of(float scale) { return __fdividef(1.f, scale); }

// The elements of an access in fp32 and back, 16-bit ones two at a time.
template <typename T, int E>
__device__ __forceinline__ void widen(const Pack<T, E>& p, float (&v)[E]) {
  if constexpr (sizeof(T) == 2 && E > 1) {
    uint32_t w[E / 2];
    memcpy(w, &p, sizeof p);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      const float2 f = Elem<T>::unpack2(w[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = Elem<T>::up(p.v[e]);
  }
}
template <typename T, int E>
__device__ __forceinline__ Pack<T, E> narrow(const float (&v)[E]) {
  Pack<T, E> p;
  if constexpr (sizeof(T) == 2 && E > 1) {
    uint32_t w[E / 2];
#pragma unroll
    for (int i = 0; i < E / 2; ++i) w[i] = Elem<T>::pack2(v[2 * i], v[2 * i + 1]);
    memcpy(&p, w, sizeof p);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) p.v[e] = Elem<T>::down(v[e]);
  }
  return p;
}

// Two fp32 operations in one instruction, and the elements of an access two at a time (the
// 8-bit output and the gradient issue in three of four cycles: 4096 rows of 7168, 8 bits, a scale
// a row 36.5 -> 33.2 us, the gradient 43.9 -> 43.0).
typedef unsigned long long u64;
__device__ __forceinline__ u64 pair(float lo, float hi) {
  return (u64)__float_as_uint(hi) << 32 | __float_as_uint(lo);
}
__device__ __forceinline__ float low(u64 p) { return __uint_as_float((uint32_t)p); }
__device__ __forceinline__ float high(u64 p) { return __uint_as_float((uint32_t)(p >> 32)); }
__device__ __forceinline__ u64 fma2(u64 a, u64 b, u64 c) {
  u64 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ u64 mul2(u64 a, u64 b) {
  u64 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ u64 add2(u64 a, u64 b) {
  u64 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
template <typename T, int E>
__device__ __forceinline__ void widen_pairs(const Pack<T, E>& p, u64 (&v)[E / 2]) {
  float f[E];
  widen(p, f);
#pragma unroll
  for (int i = 0; i < E / 2; ++i) v[i] = pair(f[2 * i], f[2 * i + 1]);
}

// x + residual, rounded.
template <typename T, int E>
__device__ __forceinline__ Pack<T, E> added(const Pack<T, E>& x, const Pack<T, E>& residual) {
  float a[E], b[E];
  widen(x, a);
  widen(residual, b);
  if constexpr (E % 2 == 0) {
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const u64 sum = add2(pair(a[e], a[e + 1]), pair(b[e], b[e + 1]));
      a[e] = low(sum);
      a[e + 1] = high(sum);
    }
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) a[e] += b[e];
  }
  return narrow<T, E>(a);
}

// How a launch lays rows on threads.
struct Shape {
  int threads;  // of a group: whole warps
  int groups;   // of a CTA
};

// A thread's place: its group, and the first access of its own in a row.
struct Place {
  int step, sub, first;
  __device__ explicit Place(const Shape& s)
      : step(s.threads), sub(threadIdx.x / s.threads), first(threadIdx.x - sub * s.threads) {}
  // The group's threads, which need not be where the others are. (Barrier 0 is the CTA's.)
  __device__ void sync() const {
    asm volatile("bar.sync %0, %1;" ::"r"(sub + 1), "r"(step) : "memory");
  }
};

// Over a group's threads, the same value in each. `red` holds a word per warp of the CTA, and
// is free again after the group's next barrier.
template <bool MAX>
__device__ __forceinline__ float group_all(float v, float* red, const Place& at) {
  v = warp_all<MAX>(v);
  if (at.step == 32) return v;
  const int lane = threadIdx.x & 31, warps = at.step / 32;
  float* mine = red + at.sub * warps;
  if (lane == 0) mine[at.first >> 5] = v;
  at.sync();
  return warp_all<MAX>(lane < warps ? mine[lane] : 0.f);
}

template <typename T, int E, int A>
__device__ __forceinline__ void load_row(Pack<T, E> (&to)[A], const Rows& m, size_t n,
                                         const Place& at, int accesses) {
  const Pack<T, E>* p =
      reinterpret_cast<const Pack<T, E>*>(static_cast<const T*>(m.p) + n * m.ld) + at.first;
#pragma unroll
  for (int j = 0; j < A; ++j)
    if (at.first + j * at.step < accesses) to[j] = p[j * at.step];
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
                                          const Place& at, int accesses) {
  Pack<T, E>* p = reinterpret_cast<Pack<T, E>*>(static_cast<T*>(m.p) + n * m.ld) + at.first;
#pragma unroll
  for (int j = 0; j < A; ++j)
    if (at.first + j * at.step < accesses) p[j * at.step] = from[j];
}

// Copies of a thread's own 16 bytes into shared memory.
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
__device__ __forceinline__ void fetch_row(uint4* to, int pitch, const Rows& m, size_t n,
                                          const Place& at, int accesses) {
  const uint4* p = reinterpret_cast<const uint4*>(static_cast<const T*>(m.p) + n * m.ld) + at.first;
#pragma unroll
  for (int j = 0; j < A; ++j)
    if (at.first + j * at.step < accesses) copy_ahead(to + j * pitch, p + j * at.step);
}

// ---- the norm ----------------------------------------------------------------------

struct RowsArgs {
  NormCall c;
  int K;
  Shape shape;
};

// 8-bit output of a row.
template <int E, int A>
__device__ __forceinline__ void store_e4m3(const RowsArgs& a, size_t n, bool there,
                                           const Place& at, float* red, const float (&y)[A][E]) {
  const NormCall& c = a.c;
  const int accesses = a.K / E;
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
    const float scale = scale_of(group_all<true>(most[0], red, at));
    if (there && at.first == 0) c.scales[n] = scale;
#pragma unroll
    for (int j = 0; j < A; ++j) most[j] = scale;
  } else {
    // The lanes that hold a block of 128 columns: 128 / E neighbours, or whole warps.
    constexpr int kLanes = 128 / E < 32 ? 128 / E : 32;
    const int blocks = (a.K + 127) / 128;
#pragma unroll
    for (int j = 0; j < A; ++j)
#pragma unroll
      for (int m = kLanes / 2; m > 0; m >>= 1)
        most[j] = fmaxf(most[j], __shfl_xor_sync(0xffffffffu, most[j], m));
    if constexpr (128 / E > 32) {
      __shared__ unsigned joined[kMostThreads * A * E / 128];  // magnitudes order as their bits do
      for (int b = threadIdx.x; b < a.shape.groups * blocks; b += blockDim.x) joined[b] = 0;
      __syncthreads();
      unsigned* mine = joined + at.sub * blocks;
#pragma unroll
      for (int j = 0; j < A; ++j)
        if ((threadIdx.x & 31) == 0 && at.first + j * at.step < accesses)
          atomicMax(&mine[(at.first + j * at.step) / (128 / E)], __float_as_uint(most[j]));
      __syncthreads();
#pragma unroll
      for (int j = 0; j < A; ++j)
        if (at.first + j * at.step < accesses)
          most[j] = __uint_as_float(mine[(at.first + j * at.step) / (128 / E)]);
    }
#pragma unroll
    for (int j = 0; j < A; ++j) {
      const int i = at.first + j * at.step;
      most[j] = scale_of(most[j]);
      if (there && i < accesses && i % (128 / E) == 0)
        c.scales[n * blocks + i / (128 / E)] = most[j];
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
      uint16_t w[E / 2];
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const u64 x = mul2(pair(y[j][e], y[j][e + 1]), pair(inverse, inverse));
        w[e / 2] = to_e4m3x2(low(x), high(x));
      }
      memcpy(&q, w, E);
    }
    const int i = at.first + j * at.step;
    if (i < accesses) reinterpret_cast<Pack<uint8_t, E>*>(out)[i] = q;
  }
}

// From the squares of a row's sum to its outputs (SUM: it is one of them). `red`: two arrays
// for group_all.
template <typename T, int E, int A, bool QUANT, bool SUM>
__device__ __forceinline__ void finish_row(const RowsArgs& a, Pack<T, E> (&s)[A],
                                           const Pack<T, E> (&gain)[A], size_t n, bool there,
                                           const Place& at, float (&red)[2][32]) {
  const NormCall& c = a.c;
  float squares = 0.f;
  if constexpr (E % 2 == 0) {
    u64 sums = 0;
#pragma unroll
    for (int j = 0; j < A; ++j) {
      u64 v[E / 2];
      widen_pairs(s[j], v);
#pragma unroll
      for (int i = 0; i < E / 2; ++i) sums = fma2(v[i], v[i], sums);
    }
    squares = low(sums) + high(sums);
  } else {
#pragma unroll
    for (int j = 0; j < A; ++j) {
      float v[E];
      widen(s[j], v);
#pragma unroll
      for (int e = 0; e < E; ++e) squares += v[e] * v[e];
    }
  }
  const float rstd = rsqrtf(group_all<false>(squares, red[0], at) / (float)a.K + c.eps);
  if (there && c.rstd && at.first == 0) c.rstd[n] = rstd;
  if (SUM && c.sum.p) store_row(s, c.sum, n, at, a.K / E);
  float y[A][E];
#pragma unroll
  for (int j = 0; j < A; ++j) {
    float g[E];
    widen(s[j], y[j]);
    widen(gain[j], g);
    if constexpr (E % 2 == 0) {
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const u64 x = mul2(mul2(pair(y[j][e], y[j][e + 1]), pair(rstd, rstd)),
                           pair(g[e], g[e + 1]));
        y[j][e] = low(x);
        y[j][e + 1] = high(x);
      }
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) y[j][e] = y[j][e] * rstd * g[e];
    }
  }
  if constexpr (QUANT) {
    store_e4m3<E, A>(a, n, there, at, red[1], y);
  } else if (there) {
#pragma unroll
    for (int j = 0; j < A; ++j) s[j] = narrow<T, E>(y[j]);
    store_row(s, c.out, n, at, a.K / E);
  }
}

// A row per group.
template <typename T, int E, int A, bool QUANT>
__global__ void __launch_bounds__(kMostThreads) rows_kernel(const __grid_constant__ RowsArgs a) {
  __shared__ float red[2][32];
  wait_for_predecessor();
  let_successor_start();
  const NormCall& c = a.c;
  const Place at(a.shape);
  const int accesses = a.K / E;
  const size_t n = (size_t)blockIdx.x * a.shape.groups + at.sub;
  const bool there = n < (size_t)c.N;
  Pack<T, E> s[A], g[A];
  clear_row(s);
  clear_row(g);
  if (there) {
    load_row(s, c.x, n, at, accesses);
    if (c.residual.p) {
      load_row(g, c.residual, n, at, accesses);
#pragma unroll
      for (int j = 0; j < A; ++j) s[j] = added(s[j], g[j]);
    }
    load_row(g, Rows{c.gain, 0}, 0, at, accesses);
    if (c.sum.p) store_row(s, c.sum, n, at, accesses);
  }
  finish_row<T, E, A, QUANT, false>(a, s, g, n, there, at, red);
}

// Every stride-th row per group, S rows of each thread (this one's among them) in the ring.
template <typename T, int A, int S, bool QUANT>
__global__ void __launch_bounds__(kMostThreads)
    rows_stream_kernel(const __grid_constant__ RowsArgs a) {
  constexpr int E = 16 / sizeof(T);
  extern __shared__ uint4 ring[];  // [stage][x, residual][A][threads]
  __shared__ float red[2][2][32];
  wait_for_predecessor();
  let_successor_start();
  const NormCall& c = a.c;
  const Place at(a.shape);
  const int accesses = a.K / E, pitch = blockDim.x;
  const size_t stride = (size_t)gridDim.x * a.shape.groups;
  auto fetch = [&](size_t row, int stage) {
    uint4* to = ring + stage * 2 * A * pitch + threadIdx.x;
    if (row < (size_t)c.N) {
      fetch_row<T, A>(to, pitch, c.x, row, at, accesses);
      if (c.residual.p) fetch_row<T, A>(to + A * pitch, pitch, c.residual, row, at, accesses);
    }
    close_copies();
  };
  size_t n = (size_t)blockIdx.x * a.shape.groups + at.sub;
#pragma unroll
  for (int i = 0; i < S - 1; ++i) fetch(n + i * stride, i);
  Pack<T, E> g[A], s[A];
  clear_row(g);
  load_row(g, Rows{c.gain, 0}, 0, at, accesses);
  int stage = 0, turn = 0;
  for (; n < (size_t)c.N; n += stride) {
    fetch(n + (S - 1) * stride, stage == 0 ? S - 1 : stage - 1);
    wait_copies<S>();
    const uint4* from = ring + stage * 2 * A * pitch + threadIdx.x;
#pragma unroll
    for (int j = 0; j < A; ++j) {
      if (at.first + j * at.step < accesses) {
        memcpy(&s[j], from + j * pitch, 16);
        if (c.residual.p) {
          Pack<T, E> r;
          memcpy(&r, from + (A + j) * pitch, 16);
          s[j] = added(s[j], r);
        }
      } else {
        memset(&s[j], 0, 16);
      }
    }
    // The sum is stored just before the output: both streams of stores are where few loads are
    // (8192 rows of 7168: 74 us stored here, 70 us there; in 8 bits, where the output comes late,
    // it is the other way about, 18.5 and 19.0 us for 2048 rows).
    if (QUANT && c.sum.p) store_row(s, c.sum, n, at, accesses);
    finish_row<T, E, A, QUANT, !QUANT>(a, s, g, n, true, at, red[turn]);
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
  auto total = [&](int k) {
    const float v = Elem<T>::up(x[k]);
    return res ? Elem<T>::down(v + Elem<T>::up(res[k])) : x[k];
  };
  float squares = 0.f;
  for (int b = warp * 128; b < a.K; b += kWarps * 128)
    for (int k = b + lane; k < b + 128 && k < a.K; k += 32) {
      const T s = total(k);
      if (sum) sum[k] = s;
      squares += Elem<T>::up(s) * Elem<T>::up(s);
    }
  const float rstd = rsqrtf(block_all<false>(squares, red) / (float)a.K + c.eps);
  if (c.rstd && threadIdx.x == 0) c.rstd[n] = rstd;
  auto normed = [&](int k) {
    const T s = sum ? sum[k] : total(k);  // this thread's own, where it was written
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

// ---- the gradient ------------------------------------------------------------------

struct GradArgs {
  GradCall c;
  int K;
  float per_column;  // 1 / K
  Shape shape;
  int parts;
  float* partial;  // [parts][K]
};

// With w = s * rstd, whose squares have a mean of 1 over a row, and d = grad_out * gain,
//   grad_x = rstd * d - w * (rstd * mean(d * w)) + grad_sum,
// and grad_gain sums grad_out * w: what is multiplied is of the size of d, of w or of the result.
// (rstd^3 and grad_out * s leave fp32's range for rows of 1e-14 or 1e15. They spare an
// instruction a pair: 4096 rows of 7168 bf16 42.7 us with them, 43.1 so.)

// Sum of d * w over an access; what its columns give to grad_gain is added to acc.
template <typename T, int E, bool GAIN>
__device__ __forceinline__ float add_products(const Pack<T, E>& s, const Pack<T, E>& up,
                                              const Pack<T, E>& gain, float rstd, float (&acc)[E]) {
  if constexpr (E % 2 == 0) {
    u64 v[E / 2], u[E / 2], g[E / 2], inner = 0;
    widen_pairs(s, v);
    widen_pairs(up, u);
    widen_pairs(gain, g);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      const u64 t = mul2(u[i], mul2(v[i], pair(rstd, rstd)));
      inner = fma2(t, g[i], inner);
      if (GAIN) {
        const u64 sum = add2(t, pair(acc[2 * i], acc[2 * i + 1]));
        acc[2 * i] = low(sum);
        acc[2 * i + 1] = high(sum);
      }
    }
    return low(inner) + high(inner);
  } else {
    float v[E], u[E], g[E], inner = 0.f;
    widen(s, v);
    widen(up, u);
    widen(gain, g);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float t = u[e] * (v[e] * rstd);
      inner += t * g[e];
      if (GAIN) acc[e] += t;
    }
    return inner;
  }
}

// grad_x of an access; inner: the row's mean of d * w, times rstd.
template <typename T, int E>
__device__ __forceinline__ Pack<T, E> grad_of_access(const Pack<T, E>& s, const Pack<T, E>& up,
                                                     const Pack<T, E>& more, const Pack<T, E>& gain,
                                                     float rstd, float inner) {
  float v[E], u[E], m[E], g[E];
  widen(s, v);
  widen(up, u);
  widen(more, m);
  widen(gain, g);
  if constexpr (E % 2 == 0) {
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const u64 w = mul2(pair(v[e], v[e + 1]), pair(rstd, rstd));
      const u64 rest = fma2(w, pair(-inner, -inner), pair(m[e], m[e + 1]));
      const u64 d = mul2(pair(u[e], u[e + 1]), pair(g[e], g[e + 1]));
      const u64 x = fma2(d, pair(rstd, rstd), rest);
      v[e] = low(x);
      v[e + 1] = high(x);
    }
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = rstd * (u[e] * g[e]) - v[e] * rstd * inner + m[e];
  }
  return narrow<T, E>(v);
}

// What a CTA's rows give to grad_gain: the groups in their order.
template <int E, int A>
__device__ __forceinline__ void store_partial(const GradArgs& a, const float (&acc)[A][E],
                                              const Place& at) {
  extern __shared__ __align__(16) float sums[];  // [groups][K], where the rows' copies were
  const int accesses = a.K / E;
  float* partial = a.partial + (size_t)blockIdx.x * a.K;
  const bool alone = a.shape.groups == 1;
  float* mine = alone ? partial : sums + at.sub * a.K;
  if (!alone) __syncthreads();
#pragma unroll
  for (int j = 0; j < A; ++j) {
    if (at.first + j * at.step >= accesses) continue;
    float* to = mine + (at.first + j * at.step) * E;
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
  if (alone) return;
  __syncthreads();
  for (int k = threadIdx.x; k < a.K; k += blockDim.x) {
    float v = sums[k];
    for (int r = 1; r < a.shape.groups; ++r) v += sums[r * a.K + k];
    partial[k] = v;
  }
}

// grad_x of a row that a group holds in registers, in place of s.
template <typename T, int E, int A, bool GAIN>
__device__ __forceinline__ void grad_row(const GradArgs& a, size_t n, const Pack<T, E> (&gain)[A],
                                         float (&acc)[A][E], const Place& at, float* red) {
  const GradCall& c = a.c;
  const int accesses = a.K / E;
  Pack<T, E> s[A], up[A], more[A];
  clear_row(s);
  clear_row(up);
  clear_row(more);
  load_row(s, c.s, n, at, accesses);
  load_row(up, c.grad_out, n, at, accesses);
  if (c.grad_sum.p && c.grad_x.p) load_row(more, c.grad_sum, n, at, accesses);
  const float rstd = c.rstd[n];
  float inner = 0.f;
#pragma unroll
  for (int j = 0; j < A; ++j)
    inner += add_products<T, E, GAIN>(s[j], up[j], gain[j], rstd, acc[j]);
  if (!c.grad_x.p) return;
  inner = group_all<false>(inner, red, at) * a.per_column * rstd;
#pragma unroll
  for (int j = 0; j < A; ++j)
    s[j] = grad_of_access<T, E>(s[j], up[j], more[j], gain[j], rstd, inner);
  store_row(s, c.grad_x, n, at, accesses);
}

// Both gradients in one pass: a group takes every stride-th row, and adds what its
// columns give to grad_gain up in registers over all of them.
template <typename T, int E, int A, bool GAIN>
__global__ void __launch_bounds__(kMostThreads) grad_kernel(const __grid_constant__ GradArgs a) {
  __shared__ float red[2][32];
  wait_for_predecessor();
  let_successor_start();
  const Place at(a.shape);
  Pack<T, E> g[A];
  clear_row(g);
  load_row(g, Rows{a.c.gain, 0}, 0, at, a.K / E);
  float acc[A][E] = {};
  int turn = 0;
  const size_t stride = (size_t)gridDim.x * a.shape.groups;
  for (size_t n = (size_t)blockIdx.x * a.shape.groups + at.sub; n < (size_t)a.c.N; n += stride) {
    grad_row<T, E, A, GAIN>(a, n, g, acc, at, red[turn]);
    turn ^= 1;
  }
  if (GAIN) store_partial<E, A>(a, acc, at);
}

constexpr int kFewColumns = 64;  // of a CTA, whose 4 to 16 groups of threads take rows in turn

// Few rows in one launch: the first N CTAs make grad_x, if it is wanted, a row each; the others
// grad_gain, which needs no sum over a row, from the rows as they lie (so grad_x is not grad_out).
template <typename T, int E>
__global__ void __launch_bounds__(kMostThreads) few_kernel(const __grid_constant__ GradArgs a) {
  __shared__ float red[32];
  __shared__ float sums[kMostThreads / kFewColumns][kFewColumns];
  wait_for_predecessor();
  let_successor_start();
  const GradCall& c = a.c;
  const int of_x = c.grad_x.p ? c.N : 0;
  if ((int)blockIdx.x < of_x) {
    const Place at(a.shape);
    if ((int)threadIdx.x >= at.step) return;
    Pack<T, E> g[1];
    clear_row(g);
    load_row(g, Rows{c.gain, 0}, 0, at, a.K / E);
    float none[1][E] = {};
    grad_row<T, E, 1, false>(a, blockIdx.x, g, none, at, red);
    return;
  }
  const int column = threadIdx.x % kFewColumns, sub = threadIdx.x / kFewColumns;
  const int subs = blockDim.x / kFewColumns, k = (blockIdx.x - of_x) * kFewColumns + column;
  float v = 0.f;
  if (k < a.K && sub < subs)
#pragma unroll 4
    for (int n = sub; n < c.N; n += subs)
      v += Elem<T>::up(static_cast<const T*>(c.grad_out.p)[n * c.grad_out.ld + k]) *
           (Elem<T>::up(static_cast<const T*>(c.s.p)[n * c.s.ld + k]) * c.rstd[n]);
  if (sub < subs) sums[sub][column] = v;
  __syncthreads();
  if (sub != 0 || k >= a.K) return;
  for (int i = 1; i < subs; ++i) v += sums[i][column];
  T* out = static_cast<T*>(c.grad_gain) + k;
  if (c.accumulate) v += Elem<T>::up(*out);
  *out = Elem<T>::down(v);
}

// Every stride-th row per group, streamed. A row is read twice, from shared memory, so that
// the registers are left to the sums of grad_gain.
template <typename T, int A, int S>
__global__ void __launch_bounds__(kMostThreads)
    grad_stream_kernel(const __grid_constant__ GradArgs a) {
  constexpr int E = 16 / sizeof(T);
  extern __shared__ uint4 ring[];  // [stage][s, grad_out, grad_sum][A][threads]
  __shared__ float red[2][32];
  wait_for_predecessor();
  let_successor_start();
  const GradCall& c = a.c;
  const Place at(a.shape);
  const int accesses = a.K / E, pitch = blockDim.x;
  const size_t stride = (size_t)gridDim.x * a.shape.groups;
  auto fetch = [&](size_t row, int stage) {
    uint4* to = ring + stage * 3 * A * pitch + threadIdx.x;
    if (row < (size_t)c.N) {
      fetch_row<T, A>(to, pitch, c.s, row, at, accesses);
      fetch_row<T, A>(to + A * pitch, pitch, c.grad_out, row, at, accesses);
      if (c.grad_sum.p && c.grad_x.p)
        fetch_row<T, A>(to + 2 * A * pitch, pitch, c.grad_sum, row, at, accesses);
    }
    close_copies();
  };
  size_t n = (size_t)blockIdx.x * a.shape.groups + at.sub;
#pragma unroll
  for (int i = 0; i < S - 1; ++i) fetch(n + i * stride, i);
  Pack<T, E> g[A];
  clear_row(g);
  load_row(g, Rows{c.gain, 0}, 0, at, accesses);
  float acc[A][E] = {};
  float next_rstd = n < (size_t)c.N ? c.rstd[n] : 0.f;
  int stage = 0, turn = 0;
  for (; n < (size_t)c.N; n += stride) {
    fetch(n + (S - 1) * stride, stage == 0 ? S - 1 : stage - 1);
    const float rstd = next_rstd;  // a row ahead: its latency would show (62 -> 52 us, one group)
    next_rstd = n + stride < (size_t)c.N ? c.rstd[n + stride] : 0.f;
    wait_copies<S>();
    const uint4* from = ring + stage * 3 * A * pitch + threadIdx.x;
    Pack<T, E> s, up, more;
    float inner = 0.f;
#pragma unroll
    for (int j = 0; j < A; ++j) {
      if (at.first + j * at.step >= accesses) continue;
      memcpy(&s, from + j * pitch, 16);
      memcpy(&up, from + (A + j) * pitch, 16);
      inner += add_products<T, E, true>(s, up, g[j], rstd, acc[j]);
    }
    if (c.grad_x.p) {
      inner = group_all<false>(inner, red[turn], at) * a.per_column * rstd;
      turn ^= 1;
      Pack<T, E>* out = reinterpret_cast<Pack<T, E>*>(static_cast<T*>(c.grad_x.p) +
                                                      n * c.grad_x.ld) + at.first;
#pragma unroll
      for (int j = 0; j < A; ++j) {
        if (at.first + j * at.step >= accesses) continue;
        memcpy(&s, from + j * pitch, 16);
        memcpy(&up, from + (A + j) * pitch, 16);
        if (c.grad_sum.p)
          memcpy(&more, from + (2 * A + j) * pitch, 16);
        else
          memset(&more, 0, 16);
        out[j * at.step] = grad_of_access<T, E>(s, up, more, g[j], rstd, inner);
      }
    }
    if (++stage == S) stage = 0;
  }
  if (c.grad_gain) store_partial<E, A>(a, acc, at);
}

// Rows of any length, read twice for grad_x and once more for the sums of grad_gain.

// grad_x, a row per CTA.
template <typename T>
__global__ void __launch_bounds__(kThreads) long_grad_x_kernel(const __grid_constant__ GradArgs a) {
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
    inner += Elem<T>::up(up[k]) * Elem<T>::up(gain[k]) * (Elem<T>::up(s[k]) * rstd);
  inner = block_all<false>(inner, red) * a.per_column * rstd;
  for (int k = threadIdx.x; k < a.K; k += kThreads) {
    float v = rstd * (Elem<T>::up(up[k]) * Elem<T>::up(gain[k])) - Elem<T>::up(s[k]) * rstd * inner;
    if (more) v += Elem<T>::up(more[k]);
    out[k] = Elem<T>::down(v);
  }
}

constexpr int kColumns = 32;
constexpr int kSubRows = kThreads / kColumns;

// Sums of grad_gain over every parts-th group of rows, 32 columns per CTA.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    long_gain_parts_kernel(const __grid_constant__ GradArgs a) {
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
           (Elem<T>::up(static_cast<const T*>(c.s.p)[n * c.s.ld + k]) * c.rstd[n]);
  sums[sub][threadIdx.x & 31] = v;
  __syncthreads();
  if (sub != 0 || k >= a.K) return;
  for (int i = 1; i < kSubRows; ++i) v += sums[i][threadIdx.x];
  a.partial[(size_t)part * a.K + k] = v;
}

constexpr int kJoinThreads = 512;

// The parts' sums, 32 columns per CTA, V of them a thread: each of the CTA's threads of
// a column adds up every subs-th part, in order, and 16 of them, then one, those sums. All of
// a thread's loads (at most 3 of the 152 parts, or 10) are under way at once.
template <typename T, int V>
__global__ void __launch_bounds__(kJoinThreads)
    gain_join_kernel(const __grid_constant__ GradArgs a) {
  constexpr int kLanes = 32 / V, kSubs = kJoinThreads / kLanes;
  __shared__ float sums[kSubs][33];
  wait_for_predecessor();
  let_successor_start();
  const int lane = threadIdx.x % kLanes, sub = threadIdx.x / kLanes;
  const int k = blockIdx.x * 32 + lane * V;
  float v[V] = {};
  if (k < a.K)
#pragma unroll(V == 4 ? 3 : 10)
    for (int p = sub; p < a.parts; p += kSubs) {
      const float* from = a.partial + (size_t)p * a.K + k;
      if constexpr (V == 4) {
        const float4 x = *reinterpret_cast<const float4*>(from);
        v[0] += x.x;
        v[1] += x.y;
        v[2] += x.z;
        v[3] += x.w;
      } else {
        v[0] += *from;
      }
    }
#pragma unroll
  for (int i = 0; i < V; ++i) sums[sub][lane * V + i] = v[i];
  __syncthreads();
  const int column = threadIdx.x / 16, part = threadIdx.x % 16;
  float total = 0.f;
#pragma unroll
  for (int i = 0; i < kSubs / 16; ++i) total += sums[part + 16 * i][column];
#pragma unroll
  for (int m = 8; m > 0; m >>= 1) total += __shfl_xor_sync(0xffffffffu, total, m);
  if (part != 0 || blockIdx.x * 32 + column >= a.K) return;
  T* out = static_cast<T*>(a.c.grad_gain) + blockIdx.x * 32 + column;
  if (a.c.accumulate) total += Elem<T>::up(*out);
  *out = Elem<T>::down(total);
}

// ---- launches ----------------------------------------------------------------------

constexpr size_t kRingMost = 220 * 1024;  // beside the kernels' static shared memory

// Groups of A accesses a thread, as many of them a CTA as `block` threads hold once every SM
// has a CTA; returns the CTAs that N rows take, at most per_sm on an SM where that is not 0.
template <int A>
unsigned lay_out(Shape& shape, int accesses, int N, int sms, int block, int per_sm) {
  shape.threads = (int)round_up(div_up(accesses, A), 32);
  long long groups = block / shape.threads;
  if (groups > N / sms) groups = N / sms;
  if (groups > 15) groups = 15;  // barriers of a CTA, beside its own
  shape.groups = groups < 1 ? 1 : (int)groups;
  const long long ctas = div_up(N, shape.groups), most = (long long)per_sm * sms;
  return (unsigned)(per_sm && ctas > most ? most : ctas);
}

template <typename T, int E, int A>
cudaError_t rows_as(const hg_norm& h, RowsArgs& a, cudaStream_t stream) {
  const unsigned grid = lay_out<A>(a.shape, a.K / E, a.c.N, h.sms, 128, 0);
  const unsigned block = (unsigned)(a.shape.threads * a.shape.groups);
  return a.c.e4m3 ? launch_dependent(rows_kernel<T, E, A, true>, a, grid, block, 0, 1, stream)
                  : launch_dependent(rows_kernel<T, E, A, false>, a, grid, block, 0, 1, stream);
}

// Rows in the ring and threads of an SM. Plain rows run at the copy rate with one group of
// 448 threads (8192 rows of 7168 bf16: 70 us, 79 with two groups); the 8-bit output's
// second round of maxima wants two (2048 rows: 25 and 19 us), and so does the gradient
// (4096 rows: 62 and 44 us).
constexpr int kStages = 3, kStagesQuant = 2;
constexpr int kRowThreads = 512;

template <typename T, int S, bool QUANT>
cudaError_t rows_stream(const hg_norm& h, RowsArgs& a, cudaStream_t stream) {
  const unsigned grid = lay_out<2>(a.shape, a.K / (16 / (int)sizeof(T)), a.c.N, h.sms,
                                   QUANT ? kMostThreads : kRowThreads, 1);
  const unsigned block = (unsigned)(a.shape.threads * a.shape.groups);
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
  if (accesses > LONG * kMostThreads)
    return launch_dependent(long_rows_kernel<T>, a, (unsigned)a.c.N, kThreads, 0, 1, stream);
  if (a.c.N <= h.sms && accesses <= kMostThreads) return rows_as<T, E, 1>(h, a, stream);
  if constexpr (kWide)
    return a.c.e4m3 ? rows_stream<T, kStagesQuant, true>(h, a, stream)
                    : rows_stream<T, kStages, false>(h, a, stream);
  else
    return rows_as<T, E, LONG>(h, a, stream);
}

template <typename T>
cudaError_t join_gain(const GradArgs& a, cudaStream_t stream) {
  const unsigned grid = (unsigned)div_up(a.K, 32);
  return a.K % 4 == 0
             ? launch_dependent(gain_join_kernel<T, 4>, a, grid, kJoinThreads, 0, 1, stream)
             : launch_dependent(gain_join_kernel<T, 1>, a, grid, kJoinThreads, 0, 1, stream);
}

template <typename T>
cudaError_t grad_of_long_rows(const hg_norm& h, GradArgs& a, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  if (a.c.grad_gain) {  // first: grad_x may be written over grad_out
    const long long parts = div_up(a.c.N, kSubRows);
    a.parts = parts < 1 ? 1 : parts < h.sms ? (int)parts : h.sms;
    const long long blocks = div_up(a.K, kColumns) * a.parts;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    e = launch_dependent(long_gain_parts_kernel<T>, a, (unsigned)blocks, kThreads, 0, 1, stream);
    if (e == cudaSuccess) e = join_gain<T>(a, stream);
  }
  if (e != cudaSuccess || !a.c.grad_x.p || a.c.N == 0) return e;
  return launch_dependent(long_grad_x_kernel<T>, a, (unsigned)a.c.N, kThreads, 0, 1, stream);
}

template <typename T, int E, int A>
cudaError_t grad_as(const hg_norm& h, GradArgs& a, cudaStream_t stream) {
  unsigned grid = lay_out<A>(a.shape, a.K / E, a.c.N, h.sms, kMostThreads, 1);
  if (grid < 1) grid = 1;  // no rows: zeros
  a.parts = (int)grid;
  const unsigned block = (unsigned)(a.shape.threads * a.shape.groups);
  if (!a.c.grad_gain)
    return launch_dependent(grad_kernel<T, E, A, false>, a, grid, block, 0, 1, stream);
  const size_t smem = a.shape.groups > 1 ? (size_t)a.shape.groups * a.K * sizeof(float) : 0;
  const cudaError_t e =
      launch_dependent(grad_kernel<T, E, A, true>, a, grid, block, smem, 1, stream);
  return e == cudaSuccess ? join_gain<T>(a, stream) : e;
}

template <typename T>
cudaError_t grad_stream(const hg_norm& h, GradArgs& a, cudaStream_t stream) {
  unsigned grid = lay_out<2>(a.shape, a.K / (16 / (int)sizeof(T)), a.c.N, h.sms, kMostThreads, 1);
  if (grid < 1) grid = 1;  // no rows: zeros
  a.parts = (int)grid;
  const unsigned block = (unsigned)(a.shape.threads * a.shape.groups);
  const size_t stage = (size_t)3 * 2 * block * 16;
  const cudaError_t e =
      3 * stage <= kRingMost
          ? launch_dependent(grad_stream_kernel<T, 2, 3>, a, grid, block, 3 * stage, 1, stream)
          : launch_dependent(grad_stream_kernel<T, 2, 2>, a, grid, block, 2 * stage, 1, stream);
  return e == cudaSuccess && a.c.grad_gain ? join_gain<T>(a, stream) : e;
}

constexpr int kFewRows = 64;

// Few rows take one launch, or few accesses a thread, as their latency counts; many rows
// in 16-byte accesses are streamed; others take A or twice as many accesses a thread. Whether
// grad_x is wanted, and over grad_out, changes nothing in the order of grad_gain's sum: of few
// rows grad_x is then made by a launch behind it.
template <typename T, int E, int A>
cudaError_t grad_by(const hg_norm& h, GradArgs& a, cudaStream_t stream) {
  const GradCall& c = a.c;
  const int accesses = a.K / E;
  if (c.N > 0 && c.N <= kFewRows && accesses <= kMostThreads && c.grad_gain) {
    const bool in_place = c.grad_x.p && c.grad_x.p == c.grad_out.p;
    GradArgs few = a;
    if (in_place) few.c.grad_x = {};
    few.shape = {(int)round_up(accesses, 32), 1};
    const unsigned block =
        few.shape.threads < 256 ? 256u : (unsigned)round_up(few.shape.threads, 64);
    const unsigned grid = (unsigned)((few.c.grad_x.p ? c.N : 0) + div_up(a.K, kFewColumns));
    const cudaError_t e = launch_dependent(few_kernel<T, E>, few, grid, block, 0, 1, stream);
    if (e != cudaSuccess || !in_place) return e;
    a.c.grad_gain = nullptr;
  }
  if (c.N <= h.sms && accesses <= kMostThreads) return grad_as<T, E, 1>(h, a, stream);
  if constexpr (E * sizeof(T) == 16) {
    if (accesses <= 2 * kMostThreads) return grad_stream<T>(h, a, stream);
  } else {
    if (accesses <= A * kMostThreads) return grad_as<T, E, A>(h, a, stream);
    if (accesses <= 2 * A * kMostThreads) return grad_as<T, E, 2 * A>(h, a, stream);
  }
  return grad_of_long_rows<T>(h, a, stream);
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

}  // namespace

cudaError_t prepare(const hg_norm& h) {
  return h.dtype == HG_BF16   ? prepare_as<__nv_bfloat16>()
         : h.dtype == HG_FP16 ? prepare_as<__half>()
                              : prepare_as<float>();
}

int grad_parts(const hg_norm& h) { return h.max_rows < h.sms ? h.max_rows : h.sms; }

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

cudaError_t rows_grad(const hg_norm& h, const GradCall& c, cudaStream_t stream) {
  GradArgs a = {c, h.K, 1.f / (float)h.K, {}, 1, h.partial};
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
