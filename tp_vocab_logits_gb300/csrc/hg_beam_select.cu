// Beam search's selection: the best continuations of each item.
//
// One pass over the logits, whose chunks are dealt out to the CTAs in order, the same number
// to each. A thread reads ahead of itself into a ring in shared memory, and of a part (what a
// CTA has of a row) keeps the largest logit and, where the logsumexp is wanted, the running
// maximum and sum of its exponentials: nothing that a chunk costs depends on the number of
// picks, and no warp waits for another. A second kernel, a CTA per item, joins the parts:
// with the rows' scores and logsumexps, the threads' best totals bound the item's n-th best
// from below, so only the threads that reach it, little more than n, have their elements read
// again (from L2) for the candidates. 32 items of 8 beams, 163840 logits, 16 picks: 22.3 us,
// 3.8 TB/s, of which the join's chain of dependent steps (sums, bound, elements, ranks) is 5 us;
// 20.2 us where the logsumexps are given. (Lists of the best that were kept up to date
// chunk by chunk, by CTA or by warp, took two to four times as long; joined by the last CTA of
// the first kernel, an item takes 12 to 20 us for 256 threads.)

#include <cmath>
#include <cstring>

#include "hg_beam.cuh"

namespace hg {
namespace beam {
namespace {

using vocab::Elem;
using vocab::div_up;
using vocab::launch_dependent;
using vocab::let_successor_start;
using vocab::wait_for_predecessor;

typedef unsigned long long u64;

constexpr int kLogThreads = 8;
static_assert(1 << kLogThreads == kThreads, "groups of threads are counted in powers of two");
constexpr int kStages = 2;       // chunks in the ring
constexpr int kMostJoinWarps = 32;
constexpr int kList = 1024;      // candidates of an item that are ranked at once
constexpr int kRanked = 128;     // that are ranked as they are: ranking takes their square
constexpr int kHits = 512;       // groups of threads whose elements are read again
constexpr int kRounds = 4;       // of closer bounds, where there are more of either
constexpr int kCtasPerSm = 4;
// Maxima that a thread of join_kernel takes. Many picks have many elements read again, of
// groups that are finer where there are more of them (163840 logits, an item of 64 beams with 128
// picks: 48 and 35 us; 8 items of 8 with 16: 11.9 and 14.0). Many parts need the room, or a part's
// threads share few maxima (an item of 32 beams with 32 picks: 21 and 17).
constexpr int kFewValues = 4, kManyValues = 16;
constexpr int kFewPicks = 32;
constexpr int kLeastGroups = 8;    // of a part's threads, at least, that have a maximum: warps
constexpr float kLog2e = 1.44269504088896341f;
constexpr double kLn2 = 0.693147180559945309417;
constexpr double kLog2eOff = 1.0 - (double)kLog2e * kLn2;

constexpr int kNone = 255;

struct SelectArgs {
  SelectCall c;
  int beams, vocab, picks;
  int chunks;          // of a row
  int each, more;      // chunks of a CTA; the first `more` CTAs have one more
  Divisor by_chunks, by_each, by_each_and_one, by_beams, by_longest;
  int all;             // chunks of the call
  int longest;         // chunks of a part, at most
  int log_groups;      // groups of a CTA's threads that have a maximum each
  float* maxima;       // [part][groups]
  float2* stats;       // [part][warp]
  int* beam_of;        // [part], kNone where it is not searched or there is no such part
  u64* list;           // [row][picks], of pick_exactly
  __device__ int first_chunk(int cta) const { return min(cta * each + min(cta, more), all); }
  __device__ int cta_of(int chunk) const {
    const int front = more * (each + 1);
    return chunk < front ? by_each_and_one.divide(chunk) : more + by_each.divide(chunk - front);
  }
  // The number of what a CTA has of a row: going through the chunks, each new part raises the
  // CTA, the row, or both.
  __device__ int part_of(int cta, int row) const { return cta + row; }
};

// Bits of a value that is no NaN, in an order of unsigned integers; both zeros alike.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}
// (64-bit arithmetic is slow: the bits are looked at.)
__device__ __forceinline__ u64 ordered(double v) {
  const u64 u = (u64)__double_as_longlong(v);
  return u >> 63 && u << 1 ? ~u : u | 1ull << 63;
}
__device__ __forceinline__ double unordered(u64 u) {
  return __longlong_as_double((long long)(u >> 63 ? u & ~(1ull << 63) : ~u));
}
// Whether it is a number that is not -inf in fp32, to which half a unit beyond the largest
// number rounds.
__device__ __forceinline__ bool counts(double v) {
  const u64 u = (u64)__double_as_longlong(v), size = u & ~(1ull << 63);
  return size <= 0x7ff0000000000000ull && !(u >> 63 && size >= 0x47effffff0000000ull);
}

// Larger keys are better candidates of a row; 0 is none.
__device__ __forceinline__ u64 key_of(float x, int token) {
  return (u64)ordered(x) << 32 | (uint32_t)~token;
}

__device__ __forceinline__ float exp2_of(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 operations in one instruction.
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
__device__ __forceinline__ u64 add2(u64 a, u64 b) {
  u64 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// A row whose logits count.
__device__ __forceinline__ bool searched(const SelectCall& c, size_t row) {
  return c.scores[row] > -INFINITY && !(c.finished && c.finished[row]);
}

// Copies 16 bytes into shared memory, where the thread reads them once its copies are there.
__device__ __forceinline__ void copy_ahead(uint4* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(to)),
               "l"(from)
               : "memory");
}
__device__ __forceinline__ void close_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits for all but the last N groups of this thread's copies.
template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// 16 bytes of logits.
template <typename T>
struct Access {
  static constexpr int E = 16 / sizeof(T);
  uint4 w;

  // Elements [e0, e0 + E) of a row of `vocab`; those that lie outside are -inf, and are not
  // read (others are in their place, so that no load waits for a branch).
  static __device__ __forceinline__ Access edge(const T* row, int e0, int vocab) {
    T v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = Elem<T>::down(-INFINITY);
    if (e0 + E > 0 && e0 < vocab) {
      T x[E];
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = row[min(max(e0 + e, 0), vocab - 1)];
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (e0 + e >= 0 && e0 + e < vocab) v[e] = x[e];
    }
    Access a;
    memcpy(&a.w, v, 16);
    return a;
  }
  static __device__ __forceinline__ bool inside(int e0, int vocab) {
    return e0 >= 0 && e0 + E <= vocab;
  }
  __device__ void widen(float (&v)[E]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    if constexpr (E == 8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = Elem<T>::unpack2(u[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(u[i]);
    }
  }
};

__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b, __nv_bfloat16) {
  uint32_t w;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(w) : "r"(a), "r"(b));
  return w;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b, __half) {
  uint32_t w;
  asm("max.f16x2 %0, %1, %2;" : "=r"(w) : "r"(a), "r"(b));
  return w;
}

// The largest element that is not NaN (-inf or NaN if there is none).
template <typename T, int R>
__device__ __forceinline__ float largest(const Access<T> (&x)[R]) {
  if constexpr (sizeof(T) == 2) {
    uint32_t m = x[0].w.x;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m = max2(m, max2(max2(x[r].w.x, x[r].w.y, T{}), max2(x[r].w.z, x[r].w.w, T{}), T{}), T{});
    }
    const float2 f = Elem<T>::unpack2(m);
    return fmaxf(f.x, f.y);
  } else {
    float m = -INFINITY;
#pragma unroll
    for (int r = 0; r < R; ++r)
      m = fmaxf(fmaxf(fmaxf(m, __uint_as_float(x[r].w.x)), __uint_as_float(x[r].w.y)),
                fmaxf(__uint_as_float(x[r].w.z), __uint_as_float(x[r].w.w)));
    return m;
  }
}

// Sum of 2^(log2e x - shift) by thread, shift = rint(log2e most): as it is whole, one rounding
// is in each exponent, and rescaling is exact. `most` need not be the maximum: it follows
// where that is kRise above it (to rescale at every new maximum took a third of the
// instructions). From kHuge on, where neighbours are further apart than exponentials reach, the
// largest elements count one each. NaN and +inf give NaN.
// (An exponent of up to 58 is off by up to 2^-19, 1.3e-6 of its exponential. With sums of up
// to 3 / 1024 of the row's elements one after another the logsumexp is off by at most 2^-17 +
// vocab * 2^-32; 5e-7 measured, rows of 1000 to a million logits.)
constexpr float kHuge = 1e30f;
constexpr float kRise = 40.f;  // 2^58

struct Exponentials {
  float most = -INFINITY, sum = 0.f;
  float limit = -INFINITY;  // up to which logits are added as they are

  static __device__ __forceinline__ bool plain(float most) {
    return fabsf(most) < kHuge || most == -INFINITY;
  }
  static __device__ __forceinline__ float shift(float most) {
    return most > -INFINITY ? rintf(most * kLog2e) : 0.f;
  }
  // What a sum with the maximum `most` counts under a maximum of `top`, not below it.
  static __device__ __forceinline__ float weight(float most, float top) {
    if (most == -INFINITY || most == top) return 1.f;
    return plain(most) && plain(top) ? exp2_of(shift(most) - shift(top)) : 0.f;
  }
  __device__ __forceinline__ void raise(float top) {
    if (!(top > most)) return;
    sum *= weight(most, top);
    most = top;
  }
  template <typename T>
  static __device__ __noinline__ float count_huge(const uint4* ring, int accesses, float most) {
    float c = 0.f;
    for (int i = 0; i < accesses * Access<T>::E; ++i) {
      const T* v = reinterpret_cast<const T*>(ring + i / Access<T>::E * kThreads);
      c += exp2_of((Elem<T>::up(v[i % Access<T>::E]) - most) * kLog2e);
    }
    return c;
  }
  // x[r] is in ring[r * kThreads] too.
  template <typename T, int R>
  __device__ __forceinline__ void add(const Access<T> (&x)[R], const uint4* ring,
                                      float chunk_most) {
    if (!(chunk_most <= limit)) {
      raise(chunk_most);
      limit = plain(most) ? most + kRise : most;
    }
    if (!plain(most)) {
      sum += count_huge<T>(ring, R, most);
      return;
    }
    const float s = shift(most);
    const u64 scale = pair(kLog2e, kLog2e), back = pair(-s, -s);
    u64 sums[2] = {pair(sum, 0.f), 0};
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float v[Access<T>::E];
      x[r].widen(v);
#pragma unroll
      for (int e = 0; e < Access<T>::E; e += 2) {
        const u64 p = fma2(pair(v[e], v[e + 1]), scale, back);
        sums[e / 2 % 2] = add2(sums[e / 2 % 2], pair(exp2_of(low(p)), exp2_of(high(p))));
      }
    }
    const u64 both = add2(sums[0], sums[1]);
    sum = low(both) + high(both);
  }
};

constexpr float kLeast = -3.402823466e38f;

constexpr int kLogGroupings = 5;  // at least 32 groups of a CTA's threads

struct BoundShared {
  uint32_t word[kMostJoinWarps][33];
  uint32_t top[2 * HG_MAX_PICKS];
  uint32_t bound;
};

// A word that at least n of the threads' words (0: none) are not under, and not many more: the n-th largest of the maxima of groups of threads, twice n of them (which
// 1.4 n words reach where they are in any order). A group takes one thread from each of some
// warps, another lane of every one: warps apart and other lanes, as neighbours are of one beam.
// 0 if there are not n.
template <int WARPS>
__device__ __forceinline__ uint32_t bound_of_best(int n, uint32_t word, BoundShared& s) {
  constexpr unsigned kAll = 0xffffffffu;
  constexpr int kThreadsHere = WARPS * 32;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int log_groups = max(kLogGroupings, 32 - __clz(2 * n - 1));
  static_assert(2 * HG_MAX_PICKS <= 256, "no more groups than threads");
  s.word[warp][(lane + warp * 5 + warp / 8) & 31] = word;
  __syncthreads();
  const int width = kThreadsHere >> log_groups;  // threads of a group
  // Warps as far apart as they can be.
  uint32_t top = s.word[tid % width * (WARPS / width) + tid % WARPS / width][tid / WARPS];
  if (width == 32) top = __reduce_max_sync(kAll, top);
  else for (int m = 1; m < width; m <<= 1) top = max(top, __shfl_xor_sync(kAll, top, m));
  const int group = tid / width, turn = tid % width;
  if (turn == 0) s.top[group] = top;
  __syncthreads();
  int rank = 0;
  for (int i = turn; i < 1 << log_groups; i += width) {
    const uint32_t other = s.top[i];
    rank += other > top || (other == top && i < group);
  }
  if (width == 32) rank = __reduce_add_sync(kAll, rank);
  else for (int m = 1; m < width; m <<= 1) rank += __shfl_xor_sync(kAll, rank, m);
  if (turn == 0 && rank == n - 1) s.bound = top;
  __syncthreads();
  return s.bound;
}

// ---- a row -------------------------------------------------------------------------

// A row, as the threads of a CTA have it.
template <typename T, int R>
struct Row {
  static constexpr int E = Access<T>::E;
  const T* row;
  int vocab;

  __device__ __forceinline__ int shift() const {
    return (int)(reinterpret_cast<uintptr_t>(row) % 16 / sizeof(T));
  }
  // The first element of a thread's access k of chunk i.
  __device__ __forceinline__ int element(int thread, int i, int k) const {
    return ((i * R + k) * kThreads + thread) * E - shift();
  }
  // Calls f(logit, token) for the elements of a thread from `least` (above -inf) on, in chunk i.
  template <typename F>
  __device__ __forceinline__ void each(int thread, int i, float least, F f) const {
    uint32_t mask = 0;
    Access<T> x[R];  // all loads before the first use
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int e0 = element(thread, i, k);
      if (Access<T>::inside(e0, vocab))
        x[k].w = *reinterpret_cast<const uint4*>(row + e0);
      else
        x[k] = Access<T>::edge(row, e0, vocab);
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
      float v[E];
      x[k].widen(v);
#pragma unroll
      for (int e = 0; e < E; ++e) mask |= v[e] >= least ? 1u << (k * E + e) : 0u;
    }
    for (; mask; mask &= mask - 1) {
      const int m = __ffs(mask) - 1, at = element(thread, i, m / E) + m % E;
      f(Elem<T>::up(row[at]), at);
    }
  }
};

// ---- joining an item's parts -------------------------------------------------------

struct JoinShared {
  u64 total[kList], key[kList];
  unsigned char beam[kList];
  int hit[kHits];  // groups of threads whose largest logit reaches the bound, and their beams
  BoundShared bound;
  double lse[HG_MAX_BEAMS], score_64[HG_MAX_BEAMS];
  float score[HG_MAX_BEAMS];
  float near[HG_MAX_BEAMS];  // score - logsumexp in fp32
  bool done[HG_MAX_BEAMS];   // finished, and still a candidate
  uint32_t largest[2];       // magnitude of near, below kHuge, as bits
  bool reaches[HG_MAX_BEAMS];  // the bound, by a logit
  int warp_count[2][kMostJoinWarps];
  double top_total[kMostJoinWarps];
  u64 top_key[kMostJoinWarps];
  int top_beam[kMostJoinWarps];
  int hits, count;

  // The total of a beam's logit, as it is compared.
  __device__ __forceinline__ double sum(int b, float x) const {
    return score_64[b] + ((double)x - lse[b]);
  }
  // The same to within `off` of it in fp32 (64-bit additions are slow, and few candidates
  // come near the best).
  __device__ __forceinline__ float nearly(int b, float x) const {
    const float t = x + near[b];
    return fabsf(near[b]) < kHuge && fabsf(t) < kHuge ? t : exactly(b, x);
  }
  // Not inlined: it would be computed for every value, to be thrown away (8000 cycles an item).
  __device__ __noinline__ float exactly(int b, float x) const { return (float)sum(b, x); }
  // Three roundings of at most half a unit in the last place of the two terms and of the sum.
  __device__ __forceinline__ float off(float t) const {
    const float most = __uint_as_float(max(largest[0], largest[1]));
    return fabsf(t) < INFINITY ? 3.f * 5.9604645e-8f * (most + fabsf(t)) : 0.f;
  }
  // Lists a group of threads, the `place`-th that an item has.
  __device__ __forceinline__ void note(int b, int place) {
    reaches[b] = true;
    const int at = atomicAdd(&hits, 1);
    if (at < kHits) hit[at] = b << 16 | place;
  }
  // Lists a candidate that fp32 can tell from -inf.
  __device__ __noinline__ void add(double t, int b, u64 k) {
    if (!counts(t)) return;
    const int at = atomicAdd(&count, 1);
    if (at >= kList) return;
    total[at] = ordered(t);
    key[at] = k;
    beam[at] = (unsigned char)b;
  }
};

// A candidate of an item, in the order of the picks.
struct Candidate {
  double total;
  int beam;  // -1: none
  u64 key;
  __device__ bool before(const Candidate& o) const {
    if (beam < 0 || o.beam < 0) return o.beam < 0 && beam >= 0;
    if (total != o.total) return total > o.total;
    if (beam != o.beam) return beam < o.beam;
    return key > o.key;
  }
};

__device__ __forceinline__ void put_id(void* p, int bytes, size_t i, int v) {
  if (bytes == 8)
    static_cast<long long*>(p)[i] = v;
  else
    static_cast<int*>(p)[i] = v;
}

__device__ __forceinline__ void put_pick(const SelectArgs& a, const JoinShared& s, int item,
                                         int rank, bool there, double total, int beam, u64 key) {
  const SelectCall& c = a.c;
  const size_t at = (size_t)item * a.picks + rank;
  const int token = there ? (int)~(uint32_t)key : -1;
  put_id(c.tokens, c.id_bytes, at, token);
  put_id(c.parents, c.id_bytes, at, there ? beam : -1);
  c.picked[at] = there ? (float)total : -INFINITY;
  if (c.picked_finished)
    c.picked_finished[at] =
        there && (token == c.end || s.done[beam]);
}

// a + b, and what the rounding left out.
__device__ __forceinline__ float2 two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return make_float2(s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t)));
}

// What parts' warps have of a row's exponentials, by one warp.
struct RowStats {
  static constexpr int kOfLane = 4;
  int first, all;  // the row's, of all that there are
  float2 v[kOfLane];

  __device__ __forceinline__ void enter(const SelectArgs& a, int row) {
    const int part0 = a.part_of(a.cta_of(row * a.chunks), row);
    first = part0 * kWarps;
    all = (a.part_of(a.cta_of((row + 1) * a.chunks - 1), row) - part0 + 1) * kWarps;
  }
  __device__ __forceinline__ void load(const SelectArgs& a, int from) {
#pragma unroll
    for (int k = 0; k < kOfLane; ++k) {
      const int i = from + k * 32 + (threadIdx.x & 31);
      v[k] = i < all ? __ldcg(a.stats + first + i) : make_float2(-INFINITY, 0.f);
    }
  }
  // The row's logsumexp, as hi + lo; the first values are loaded.
  __device__ __forceinline__ float2 lse(const SelectArgs& a) {
    float most = -INFINITY, sum = 0.f;
    for (int from = 0;;) {
      float top = most;
#pragma unroll
      for (int k = 0; k < kOfLane; ++k) top = fmaxf(top, v[k].x);
      top = unordered(__reduce_max_sync(0xffffffffu, ordered(top)));
      sum *= Exponentials::weight(most, top);
#pragma unroll
      for (int k = 0; k < kOfLane; ++k) sum += v[k].y * Exponentials::weight(v[k].x, top);
      most = top;
      from += kOfLane * 32;
      if (from >= all) break;
      load(a, from);
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    if (!(sum < INFINITY)) return make_float2(sum, 0.f);  // NaN
    if (!Exponentials::plain(most)) return make_float2(most, 0.f);
    if (!(sum > 0.f)) return make_float2(-INFINITY, 0.f);
    int exponent = 0;
    float f = frexpf(sum, &exponent);  // in [0.5, 1)
    if (f < 0.70710678f) {
      f *= 2.f;
      --exponent;
    }
    // The logarithm of the powers of two is a sum of two numbers, that of the mantissa, below
    // 0.35, one. kLog2e is 1 - kLog2eOff times log2(e): its share of the logits, nearly the
    // largest one's.
    constexpr float kHi = (float)kLn2, kLo = (float)(kLn2 - (double)kHi);
    const float n = Exponentials::shift(most), e = (float)exponent;
    const float p = __fmul_rn(n, kHi), q = __fmul_rn(e, kHi);
    const float2 first = two_sum(p, q), second = two_sum(first.x, logf(f));
    const float lo = fmaf(n, kHi, -p) + fmaf(e, kHi, -q) + first.y + second.y + (n + e) * kLo +
                     most * (float)kLog2eOff;
    return two_sum(second.x, lo);
  }
};

// Over the CTA's threads, the same value in each. One barrier orders a call's writes before its
// reads; the next call writes while others may still read this one's, so `turn`, which has to
// be another than the call before had, says which of two places is used.
template <int WARPS>
__device__ __forceinline__ int count_all(int c, int turn, JoinShared& s) {
  c = __reduce_add_sync(0xffffffffu, c);
  if ((threadIdx.x & 31) == 0) s.warp_count[turn][threadIdx.x >> 5] = c;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  return __reduce_add_sync(0xffffffffu, lane < WARPS ? s.warp_count[turn][lane] : 0);
}

// Where too many candidates are alike for the list: the best of each row that has some,
// exactly (the key of the n-th best, one bit after another, reading the row again for each),
// and of those one pick after another. About 1.3 ms a row of 163840 equal logits, the rows of an
// item one after another; 1.5 ms for 32 items of 8 beams of which all but one are out by a score
// of -1e9, whose magnitude is in every total's bound (JoinShared::off; 27 us with -inf).
template <typename T, int R, int THREADS>
__device__ __noinline__ void pick_exactly(const SelectArgs& a, int item, JoinShared& s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int thread = threadIdx.x % kThreads, first = threadIdx.x / kThreads;
  constexpr int kStep = THREADS / kThreads;
  const int row0 = item * a.beams, n = a.picks;
  int turn = 0;
  for (int b = 0; b < a.beams; ++b) {
    u64* list = a.list + (size_t)(row0 + b) * n;
    for (int i = threadIdx.x; i < n; i += THREADS) list[i] = 0;
    if (!s.reaches[b]) continue;
    const Row<T, R> one = {static_cast<const T*>(a.c.logits) + (size_t)(row0 + b) * a.c.ld,
                             a.vocab};
    // All tokens' complements have the bits above the vocabulary's.
    const int low = 32 - __clz(a.vocab);
    u64 bound = 0;
    for (int bit = 63; bit >= 0; --bit) {
      if (bit == 31) {
        bound |= ~0u << low;
        bit = low - 1;
      }
      const u64 next = bound | 1ull << bit;
      int c = 0;
      for (int i = first; i < a.chunks; i += kStep)
        one.each(thread, i, kLeast, [&](float x, int token) { c += key_of(x, token) >= next; });
      c = count_all<THREADS / 32>(c, turn ^= 1, s);  // not the bit's parity: bits are skipped
      if (c >= n) bound = next;
      if (c == n) break;
    }
    __syncthreads();
    if (threadIdx.x == 0) s.count = 0;
    __syncthreads();
    for (int i = first; i < a.chunks; i += kStep)
      one.each(thread, i, kLeast, [&](float x, int token) {
        if (key_of(x, token) < bound) return;
        const int at = atomicAdd(&s.count, 1);
        if (at < n) list[at] = key_of(x, token);
      });
  }
  __syncthreads();  // the lists are this CTA's own
  const int listed = a.beams * n, all = listed + (a.c.finished ? a.beams : 0);
  Candidate under;
  for (int i = 0; i < n; ++i) {
    Candidate top;
    top.beam = -1;
    for (int j = threadIdx.x; j < all; j += THREADS) {
      Candidate t;
      if (j < listed) {
        t.beam = j / n;
        t.key = a.list[(size_t)row0 * n + j];
        if (!t.key) continue;
        t.total = s.sum(t.beam, unordered((uint32_t)(t.key >> 32)));
      } else {
        t.beam = j - listed;
        t.key = (uint32_t)~a.c.end;
        if (!s.done[t.beam]) continue;
        t.total = s.score[t.beam];
      }
      if (!counts(t.total)) continue;
      if ((i == 0 || under.before(t)) && t.before(top)) top = t;
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) {
      Candidate o;
      o.total = __shfl_xor_sync(0xffffffffu, top.total, m);
      o.beam = __shfl_xor_sync(0xffffffffu, top.beam, m);
      o.key = __shfl_xor_sync(0xffffffffu, top.key, m);
      if (o.before(top)) top = o;
    }
    __syncthreads();
    if (lane == 0) {
      s.top_total[warp] = top.total;
      s.top_beam[warp] = top.beam;
      s.top_key[warp] = top.key;
    }
    __syncthreads();
    for (int w = 0; w < (THREADS / 32); ++w) {
      const Candidate o = {s.top_total[w], s.top_beam[w], s.top_key[w]};
      if (o.before(top)) top = o;
    }
    under = top;  // once none, nothing comes after it
    if (threadIdx.x == 0) put_pick(a, s, item, i, top.beam >= 0, top.total, top.beam, top.key);
  }
}

// Lists the elements of the listed groups whose totals may reach the bound, a thread's of a
// chunk each.
template <typename T, int R, int THREADS>
__device__ __forceinline__ void collect(const SelectArgs& a, int row0, int part0, float from,
                                        JoinShared& s) {
  const int log_width = kLogThreads - a.log_groups;
  const unsigned units = (unsigned)(min(s.hits, kHits) * a.longest) << log_width;
  for (unsigned u = threadIdx.x; u < units; u += THREADS) {
    const int pair = (int)(u >> log_width), h = a.by_longest.divide(pair);
    const int hit = s.hit[h], b = hit >> 16, in = hit & 0xffff;
    const int part = in >> a.log_groups, group = in - (part << a.log_groups);
    // What the group has of the row.
    const int row = row0 + b, begin = row * a.chunks;
    const int first = max(begin, a.first_chunk(part0 + part - row));
    const int last = min(begin + a.chunks, a.first_chunk(part0 + part - row + 1));
    const int chunk = first + pair - h * a.longest;
    if (chunk >= last) continue;
    const Row<T, R> whole = {static_cast<const T*>(a.c.logits) + (size_t)row * a.c.ld, a.vocab};
    // From which logit on a total may reach the bound: well below it.
    const float least = from - s.near[b];
    const bool plain = fabsf(s.near[b]) < kHuge && fabsf(least) < kHuge;
    whole.each((group << log_width) + (int)(u & ((1 << log_width) - 1)), chunk - begin,
               plain ? least - 4.f * s.off(fabsf(from) + fabsf(least)) : kLeast,
               [&](float x, int token) {
                 const float t = s.nearly(b, x);
                 if (t + s.off(t) >= from) s.add(s.sum(b, x), b, key_of(x, token));
               });
  }
}

// Where there are too many, as where the best are neighbours: of those that are listed the n-th
// best is a closer bound, if they are not alike. Returns whether all fit then. (Logits that fall
// with the token, an item of 32 beams with 32 picks: 14.6 ms by pick_exactly, 38 us so.)
template <typename T, int R, int THREADS>
__device__ __noinline__ bool narrow(const SelectArgs& a, int row0, int part0, int listed,
                                    float from, JoinShared& s) {
  const float* maxima = a.maxima + ((size_t)part0 << a.log_groups);
  for (int round = 0; round < kRounds; ++round) {
    uint32_t top = 0;
    for (int i = threadIdx.x; i < min(s.count, kList); i += THREADS)
      top = max(top, (uint32_t)(s.total[i] >> 32));
    const uint32_t bound = bound_of_best<THREADS / 32>(a.picks, top, s.bound);
    float next = bound ? (float)unordered((u64)bound << 32) : kLeast;
    next -= s.off(next);
    if (!(next > from)) return false;
    from = next;
    if (threadIdx.x == 0) s.hits = s.count = 0;
    __syncthreads();
    if ((int)threadIdx.x < a.beams && s.done[threadIdx.x] && s.score[threadIdx.x] >= from)
      s.add(s.score[threadIdx.x], threadIdx.x, (uint32_t)~a.c.end);
    for (int i = threadIdx.x; i < listed; i += THREADS) {
      const float value = __ldcg(maxima + i);
      const int b = __ldcg(a.beam_of + part0 + (i >> a.log_groups));
      if (b == kNone || !(value > -INFINITY)) continue;
      const float t = s.nearly(b, value);
      if (t + s.off(t) >= from) s.note(b, i);
    }
    __syncthreads();
    collect<T, R, THREADS>(a, row0, part0, from, s);
    __syncthreads();
    if (s.hits <= kHits && s.count <= kList) return true;
  }
  return false;
}

template <typename T, int R, int THREADS, int VALUES>
__global__ void __launch_bounds__(THREADS, 1) join_kernel(const __grid_constant__ SelectArgs a) {
  __shared__ JoinShared s;
  const SelectCall& c = a.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int item = blockIdx.x, row0 = item * a.beams, row_last = row0 + a.beams - 1;
  const int part0 = a.part_of(a.cta_of(row0 * a.chunks), row0);
  const int parts = a.part_of(a.cta_of((row_last + 1) * a.chunks - 1), row_last) - part0 + 1;
  const int listed = parts << a.log_groups;
  const float* maxima = a.maxima + ((size_t)part0 << a.log_groups);
  RowStats stats;
  const bool sums = !c.lse && warp < a.beams;
  if (sums) stats.enter(a, row0 + warp);
  wait_for_predecessor();
  let_successor_start();
  constexpr int kValues = VALUES + 1;  // the last is a finished beam's score
  float value[kValues];
  int beam[kValues];
#pragma unroll
  for (int k = 0; k < kValues - 1; ++k) {
    const int i = min((int)threadIdx.x + k * THREADS, listed - 1);
    value[k] = __ldcg(maxima + i);
    beam[k] = __ldcg(a.beam_of + part0 + (i >> a.log_groups));
  }
  if (sums) stats.load(a, 0);
  // How large the terms of a total are at most, for its rounding.
  auto magnitude = [](float near) { return fabsf(near) < kHuge ? __float_as_uint(fabsf(near)) : 0u; };
  uint32_t most = 0;
  value[kValues - 1] = -INFINITY;
  if ((int)threadIdx.x < a.beams) {
    const int b = threadIdx.x, row = row0 + b;
    const float score = c.scores[row];
    const bool done = c.finished && c.finished[row] && score > -INFINITY;
    const float lse = c.lse ? c.lse[row * c.lse_stride] : 0.f;
    const float near = score - lse;
    s.score[b] = score;
    s.score_64[b] = (double)score;
    s.done[b] = done;
    s.lse[b] = (double)lse;
    s.near[b] = near;
    s.reaches[b] = false;
    if (done) value[kValues - 1] = score;
    most = magnitude(near);
  }
  if (threadIdx.x == 0) s.hits = s.count = 0;
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 0 && warp < 2) s.largest[warp] = most;
  static_assert(HG_MAX_BEAMS <= 64, "two warps have the beams");
  static_assert(THREADS * VALUES <= 1 << 16, "a hit's place and beam are a word");
  __syncthreads();
  if (!c.lse) {
    for (int b = warp; b < a.beams; b += THREADS / 32) {
      if (!(s.score[b] > -INFINITY) || s.done[b]) continue;
      if (b != warp) {
        stats.enter(a, row0 + b);
        stats.load(a, 0);
      }
      const float2 lse = stats.lse(a);
      if (lane == 0) {
        const float2 d = two_sum(s.score[b], -lse.x);
        const float near = fabsf(d.x) < kHuge ? d.x + (d.y - lse.y) : d.x;
        s.lse[b] = (double)lse.x + (double)lse.y;
        s.near[b] = near;
        atomicMax(&s.largest[0], magnitude(near));
      }
    }
    __syncthreads();
  }

  // The groups' best totals, nearly, and the word of the best of them from below.
  float best = -INFINITY;
#pragma unroll
  for (int k = 0; k < kValues; ++k) {
    float t = value[k];
    if (k < kValues - 1) {
      const bool there = (int)threadIdx.x + k * THREADS < listed && beam[k] != kNone;
      t = there && t > -INFINITY ? s.nearly(beam[k], t) : -INFINITY;
    }
    value[k] = t;
    best = fmaxf(best, t);
  }
  const uint32_t word = best > -INFINITY ? ordered(best - s.off(best)) : 0;
  const uint32_t bound = bound_of_best<THREADS / 32>(a.picks, word, s.bound);
  const float from = bound < ordered(kLeast) ? kLeast : unordered(bound);
#pragma unroll
  for (int k = 0; k < kValues; ++k) {
    if (!(best + s.off(best) >= from)) break;
    if (!(value[k] + s.off(value[k]) >= from)) continue;
    if (k == kValues - 1)
      s.add(value[k], threadIdx.x, (uint32_t)~c.end);
    else
      s.note(beam[k], threadIdx.x + k * THREADS);
  }
  __syncthreads();
  collect<T, R, THREADS>(a, row0, part0, from, s);
  __syncthreads();
  if ((s.hits > kHits || s.count > kList) &&
      !narrow<T, R, THREADS>(a, row0, part0, listed, from, s)) {
    pick_exactly<T, R, THREADS>(a, item, s);
    return;
  }
  int found = s.count;
  if (found > kRanked && found > 2 * a.picks) {
    // Of too many those whose totals' upper words reach the n-th best one's.
    constexpr int kOwn = kList / THREADS;
    u64 total[kOwn], key[kOwn];
    int of[kOwn];
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < kOwn; ++k) {
      const int i = threadIdx.x + k * THREADS;
      total[k] = i < found ? s.total[i] : 0;
      key[k] = s.key[i];
      of[k] = s.beam[i];
      top = max(top, (uint32_t)(total[k] >> 32));
    }
    const uint32_t least = bound_of_best<THREADS / 32>(a.picks, top, s.bound);
    if (threadIdx.x == 0) s.count = 0;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kOwn; ++k) {
      if (total[k] == 0 || (uint32_t)(total[k] >> 32) < least) continue;
      const int at = atomicAdd(&s.count, 1);
      s.total[at] = total[k];
      s.key[at] = key[k];
      s.beam[at] = (unsigned char)of[k];
    }
    __syncthreads();
    found = s.count;
  }
  // Each candidate's rank; eight lanes count what comes before it.
  const int eighth = threadIdx.x % 8;
  for (int i0 = warp * 4; i0 < found; i0 += THREADS / 8) {
    const int i = i0 + lane / 8;
    const bool there = i < found;
    const u64 total = there ? s.total[i] : ~0ull, key = there ? s.key[i] : ~0ull;
    const int b = there ? s.beam[i] : 0;
    int rank = 0;
#pragma unroll 4
    for (int j = eighth; j < found; j += 8) {
      const u64 t = s.total[j], k = s.key[j];
      const int o = s.beam[j];
      rank += (t > total) | ((t == total) & ((o < b) | ((o == b) & (k > key))));
    }
#pragma unroll
    for (int m = 4; m > 0; m >>= 1) rank += __shfl_xor_sync(0xffffffffu, rank, m);
    if (there && eighth == 0 && rank < a.picks) {
      put_pick(a, s, item, rank, true, unordered(total), b, key);
    }
  }
  for (int i = found + threadIdx.x; i < a.picks; i += THREADS)
    put_pick(a, s, item, i, false, 0.0, -1, 0);
}

template <typename T, int R>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    select_kernel(const __grid_constant__ SelectArgs a) {
  constexpr int E = Access<T>::E;
  extern __shared__ uint4 ring[];  // [stage][R][threads]: a thread reads what it copied
  wait_for_predecessor();
  let_successor_start();
  const int g0 = a.first_chunk(blockIdx.x), g1 = a.first_chunk(blockIdx.x + 1);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

  // The chunk that is copied next, and its row (null: its logits do not count).
  int ahead = g0, ahead_row = a.by_chunks.divide(g0), ahead_chunk = g0 - ahead_row * a.chunks;
  const T* ahead_at = nullptr;
  auto enter = [&](int row) {
    return searched(a.c, (size_t)row) ? static_cast<const T*>(a.c.logits) + (size_t)row * a.c.ld
                                      : nullptr;
  };
  auto copy = [&](int stage) {
    if (ahead < g1) {
      if (ahead_chunk == 0 || ahead == g0) ahead_at = enter(ahead_row);
      if (ahead_at) {
        const int shift = (int)(reinterpret_cast<uintptr_t>(ahead_at) % 16 / sizeof(T));
        const int e0 = ahead_chunk * (kThreads * R * E) - shift;
        uint4* to = ring + stage * R * kThreads + threadIdx.x;
        if (e0 >= 0 && e0 + kThreads * R * E <= a.vocab) {
          const uint4* from = reinterpret_cast<const uint4*>(ahead_at + e0) + threadIdx.x;
#pragma unroll
          for (int k = 0; k < R; ++k) copy_ahead(to + k * kThreads, from + k * kThreads);
        } else {
#pragma unroll 1
          for (int k = 0; k < R; ++k) {
            const int e = e0 + (k * kThreads + (int)threadIdx.x) * E;
            if (Access<T>::inside(e, a.vocab))
              copy_ahead(to + k * kThreads, ahead_at + e);
            else
              to[k * kThreads] = Access<T>::edge(ahead_at, e, a.vocab).w;
          }
        }
      }
      ++ahead;
      if (++ahead_chunk == a.chunks) {
        ahead_chunk = 0;
        ++ahead_row;
      }
    }
    close_copies();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) copy(i);
  int row = a.by_chunks.divide(g0), chunk = g0 - row * a.chunks, stage = 0;
  // A part's number that the last CTA's end and this one's beginning leave out.
  if (chunk == 0 && blockIdx.x > 0 && threadIdx.x == 0)
    a.beam_of[a.part_of(blockIdx.x, row) - 1] = kNone;
  Exponentials sums;
  float best = -INFINITY;
  bool on = enter(row) != nullptr;
  for (int g = g0; g < g1; ++g) {
    copy(stage == 0 ? kStages - 1 : stage - 1);
    wait_copies<kStages - 1>();
    if (on) {
      const uint4* mine = ring + stage * R * kThreads + threadIdx.x;
      Access<T> x[R];
#pragma unroll
      for (int k = 0; k < R; ++k) x[k].w = mine[k * kThreads];
      const float most = largest<T, R>(x);
      if (!a.c.lse) sums.add(x, mine, most);
      best = fmaxf(best, most);
    }
    if (++stage == kStages) stage = 0;
    if (++chunk < a.chunks && g + 1 < g1) continue;
    // The part's end: its warps leave what they have, without waiting for one another.
    const int part = a.part_of(blockIdx.x, row);
    if (threadIdx.x == 0) a.beam_of[part] = on ? row - a.by_beams.divide(row) * a.beams : kNone;
    if (on) {
      if (!a.c.lse) {
        const float top = unordered(__reduce_max_sync(0xffffffffu, ordered(best)));
        float sum = sums.sum * Exponentials::weight(sums.most, top);
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
        if (lane == 0) a.stats[(size_t)part * kWarps + warp] = make_float2(top, sum);
      }
      const int log_width = kLogThreads - a.log_groups;
      for (int m = 1; m < 1 << log_width; m <<= 1)
        best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, m));
      if ((threadIdx.x & ((1 << log_width) - 1)) == 0)
        a.maxima[((size_t)part << a.log_groups) + (threadIdx.x >> log_width)] = best;
    }
    sums = Exponentials();
    best = -INFINITY;
    chunk = 0;
    if (g + 1 < g1) on = enter(++row) != nullptr;
  }
}

template <typename T, int R>
cudaError_t select_as(const hg_beam& h, SelectArgs& a, cudaStream_t stream) {
  constexpr int E = 16 / sizeof(T);
  const long long rows = (long long)a.c.items * h.beams;
  a.chunks = (int)div_up((long long)h.vocab + E - 1, kThreads * R * E);
  const long long all = rows * a.chunks;
  if (all > 0x3fffffffLL) return cudaErrorInvalidValue;  // more logits than any device holds
  const long long full = (long long)kCtasPerSm * h.sms;
  const long long ctas = full < all ? full : all;
  a.all = (int)all;
  a.each = (int)(all / ctas);
  a.more = (int)(all % ctas);
  // An item's parts at most: a CTA's share may end in its rows, and begin, anywhere. A share is
  // more than half of all / full chunks, so that 152 SMs make at most 1281 parts of an item.
  const long long parts = div_up((long long)h.beams * a.chunks, a.each) + 1 + h.beams;
  if (parts > 1024 * kManyValues / kLeastGroups) return cudaErrorInvalidValue;
  const int values =
      h.picks > kFewPicks || parts * kLeastGroups > 1024 * kFewValues ? kManyValues : kFewValues;
  // As many groups of threads as there is room for values of their maxima; less where that
  // lets small CTAs join, which more items than SMs need (256 items: 28 and 24 us).
  const bool small = values == kFewValues && a.c.items > h.sms && parts * kLeastGroups <= 256 * values;
  a.log_groups = kLogThreads;
  while (parts << a.log_groups > (small ? 256 : 1024) * values) --a.log_groups;
  a.longest = a.each + (a.more > 0) < a.chunks ? a.each + (a.more > 0) : a.chunks;
  a.by_chunks = Divisor(a.chunks);
  a.by_each = Divisor(a.each);
  a.by_each_and_one = Divisor(a.each + 1);
  a.by_beams = Divisor(h.beams);
  a.by_longest = Divisor(a.longest);
  const cudaError_t e =
      launch_dependent(select_kernel<T, R>, a, (unsigned)ctas, kThreads,
                       (size_t)kStages * R * kThreads * 16, 1, stream);
  if (e != cudaSuccess) return e;
  if (values == kManyValues)
    return launch_dependent(join_kernel<T, R, 1024, kManyValues>, a, (unsigned)a.c.items, 1024, 0,
                            1, stream);
  return parts << a.log_groups <= 256 * values
             ? launch_dependent(join_kernel<T, R, 256, kFewValues>, a, (unsigned)a.c.items, 256, 0,
                                1, stream)
             : launch_dependent(join_kernel<T, R, 1024, kFewValues>, a, (unsigned)a.c.items, 1024,
                                0, 1, stream);
}

// Chunks of 16 KB, or smaller ones where there would be few.
template <typename T>
cudaError_t select_by(const hg_beam& h, SelectArgs& a, cudaStream_t stream) {
  const long long rows = (long long)a.c.items * h.beams;
  const long long bytes = rows * h.vocab * (long long)sizeof(T);
  const long long few = 64ll * kThreads * 16;
  if (bytes >= 4 * few) return select_as<T, 4>(h, a, stream);
  return bytes >= 2 * few ? select_as<T, 2>(h, a, stream) : select_as<T, 1>(h, a, stream);
}

template <typename T>
cudaError_t prepare_as() {
  cudaError_t e = cudaSuccess;
  for (void (*kernel)(SelectArgs) : {select_kernel<T, 1>, select_kernel<T, 2>, select_kernel<T, 4>})
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               kStages * 4 * kThreads * 16);
  return e;
}

}  // namespace

cudaError_t select_prepare(const hg_beam& h) {
  return h.dtype == HG_BF16   ? prepare_as<__nv_bfloat16>()
         : h.dtype == HG_FP16 ? prepare_as<__half>()
                              : prepare_as<float>();
}

long long part_slots(const hg_beam& h) {
  return (long long)h.max_items * h.beams + (long long)kCtasPerSm * h.sms;
}

cudaError_t select(const hg_beam& h, const SelectCall& c, cudaStream_t stream) {
  SelectArgs a = {};
  a.c = c;
  a.beams = h.beams;
  a.vocab = h.vocab;
  a.picks = h.picks;
  a.list = h.list;
  a.stats = h.stats;
  a.maxima = h.maxima;
  a.beam_of = h.beam_of;
  switch (h.dtype) {
    case HG_BF16:
      return select_by<__nv_bfloat16>(h, a, stream);
    case HG_FP16:
      return select_by<__half>(h, a, stream);
    default:
      return select_by<float>(h, a, stream);
  }
}

}  // namespace beam
}  // namespace hg
