// Beam search's selection: the best continuations of each item.
//
// One pass over the logits. A row's candidates are ordered by their logits alone, whatever
// its score and logsumexp are, so a part of a row gives its best `picks` as keys (ordered
// logit, complement of the token) and, where the logsumexp is wanted, the running
// maximum and sum of its exponentials. The rows' chunks are dealt out to the CTAs in
// order, the same number to each; the last CTA to finish an item's chunks joins its parts.
//
// A thread reads ahead of itself into a ring in shared memory, and keeps the largest logit of
// each of its cells, the elements that it has of a chunk. At the end of a part, the n-th
// largest of the threads' maxima bounds the n-th best element from below, so only the cells
// that reach it, little more than n, are read again (from L2) for the elements that do. What
// a chunk costs beside its loads is a maximum and the exponentials. (Lists of the best that
// were kept up to date chunk by chunk, by CTA or by warp, took two to four times as long.)

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

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kStages = 3;      // chunks in the ring
constexpr int kCells = 16;      // of a thread, at most, in a part
constexpr int kList = 512;      // elements of a part, or of an item, that are ranked at once
constexpr int kCtasPerSm = 3;
constexpr int kMostEntries = HG_MAX_BEAMS * HG_MAX_PICKS;  // of the lists that one CTA joins
constexpr float kLog2e = 1.44269504088896341f;
constexpr double kLn2 = 0.693147180559945309417;
constexpr double kLog2eOff = 1.0 - (double)kLog2e * kLn2;

constexpr int kNone = 255;

// Division of numbers below 2^31 by one that is known when the kernel is launched.
struct Divisor {
  uint32_t by = 1, factor = 0;
  int shift = 0;
  Divisor() = default;
  explicit Divisor(uint32_t d) : by(d) {
    while ((1ull << shift) < d) ++shift;
    factor = (uint32_t)((1ull << (31 + shift)) / d + 1);
    shift += 31;
  }
  __device__ int divide(int n) const {
    return by == 1 ? n : (int)((unsigned long long)(uint32_t)n * factor >> shift);
  }
};

struct SelectArgs {
  SelectCall c;
  int beams, vocab, picks;
  int chunks;          // of a row
  int each, more;      // chunks of a CTA; the first `more` CTAs have one more
  Divisor by_chunks, by_each, by_each_and_one, by_picks, by_beams;
  int all;             // chunks of the call
  int whole_rows;      // CTAs have whole rows
  int cell_chunks;     // chunks of a cell
  u64* list;           // [part][picks], best first
  float2* stats;       // [part]
  int* beam_of;        // [part], kNone where it is not searched or there is no such part
  unsigned* arrived;   // [item]
  __device__ int first_chunk(int cta) const { return min(cta * each + min(cta, more), all); }
  __device__ int cta_of(int chunk) const {
    const int front = more * (each + 1);
    return chunk < front ? by_each_and_one.divide(chunk) : more + by_each.divide(chunk - front);
  }
  // The number of what a CTA has of a row: going through the chunks, each new part raises the
  // CTA, the row, or both.
  __device__ int part_of(int cta, int row) const { return whole_rows ? row : cta + row; }
};

// Bits of a value that is no NaN, in an order of unsigned integers; both zeros alike.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}
__device__ __forceinline__ u64 ordered(double v) {
  const u64 u = (u64)__double_as_longlong(v + 0.0);
  return u >> 63 ? ~u : u | 1ull << 63;
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

// A row whose logits count.
__device__ __forceinline__ bool searched(const SelectCall& c, size_t row) {
  return c.scores[row] > -INFINITY && !(c.finished && c.finished[row]);
}

// 16 bytes of logits.
template <typename T>
struct Access {
  static constexpr int E = 16 / sizeof(T);
  uint4 w;

  // Copies 16 bytes ahead.
  static __device__ __forceinline__ void copy(uint4* to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(to)),
                 "l"(from)
                 : "memory");
  }
  // The same for elements [e0, e0 + E) of a row of `vocab`, some of which may lie outside:
  // those are -inf, and are not read.
  static __device__ __forceinline__ void copy_edge(uint4* to, const T* row, int e0, int vocab) {
    if (e0 >= 0 && e0 + E <= vocab) {
      copy(to, row + e0);
      return;
    }
    T v[E];
#pragma unroll
    for (int e = 0; e < E; ++e)
      v[e] = e0 + e >= 0 && e0 + e < vocab ? row[e0 + e] : Elem<T>::down(-INFINITY);
    memcpy(to, v, 16);
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
template <typename T>
__device__ __forceinline__ float largest_of(const Access<T>& x) {
  if constexpr (sizeof(T) == 2) {
    const float2 f = Elem<T>::unpack2(
        max2(max2(x.w.x, x.w.y, T{}), max2(x.w.z, x.w.w, T{}), T{}));
    return fmaxf(f.x, f.y);
  } else {
    return fmaxf(fmaxf(__uint_as_float(x.w.x), __uint_as_float(x.w.y)),
                 fmaxf(__uint_as_float(x.w.z), __uint_as_float(x.w.w)));
  }
}
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
// is in each exponent, and rescaling as the maximum rises is exact. From kHuge on, where
// neighbours are further apart than exponentials reach, the largest elements count one each.
// NaN and +inf give NaN.
constexpr float kHuge = 1e30f;

struct Exponentials {
  float most = -INFINITY, sum = 0.f;

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
    raise(chunk_most);
    if (!plain(most)) {
      sum += count_huge<T>(ring, R, most);
      return;
    }
    const float s = shift(most);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float v[Access<T>::E];
      x[r].widen(v);
#pragma unroll
      for (int e = 0; e < Access<T>::E; ++e) sum += exp2_of(fmaf(v[e], kLog2e, -s));
    }
  }
  __device__ __forceinline__ void join(float other_most, float other_sum) {
    raise(other_most);
    sum += other_sum * weight(other_most, most);
  }
};

constexpr float kLeast = -3.402823466e38f;

// A bin for every eighth of an octave of the distance from the best.
constexpr int kBins = 240;
__device__ __forceinline__ int bin_of(uint32_t d) {
  if (d < 8) return (int)d;
  const int e = 31 - __clz(d);
  return (e - 2) * 8 + (int)((d >> (e - 3)) & 7);
}
__device__ __forceinline__ uint32_t bin_end(int bin) {
  if (bin < 8) return (uint32_t)bin;
  return ((uint32_t)(8 + bin % 8 + 1) << (bin / 8 - 1)) - 1;
}

struct BoundShared {
  int bins[kBins];
  uint32_t top[kWarps];
};

// A value that at least n of the CTA's words (ordered values; 0: none) are not under, and not
// many more: the end of the bin that the n-th largest is in. words(f) calls f for each word
// of a thread, `top` is the thread's largest. The least finite value if there are not n.
template <typename Words>
__device__ __forceinline__ float bound_of_best(int n, uint32_t top, BoundShared& s, Words words) {
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  top = __reduce_max_sync(kAll, top);
  if (lane == 0) s.top[threadIdx.x >> 5] = top;
  for (int i = threadIdx.x; i < kBins; i += kThreads) s.bins[i] = 0;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) top = max(top, s.top[w]);
  words([&](uint32_t word) {
    if (word) atomicAdd(&s.bins[bin_of(top - word)], 1);
  });
  __syncthreads();
  // The first bin up to which there are enough; each warp for itself, eight bins a lane.
  int upto[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    upto[i] = (lane * 8 + i < kBins ? s.bins[lane * 8 + i] : 0) + (i ? upto[i - 1] : 0);
  int before = upto[7];
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int other = __shfl_up_sync(kAll, before, m);
    if (lane >= m) before += other;
  }
  const unsigned reach = __ballot_sync(kAll, before >= n);
  before -= upto[7];
  int bin = lane * 8 + 7;
#pragma unroll
  for (int i = 6; i >= 0; --i)
    if (before + upto[i] >= n) bin = lane * 8 + i;
  if (!reach) return kLeast;
  const uint32_t far = bin_end(__shfl_sync(kAll, bin, __ffs(reach) - 1));
  const uint32_t word = far < top ? top - far : 0;
  return word < ordered(kLeast) ? kLeast : unordered(word);
}

struct PartShared {
  float cell[kCells][kThreads];
  u64 list[kList];
  BoundShared bound;
  float most[kWarps], sum[kWarps];
  int warp_count[2][kWarps];
  int count;
};

// A part: chunks [first, first + chunks) of a row.
template <typename T, int R>
struct Part {
  static constexpr int E = Access<T>::E;
  const T* row;  // null: its logits do not count
  int first, chunks, vocab;

  __device__ __forceinline__ int shift() const {
    return (int)(reinterpret_cast<uintptr_t>(row) % 16 / sizeof(T));
  }
  // The first element of this thread's access k of chunk i.
  __device__ __forceinline__ int element(int i, int k) const {
    return (((first + i) * R + k) * kThreads + (int)threadIdx.x) * E - shift();
  }
  // Calls f(logit, token) for the elements of this thread from `least` on, in chunk i.
  template <typename F>
  __device__ __forceinline__ void each(int i, float least, F f) const {
    uint32_t mask = 0;
    const int e0 = element(i, 0) - (int)threadIdx.x * E;
    if (e0 >= 0 && e0 + kThreads * R * E <= vocab) {
      Access<T> x[R];  // all loads before the first use
#pragma unroll
      for (int k = 0; k < R; ++k) x[k].w = *reinterpret_cast<const uint4*>(row + element(i, k));
#pragma unroll
      for (int k = 0; k < R; ++k) {
        float v[E];
        x[k].widen(v);
#pragma unroll
        for (int e = 0; e < E; ++e) mask |= v[e] >= least ? 1u << (k * E + e) : 0u;
      }
    } else {
#pragma unroll 4
      for (int m = 0; m < R * E; ++m) {
        const int at = element(i, m / E) + m % E;
        if (at >= 0 && at < vocab && Elem<T>::up(row[at]) >= least) mask |= 1u << m;
      }
    }
    for (; mask; mask &= mask - 1) {
      const int m = __ffs(mask) - 1, at = element(i, m / E) + m % E;
      f(Elem<T>::up(row[at]), at);
    }
  }
};

__device__ __forceinline__ int count_all(int c, int turn, PartShared& s) {
  c = __reduce_add_sync(0xffffffffu, c);
  if ((threadIdx.x & 31) == 0) s.warp_count[turn][threadIdx.x >> 5] = c;
  __syncthreads();
  c = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) c += s.warp_count[turn][w];
  return c;
}

// Where too many elements of a part are alike for the list: the key of its n-th best, one
// bit after another, and the keys from that on. Reads the part again for each bit.
template <typename T, int R>
__device__ __noinline__ void list_exactly(const Part<T, R> part, int n, PartShared& s) {
  u64 bound = 0;
  for (int bit = 63; bit >= 0; --bit) {
    const u64 next = bound | 1ull << bit;
    int c = 0;
    for (int i = 0; i < part.chunks; ++i)
      part.each(i, kLeast, [&](float x, int token) { c += key_of(x, token) >= next; });
    if (count_all(c, bit & 1, s) >= n) bound = next;
  }
  __syncthreads();
  if (threadIdx.x == 0) s.count = 0;
  __syncthreads();
  for (int i = 0; i < part.chunks; ++i)
    part.each(i, kLeast, [&](float x, int token) {
      if (key_of(x, token) >= bound) s.list[atomicAdd(&s.count, 1)] = key_of(x, token);
    });
  __syncthreads();
}

template <typename T, int R>
__device__ __forceinline__ void finish_part(const SelectArgs& a, int number, int beam,
                                            const Part<T, R>& part, Exponentials& sums,
                                            PartShared& s) {
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  u64* out = a.list + (size_t)number * a.picks;
  if (threadIdx.x == 0) a.beam_of[number] = part.row ? beam : kNone;
  if (!part.row) return;
  if (!a.c.lse) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1)
      sums.join(__shfl_xor_sync(kAll, sums.most, m), __shfl_xor_sync(kAll, sums.sum, m));
    if (lane == 0) {
      s.most[warp] = sums.most;
      s.sum[warp] = sums.sum;
    }
  }
  if (threadIdx.x == 0) s.count = 0;
  const int cells = (part.chunks + a.cell_chunks - 1) / a.cell_chunks;
  float most = -INFINITY;
  for (int i = 0; i < cells; ++i) most = fmaxf(most, s.cell[i][threadIdx.x]);
  const uint32_t word = most > -INFINITY ? ordered(most) : 0;
  const float from = bound_of_best(a.picks, word, s.bound, [&](auto f) { f(word); });
  if (!a.c.lse && threadIdx.x == 0) {
    for (int w = 1; w < kWarps; ++w) sums.join(s.most[w], s.sum[w]);
    a.stats[number] = make_float2(sums.most, sums.sum);
  }
  if (most >= from)
    for (int i = 0; i < cells; ++i) {
      if (!(s.cell[i][threadIdx.x] >= from)) continue;
      for (int j = i * a.cell_chunks; j < min((i + 1) * a.cell_chunks, part.chunks); ++j)
        part.each(j, from, [&](float x, int token) {
          const int at = atomicAdd(&s.count, 1);
          if (at < kList) s.list[at] = key_of(x, token);
        });
    }
  __syncthreads();
  int all = s.count;
  if (all > kList) {
    list_exactly(part, a.picks, s);
    all = s.count;
  }
  // Each key's rank among them; eight lanes count what is above it.
  const int eighth = threadIdx.x % 8;
  for (int i0 = 0; i0 < all; i0 += kThreads / 8) {
    const int i = i0 + threadIdx.x / 8;
    const u64 mine = i < all ? s.list[i] : ~0ull;
    int rank = 0;
#pragma unroll 4
    for (int j = eighth; j < all; j += 8) rank += s.list[j] > mine;
#pragma unroll
    for (int m = 4; m > 0; m >>= 1) rank += __shfl_xor_sync(kAll, rank, m);
    if (eighth == 0 && i < all && rank < a.picks) out[rank] = mine;
  }
  for (int i = all + threadIdx.x; i < a.picks; i += kThreads) out[i] = 0;
  __syncthreads();
  sums = Exponentials();
}

// ---- joining an item's parts -------------------------------------------------------

struct JoinShared {
  u64 total[kList], key[kList];
  unsigned char beam[kList];
  double lse[HG_MAX_BEAMS];
  float score[HG_MAX_BEAMS];
  float near[HG_MAX_BEAMS];  // score - logsumexp in fp32
  bool done[HG_MAX_BEAMS];   // finished, and still a candidate
  float largest[2];          // magnitude of near, below kHuge, of 32 beams each
  BoundShared bound;
  double top_total[kWarps];
  u64 top_key[kWarps];
  int top_beam[kWarps];
  int count;
};

union Shared {
  PartShared part;
  JoinShared join;
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

__device__ void put_pick(const SelectArgs& a, int item, int rank, bool there, double total,
                         int beam, u64 key) {
  const SelectCall& c = a.c;
  const size_t at = (size_t)item * a.picks + rank;
  const int token = there ? (int)~(uint32_t)key : -1;
  put_id(c.tokens, c.id_bytes, at, token);
  put_id(c.parents, c.id_bytes, at, there ? beam : -1);
  c.picked[at] = there ? (float)total : -INFINITY;
  if (c.picked_finished)
    c.picked_finished[at] =
        there && (token == c.end || (c.finished && c.finished[(size_t)item * a.beams + beam]));
}

// Logsumexp of a row from its parts, by one warp. The logarithm of the sum's exponent is
// exact to 64 bits, that of its mantissa, below 0.35, to 32.
__device__ __forceinline__ double row_lse(const SelectArgs& a, int part0, int parts) {
  const int lane = threadIdx.x & 31;
  Exponentials t;
  for (int i = lane; i < parts; i += 32) {
    const float2 s = __ldcg(a.stats + part0 + i);
    t.join(s.x, s.y);
  }
#pragma unroll
  for (int m = 16; m > 0; m >>= 1)
    t.join(__shfl_xor_sync(0xffffffffu, t.most, m), __shfl_xor_sync(0xffffffffu, t.sum, m));
  if (!(t.sum < INFINITY)) return t.sum;  // NaN
  if (!Exponentials::plain(t.most)) return t.most;
  int e = 0;
  float f = frexpf(t.sum, &e);  // in [0.5, 1)
  if (f < 0.70710678f) {
    f *= 2.f;
    --e;
  }
  // kLog2e is 1 - kLog2eOff times log2(e): its share of the logits, nearly the largest one's.
  return t.sum > 0.f ? ((double)Exponentials::shift(t.most) + e) * kLn2 + (double)logf(f) +
                           (double)t.most * kLog2eOff
                     : -INFINITY;
}

// What join_item compares: the entries of the parts' lists, and behind them one of each
// finished beam.
struct Entries {
  const SelectArgs& a;
  const JoinShared& s;
  int listed, all;
  const u64* list;     // of the item's first part
  const int* beam_of;

  // Entry i's beam (kNone: no candidate) and key; both loads are in flight together.
  __device__ __forceinline__ void get(int i, int& beam, u64& key) const {
    const int in = min(i, listed - 1);
    key = __ldcg(list + in);
    beam = __ldcg(beam_of + a.by_picks.divide(in));
    if (key == 0) beam = kNone;
    if (i >= listed) {
      key = (uint32_t)~a.c.end;
      beam = i < all && s.done[i - listed] ? i - listed : kNone;
    }
  }
  __device__ __forceinline__ double total(int i, int beam, u64 key) const {
    const double score = s.score[beam];
    return i < listed ? score + ((double)unordered((uint32_t)(key >> 32)) - s.lse[beam]) : score;
  }
  // A total to within `off` of it in fp32 (64-bit additions are slow, and few entries come
  // near the best).
  __device__ __forceinline__ float near(int i, int beam, u64 key) const {
    if (i >= listed) return s.score[beam];
    const float near = s.near[beam], t = unordered((uint32_t)(key >> 32)) + near;
    return fabsf(near) < kHuge && fabsf(t) < kHuge ? t : (float)total(i, beam, key);
  }
  // Three roundings of at most half a unit in the last place of the two terms and of the sum.
  __device__ __forceinline__ float off(float t) const {
    const float near = fmaxf(s.largest[0], s.largest[1]);
    return fabsf(t) < INFINITY ? 3.f * 5.9604645e-8f * (near + fabsf(t)) : 0.f;
  }
};

__device__ __noinline__ void join_item(const SelectArgs& a, int item, JoinShared& s,
                                       float* value) {
  const SelectCall& c = a.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row0 = item * a.beams, row_last = row0 + a.beams - 1;
  const int part0 = a.part_of(a.cta_of(row0 * a.chunks), row0);
  const int parts = a.part_of(a.cta_of((row_last + 1) * a.chunks - 1), row_last) - part0 + 1;
  const int listed = parts * a.picks;
  const Entries entries{a, s, listed, listed + (c.finished ? a.beams : 0),
                        a.list + (size_t)part0 * a.picks, a.beam_of + part0};
  // What of the entries is loaded at once, and first of all.
  constexpr int kBatch = 4;
  u64 key[kBatch];
  int beam[kBatch];
  auto load = [&](int i0) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) entries.get(i0 + k * kThreads, beam[k], key[k]);
  };
  float near = 0.f;
  if (threadIdx.x < a.beams) {
    const int b = threadIdx.x, row = row0 + b;
    const float score = c.scores[row];
    s.score[b] = score;
    s.done[b] = c.finished && c.finished[row] && score > -INFINITY;
    if (c.lse) {
      const double lse = c.lse[row * c.lse_stride];
      s.lse[b] = lse;
      near = (float)((double)score - lse);
      s.near[b] = near;
    }
  }
  if (threadIdx.x == 0) s.count = 0;
  if (!c.lse) {
    for (int b = warp; b < a.beams; b += kWarps) {
      const int row = row0 + b, first = a.part_of(a.cta_of(row * a.chunks), row);
      const double lse =
          searched(c, row)
              ? row_lse(a, first, a.part_of(a.cta_of((row + 1) * a.chunks - 1), row) - first + 1)
              : 0.0;
      if (lane == 0) {
        s.lse[b] = lse;
        s.near[b] = (float)((double)c.scores[row] - lse);
      }
    }
  }
  __syncthreads();
  load(threadIdx.x);
  // How large the terms of a total are at most, for its rounding.
  if (!c.lse && threadIdx.x < a.beams) near = s.near[threadIdx.x];
  near = fabsf(near) < kHuge ? fabsf(near) : 0.f;
  const uint32_t largest = __reduce_max_sync(0xffffffffu, __float_as_uint(near));
  if (lane == 0 && warp < 2) s.largest[warp] = __uint_as_float(largest);
  static_assert(HG_MAX_BEAMS <= 64, "two warps have the beams");
  __syncthreads();
  // The entries' totals, nearly; the words of a bound from below.
  uint32_t top = 0;
  for (int i0 = threadIdx.x;;) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * kThreads;
      if (i >= entries.all) break;
      const float t = beam[k] != kNone ? entries.near(i, beam[k], key[k]) : -INFINITY;
      value[i] = t;
      if (t > -INFINITY) top = max(top, ordered(t - entries.off(t)));
    }
    i0 += kBatch * kThreads;
    if (i0 >= entries.all) break;
    load(i0);
  }
  const float from = bound_of_best(a.picks, top, s.bound, [&](auto f) {
#pragma unroll 4
    for (int i = threadIdx.x; i < entries.all; i += kThreads)
      f(value[i] > -INFINITY ? ordered(value[i] - entries.off(value[i])) : 0);
  });
  for (int i = threadIdx.x; i < entries.all; i += kThreads) {
    if (!(value[i] + entries.off(value[i]) >= from)) continue;
    int beam;
    u64 key;
    entries.get(i, beam, key);
    if (beam == kNone) continue;
    const double total = entries.total(i, beam, key);
    if (!((float)total > -INFINITY)) continue;
    const int at = atomicAdd(&s.count, 1);
    if (at >= kList) continue;
    s.total[at] = ordered(total);
    s.key[at] = key;
    s.beam[at] = (unsigned char)beam;
  }
  __syncthreads();
  const int all = s.count;
  if (all <= kList) {
    // Eight lanes count what comes before a candidate.
    const int eighth = threadIdx.x % 8;
    for (int i0 = 0; i0 < all; i0 += kThreads / 8) {
      const int i = i0 + threadIdx.x / 8;
      const bool there = i < all;
      const u64 total = there ? s.total[i] : ~0ull, key = there ? s.key[i] : ~0ull;
      const int beam = there ? s.beam[i] : 0;
      int rank = 0;
#pragma unroll 4
      for (int j = eighth; j < all; j += 8) {
        const u64 t = s.total[j], k = s.key[j];
        const int b = s.beam[j];
        rank += (t > total) | ((t == total) & ((b < beam) | ((b == beam) & (k > key))));
      }
#pragma unroll
      for (int m = 4; m > 0; m >>= 1) rank += __shfl_xor_sync(0xffffffffu, rank, m);
      if (there && eighth == 0 && rank < a.picks) {
        const double d =
            __longlong_as_double((long long)(total >> 63 ? total & ~(1ull << 63) : ~total));
        put_pick(a, item, rank, true, d, beam, key);
      }
    }
    for (int i = all + threadIdx.x; i < a.picks; i += kThreads)
      put_pick(a, item, i, false, 0.0, -1, 0);
    return;
  }
  // Too many alike: one pick after another.
  Candidate under;
  for (int i = 0; i < a.picks; ++i) {
    Candidate top;
    top.beam = -1;
    for (int j = threadIdx.x; j < entries.all; j += kThreads) {
      Candidate t;
      entries.get(j, t.beam, t.key);
      if (t.beam == kNone) continue;
      t.total = entries.total(j, t.beam, t.key);
      if (!((float)t.total > -INFINITY)) continue;
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
    for (int w = 0; w < kWarps; ++w) {
      const Candidate o = {s.top_total[w], s.top_beam[w], s.top_key[w]};
      if (o.before(top)) top = o;
    }
    under = top;  // once none, nothing comes after it
    if (threadIdx.x == 0) put_pick(a, item, i, top.beam >= 0, top.total, top.beam, top.key);
  }
}

template <typename T, int R>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    select_kernel(const __grid_constant__ SelectArgs a) {
  constexpr int E = Access<T>::E;
  extern __shared__ uint4 ring[];  // [stage][R][threads]: a thread reads what it copied
  __shared__ Shared s;
  __shared__ bool last;
  wait_for_predecessor();
  let_successor_start();
  const int g0 = a.first_chunk(blockIdx.x), g1 = a.first_chunk(blockIdx.x + 1);

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
          for (int k = 0; k < R; ++k) Access<T>::copy(to + k * kThreads, from + k * kThreads);
        } else {
#pragma unroll 1
          for (int k = 0; k < R; ++k)
            Access<T>::copy_edge(to + k * kThreads, ahead_at,
                                 e0 + (k * kThreads + (int)threadIdx.x) * E, a.vocab);
        }
      }
      ++ahead;
      if (++ahead_chunk == a.chunks) {
        ahead_chunk = 0;
        ++ahead_row;
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) copy(i);
  int row = a.by_chunks.divide(g0), chunk = g0 - row * a.chunks, stage = 0;
  // A part's number that the last CTA's end and this one's beginning leave out.
  if (chunk == 0 && blockIdx.x > 0 && !a.whole_rows && threadIdx.x == 0)
    a.beam_of[a.part_of(blockIdx.x, row) - 1] = kNone;
  const T* at = enter(row);
  Exponentials sums;
  Part<T, R> part = {enter(row), chunk, 0, a.vocab};
  float cell = -INFINITY;
  int in_cell = 0, cells = 0;
  for (int g = g0; g < g1; ++g) {
    copy(stage == 0 ? kStages - 1 : stage - 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    if (part.row) {
      const uint4* mine = ring + stage * R * kThreads + threadIdx.x;
      Access<T> x[R];
#pragma unroll
      for (int k = 0; k < R; ++k) x[k].w = mine[k * kThreads];
      const float most = largest<T, R>(x);
      if (!a.c.lse) sums.add(x, mine, most);
      cell = fmaxf(cell, most);
    }
    if (++stage == kStages) stage = 0;
    ++part.chunks;
    const bool ends = ++chunk == a.chunks || g + 1 == g1;
    if (++in_cell == a.cell_chunks || ends) {
      s.part.cell[cells++][threadIdx.x] = cell;
      cell = -INFINITY;
      in_cell = 0;
    }
    if (ends) {
      finish_part(a, a.part_of(blockIdx.x, row), row - a.by_beams.divide(row) * a.beams, part, sums,
                  s.part);
      cells = chunk = 0;
      if (g + 1 < g1) part = {enter(++row), 0, 0, a.vocab};
    }
  }
  __threadfence();
  const int item_chunks = a.beams * a.chunks;
  const int last_item = a.by_beams.divide(a.by_chunks.divide(g1 - 1));
  for (int item = a.by_beams.divide(a.by_chunks.divide(g0)); item <= last_item; ++item) {
    __syncthreads();
    if (threadIdx.x == 0) {
      const int from = item * item_chunks;
      const unsigned before = (unsigned)(a.cta_of(from + item_chunks - 1) - a.cta_of(from));
      last = atomicInc(a.arrived + item, before) == before;  // and back to 0
    }
    __syncthreads();
    if (!last) continue;
    __threadfence();
    join_item(a, item, s.join, reinterpret_cast<float*>(ring));
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
  // An item's parts, of its beams and CTAs, are joined by one CTA: where that would be
  // too many entries, CTAs have whole rows.
  const long long per_item = kMostEntries / h.picks - h.beams - 2;
  long long ctas = per_item * a.c.items < full ? per_item * a.c.items : full;
  if (ctas > all) ctas = all;
  a.whole_rows = per_item < h.beams;
  a.all = (int)all;
  if (a.whole_rows) {
    a.each = (int)div_up(rows, full) * a.chunks;
    ctas = div_up(all, a.each);
  } else {
    a.each = (int)(all / ctas);
    a.more = (int)(all % ctas);
  }
  const int longest = a.each + (a.more > 0) < a.chunks ? a.each + (a.more > 0) : a.chunks;
  a.cell_chunks = (longest + kCells - 1) / kCells;
  a.by_chunks = Divisor(a.chunks);
  a.by_each = Divisor(a.each);
  a.by_each_and_one = Divisor(a.each + 1);
  a.by_picks = Divisor(h.picks);
  a.by_beams = Divisor(h.beams);
  // The ring, or the entries of an item (join_item).
  const size_t held = (size_t)kStages * R * kThreads * 16;
  const size_t joined = (size_t)(kMostEntries + HG_MAX_BEAMS) * sizeof(float);
  const size_t smem = held > joined ? held : joined;
  return launch_dependent(select_kernel<T, R>, a, (unsigned)ctas, kThreads, smem, 1, stream);
}

// Chunks of 16 KB, or smaller ones where there would be few: the more parts, the more there
// is to join.
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

long long list_slots(const hg_beam& h) {
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
  a.beam_of = h.beam_of;
  a.arrived = h.arrived;
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
