// Beam search's selection: the best continuations of each item.
//
// A row's candidates are ordered by their logits alone, whatever its score and
// logsumexp are, so that each slice of a row gives its best `picks`, as keys (ordered
// logit, complement of the token), and the running maximum and sum of its
// exponentials. A second kernel joins an item's slices: the rows' logsumexps first, then
// the totals in 64 bits.

#include <cmath>

#include "hg_beam.cuh"

namespace hg {
namespace beam {
namespace {

using vocab::Elem;
using vocab::div_up;
using vocab::launch_dependent;
using vocab::let_successor_start;
using vocab::wait_for_predecessor;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr float kLog2e = 1.44269504088896341f;

struct SelectArgs {
  SelectCall c;
  int beams, vocab, picks, slices, slice;  // slice: columns of one
  unsigned long long* list;
  float2* stats;
};

// Bits of a value that is no NaN, in an order of unsigned integers; both zeros alike.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}

// Larger keys are better candidates of a row; 0 is none.
__device__ __forceinline__ unsigned long long key_of(float x, int token) {
  if (!(x > -INFINITY)) return 0;
  return (unsigned long long)ordered(x) << 32 | (uint32_t)~token;
}

__device__ __forceinline__ float exp_of(float x) { return exp2f(x * kLog2e); }

// A row whose logits count.
__device__ __forceinline__ bool searched(const SelectCall& c, size_t row) {
  return c.scores[row] > -INFINITY && !(c.finished && c.finished[row]);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) slice_kernel(const __grid_constant__ SelectArgs a) {
  __shared__ unsigned long long best[kWarps];
  __shared__ float red[2][kWarps];
  wait_for_predecessor();
  let_successor_start();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const size_t slot = blockIdx.x;
  const size_t row = slot / a.slices;
  const int first = (int)(slot - row * a.slices) * a.slice;
  const int last = min(first + a.slice, a.vocab);
  const T* x = static_cast<const T*>(a.c.logits) + row * a.c.ld;
  unsigned long long* list = a.list + slot * a.picks;
  if (!searched(a.c, row)) {
    for (int i = threadIdx.x; i < a.picks; i += kThreads) list[i] = 0;
    return;
  }
  if (!a.c.lse) {
    float most = -INFINITY;
    for (int v = first + threadIdx.x; v < last; v += kThreads) most = fmaxf(most, Elem<T>::up(x[v]));
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, m));
    if (lane == 0) red[0][warp] = most;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) most = fmaxf(most, red[0][w]);
    float sum = 0.f;
    // NaN goes through; of -inf there is nothing to add.
    for (int v = first + threadIdx.x; v < last; v += kThreads) {
      const float t = Elem<T>::up(x[v]);
      if (!(t == -INFINITY)) sum += exp_of(t - most);
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    if (lane == 0) red[1][warp] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < kWarps; ++w) sum += red[1][w];
      a.stats[slot] = make_float2(most, sum);
    }
  }
  unsigned long long under = ~0ull;
  for (int i = 0; i < a.picks; ++i) {
    unsigned long long key = 0;
    for (int v = first + threadIdx.x; v < last; v += kThreads) {
      const unsigned long long k = key_of(Elem<T>::up(x[v]), v);
      if (k < under && k > key) key = k;
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) key = max(key, __shfl_xor_sync(0xffffffffu, key, m));
    __syncthreads();
    if (lane == 0) best[warp] = key;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) key = max(key, best[w]);
    under = key;  // once 0, nothing is below it
    if (threadIdx.x == 0) list[i] = key;
  }
}

// A candidate of an item, in the order of the picks.
struct Candidate {
  double total;
  int beam;  // -1: none
  unsigned long long key;
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

__global__ void __launch_bounds__(kThreads) join_kernel(const __grid_constant__ SelectArgs a) {
  __shared__ double lse[HG_MAX_BEAMS];
  __shared__ Candidate best[kWarps];
  wait_for_predecessor();
  let_successor_start();
  const SelectCall& c = a.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int item = blockIdx.x;
  const size_t row0 = (size_t)item * a.beams;
  for (int b = threadIdx.x; b < a.beams; b += kThreads) {
    if (c.lse) {
      lse[b] = c.lse[(row0 + b) * c.lse_stride];
      continue;
    }
    const float2* s = a.stats + (row0 + b) * a.slices;
    float most = -INFINITY;
    double sum = 0.0;
    for (int i = 0; i < a.slices; ++i) most = fmaxf(most, s[i].x);
    for (int i = 0; i < a.slices; ++i)
      if (s[i].x > -INFINITY || s[i].y != 0.f) sum += (double)s[i].y * exp((double)s[i].x - most);
    lse[b] = most + log(sum);
  }
  __syncthreads();
  const int per_beam = a.slices * a.picks;
  const int entries = a.beams * per_beam;
  const unsigned long long* list = a.list + row0 * per_beam;
  auto candidate = [&](int i) {
    Candidate t;
    t.beam = i / per_beam;
    t.key = list[i];
    const size_t row = row0 + t.beam;
    const float score = c.scores[row];
    if (c.finished && c.finished[row]) {
      if (i % per_beam == 0) t.key = (uint32_t)~c.end;
      else t.key = 0;
      t.total = score;
    } else {
      t.total = (double)score + ((double)unordered((uint32_t)(t.key >> 32)) - lse[t.beam]);
    }
    if (t.key == 0 || !((float)t.total > -INFINITY)) t.beam = -1;
    return t;
  };
  Candidate under;
  for (int i = 0; i < a.picks; ++i) {
    Candidate top;
    top.beam = -1;
    for (int j = threadIdx.x; j < entries; j += kThreads) {
      const Candidate t = candidate(j);
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
    if (lane == 0) best[warp] = top;
    __syncthreads();
    top = best[0];
    for (int w = 1; w < kWarps; ++w)
      if (best[w].before(top)) top = best[w];
    under = top;  // once none, nothing comes after it
    if (threadIdx.x == 0) {
      const size_t at = (size_t)item * a.picks + i;
      const bool there = top.beam >= 0;
      const int token = there ? (int)~(uint32_t)top.key : -1;
      put_id(c.tokens, c.id_bytes, at, token);
      put_id(c.parents, c.id_bytes, at, there ? top.beam : -1);
      c.picked[at] = there ? (float)top.total : -INFINITY;
      if (c.picked_finished)
        c.picked_finished[at] =
            there && (token == c.end || (c.finished && c.finished[row0 + top.beam]));
    }
  }
}

// CTAs that fill the device, and the most entries that one CTA is to join.
constexpr int kCtasPerSm = 4;
constexpr int kMostEntries = 16384;
constexpr int kLeastSlice = 4096;

}  // namespace

int slices(const hg_beam& h, int items) {
  const long long rows = (long long)items * h.beams;
  long long n = div_up((long long)kCtasPerSm * h.sms, rows);
  if (n > kMostEntries / (h.beams * h.picks)) n = kMostEntries / (h.beams * h.picks);
  if (n > div_up(h.vocab, kLeastSlice)) n = div_up(h.vocab, kLeastSlice);
  return n < 1 ? 1 : (int)n;
}

long long list_slots(const hg_beam& h) {
  // rows * ceil(full / rows) < rows + full, whatever the call's items.
  return (long long)h.max_items * h.beams + (long long)kCtasPerSm * h.sms;
}

cudaError_t select(const hg_beam& h, const SelectCall& c, cudaStream_t stream) {
  SelectArgs a = {};
  a.c = c;
  a.beams = h.beams;
  a.vocab = h.vocab;
  a.picks = h.picks;
  a.slices = slices(h, c.items);
  a.slice = (int)div_up(h.vocab, a.slices);
  a.list = h.list;
  a.stats = h.stats;
  const unsigned grid = (unsigned)(c.items * h.beams * a.slices);
  cudaError_t e;
  switch (h.dtype) {
    case HG_BF16:
      e = launch_dependent(slice_kernel<__nv_bfloat16>, a, grid, kThreads, 0, 1, stream);
      break;
    case HG_FP16:
      e = launch_dependent(slice_kernel<__half>, a, grid, kThreads, 0, 1, stream);
      break;
    default:
      e = launch_dependent(slice_kernel<float>, a, grid, kThreads, 0, 1, stream);
  }
  if (e != cudaSuccess) return e;
  return launch_dependent(join_kernel, a, (unsigned)c.items, kThreads, 0, 1, stream);
}

}  // namespace beam
}  // namespace hg
