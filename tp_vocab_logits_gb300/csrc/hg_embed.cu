// Embedding lookup with scaling, and its gradient by sorted tokens.
//
// Lookup: out[n] = scale * table[tokens[n]], a copy of N rows of K elements
// bound by memory: each row read and each output written once. One warp moves
// A accesses per lane of one row, all loads in flight before the first store:
// four of 16 bytes, eight of 4 bytes where rows are aligned to that only, else
// sixteen single elements. 32768 rows of 7168 bf16 take 109 us, 6.2 TB/s.
//
// Gradient: grad_table[v] (+)= scale * sum of grad[n] over tokens[n] = v. The
// positions are sorted by token (stable, so that a token's rows come in the
// order of their positions), and the sorted sequence is cut into chunks of
// 32 rows (8 or 16 where there are few: run_rows) whatever the tokens are: text
// repeats a few tokens thousands of times, and a chunk is the same work for one
// token as for 32. A warp sums one chunk over the columns of its lanes in fp32
// registers. A run of equal tokens that lies within a chunk is finished there; one
// that crosses a chunk's end leaves its partial sums in `runs` (slot 0: the run a
// chunk continues, slot 1: the run it starts and does not finish), and join_kernel
// adds those in chunk order. No atomics, so the order of every sum is fixed. Memory
// bounds it once the table is written whole (16384 rows of 7168 bf16, V=163840: 385 us,
// 6.7 TB/s); added to a table, 8192 rows take 64 us, of which the sums are 42 (the rows
// come in pieces of 512 bytes: 59 % of DRAM throughput) and the sort's latency 13.

#include <cooperative_groups.h>

#include "hg_vocab.cuh"

namespace cg = cooperative_groups;

namespace hg {
namespace vocab {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kLookupThreads = 128;

struct Table {
  void* shard[HG_MAX_TP];
};

template <typename T>
__device__ __forceinline__ T* table_row(const Table& t, uint32_t id, int W, int K) {
  const uint32_t r = id / (uint32_t)W;
  return static_cast<T*>(t.shard[r]) + (size_t)(id - r * (uint32_t)W) * K;
}

// Store of what this kernel does not read again: evicted first, so that L2 keeps
// the table's rows that other tokens share (32768 rows 111 -> 109 us).
template <typename P>
__device__ __forceinline__ void store_streaming(P* p, const P& x) {
  if constexpr (sizeof(P) == 16)
    __stcs(reinterpret_cast<uint4*>(p), *reinterpret_cast<const uint4*>(&x));
  else
    *p = x;
}

struct EmbedArgs {
  Table table;
  Ids tokens;
  int N, K, W, vocab;
  int units_per_row;
  float scale;
  void* out;
  size_t ld;
};

template <typename T, int E, int A>
__global__ void __launch_bounds__(kLookupThreads)
    embed_kernel(const __grid_constant__ EmbedArgs a) {
  wait_for_predecessor();
  let_successor_start();
  const int lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * (kLookupThreads / 32) + (threadIdx.x >> 5);
  const long long n = unit / a.units_per_row;
  if (n >= a.N) return;
  const int first = (int)(unit - n * a.units_per_row) * (A * 32) + lane;
  const int accesses = a.K / E;
  using P = Pack<T, E>;
  P x[A];
  const long long id = load_id(a.tokens, (size_t)n);
  const bool inside = id >= 0 && id < a.vocab;
  const P* src =
      reinterpret_cast<const P*>(table_row<T>(a.table, inside ? (uint32_t)id : 0, a.W, a.K));
#pragma unroll
  for (int j = 0; j < A; ++j) {
    const int i = first + j * 32;
    if (inside && i < accesses) {
      x[j] = src[i];
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) x[j].v[e] = Elem<T>::down(0.f);
    }
  }
  P* dst = reinterpret_cast<P*>(static_cast<T*>(a.out) + (size_t)n * a.ld);
#pragma unroll
  for (int j = 0; j < A; ++j) {
    const int i = first + j * 32;
    if (i >= accesses) continue;
    if (a.scale != 1.f && inside) {
#pragma unroll
      for (int e = 0; e < E; ++e) x[j].v[e] = Elem<T>::down(Elem<T>::up(x[j].v[e]) * a.scale);
    }
    store_streaming(dst + i, x[j]);
  }
}

// ---- sort of the positions by token ------------------------------------------
// Least-significant-digit radix sort by one cluster of kSortCtas CTAs. Each
// warp of the cluster owns a contiguous part of the sequence; a pass counts the
// digits of every part, turns the counts into the first place of each (digit,
// part) pair, and moves the entries in order. The CTAs exchange their counts
// through distributed shared memory and the entries through L2. Latency bounds it
// (8192 tokens: 13 us for two passes, mostly barriers); one cluster, since more
// CTAs would have to meet through global memory.

constexpr int kSortCtas = 8;
constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxDigitBits = 9;  // a thread per digit
static_assert((1 << kMaxDigitBits) <= kSortThreads && kSortWarps <= 32, "sort_pass's layout");
constexpr int kKeys = 4;  // keys of a lane whose loads are in flight at once

struct SortArgs {
  Ids tokens;
  int N, vocab;
  int digit_bits, passes;
  uint32_t* key[2];
  int* pos[2];
};

struct SortShared {
  uint32_t hist[1 << kMaxDigitBits];  // this CTA's digit counts, read by the others
  uint32_t base[1 << kMaxDigitBits];  // first place of this CTA's entries of a digit
  uint32_t warp_sum[kSortWarps];
};

size_t sort_smem(int digit_bits) {
  return sizeof(SortShared) + ((size_t)kSortWarps << digit_bits) * sizeof(uint32_t);
}

// Pass 0 reads the tokens (one outside the vocabulary gets the key `vocab`,
// after every real one) and writes buffer 0; pass p moves buffer (p - 1) & 1
// to buffer p & 1.
__device__ void sort_pass(const SortArgs& a, int pass, SortShared* sh, uint32_t* place) {
  cg::cluster_group cluster = cg::this_cluster();
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int cta = (int)cluster.block_rank();
  const int D = 1 << a.digit_bits;
  const int shift = pass * a.digit_bits;
  const uint32_t* in_key = a.key[(pass + 1) & 1];
  const int* in_pos = a.pos[(pass + 1) & 1];
  uint32_t* out_key = a.key[pass & 1];
  int* out_pos = a.pos[pass & 1];
  const long long part = round_up(div_up(a.N, kSortCtas * kSortWarps), 32);
  const long long lo = ((long long)cta * kSortWarps + warp) * part;
  const long long hi = lo + part < a.N ? lo + part : a.N;
  uint32_t* mine = place + warp * D;  // counts, then places, of this warp's entries

  auto key_at = [&](long long i) -> uint32_t {
    if (pass > 0) return __ldcg(in_key + i);
    const long long id = load_id(a.tokens, (size_t)i);
    return (uint32_t)(id >= 0 && id < a.vocab ? id : a.vocab);
  };

  for (int d = lane; d < D; d += 32) mine[d] = 0;
  __syncwarp();
  for (long long i0 = lo; i0 < hi; i0 += 32 * kKeys) {
    uint32_t digit[kKeys];
#pragma unroll
    for (int j = 0; j < kKeys; ++j) {
      const long long i = i0 + j * 32 + lane;
      digit[j] = i < hi ? (key_at(i) >> shift) & (D - 1) : D;
    }
#pragma unroll
    for (int j = 0; j < kKeys; ++j) {
      if (i0 + j * 32 >= hi) break;
      const unsigned peers = __match_any_sync(0xffffffffu, digit[j]);
      if (digit[j] < D && lane == __ffs(peers) - 1) mine[digit[j]] += __popc(peers);
      __syncwarp();
    }
  }
  __syncthreads();
  if (threadIdx.x < D) {
    uint32_t c[kSortWarps], sum = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) c[w] = place[w * D + threadIdx.x];
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      place[w * D + threadIdx.x] = sum;
      sum += c[w];
    }
    sh->hist[threadIdx.x] = sum;
  }
  cluster.sync();
  uint32_t all = 0, before = 0;
  if (threadIdx.x < D) {
#pragma unroll
    for (int c = 0; c < kSortCtas; ++c) {
      const uint32_t x = cluster.map_shared_rank(sh->hist, c)[threadIdx.x];
      if (c < cta) before += x;
      all += x;
    }
  }
  const bool final = pass + 1 == a.passes;
  // The counts have been read: after the last pass nothing else is shared.
  if (final) cluster.barrier_arrive();
  // Exclusive sum of `all` over the digits (threads D.. add nothing).
  uint32_t incl = all;
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) sh->warp_sum[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    uint32_t w = lane < kSortWarps ? sh->warp_sum[lane] : 0;
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += x;
    }
    if (lane < kSortWarps) sh->warp_sum[lane] = w;
  }
  __syncthreads();
  if (threadIdx.x < D)
    sh->base[threadIdx.x] = incl - all + before + (warp ? sh->warp_sum[warp - 1] : 0);
  __syncthreads();
  for (long long i0 = lo; i0 < hi; i0 += 32 * kKeys) {
    uint32_t key[kKeys];
    int from[kKeys];
#pragma unroll
    for (int j = 0; j < kKeys; ++j) {
      const long long i = i0 + j * 32 + lane;
      key[j] = i < hi ? key_at(i) : 0;
      from[j] = i < hi ? (pass > 0 ? __ldcg(in_pos + i) : (int)i) : 0;
    }
#pragma unroll
    for (int j = 0; j < kKeys; ++j) {
      if (i0 + j * 32 >= hi) break;
      const bool on = i0 + j * 32 + lane < hi;
      const uint32_t digit = on ? (key[j] >> shift) & (D - 1) : D;
      const unsigned peers = __match_any_sync(0xffffffffu, digit);
      const int rank = __popc(peers & ((1u << lane) - 1));
      if (on) {
        const uint32_t to = sh->base[digit] + mine[digit] + rank;
        out_key[to] = key[j];
        out_pos[to] = from[j];
      }
      __syncwarp();
      if (on && rank == 0) mine[digit] += __popc(peers);
      __syncwarp();
    }
  }
  if (final)
    cluster.barrier_wait();
  else
    cluster.sync();  // every entry moved, every count read
}

// The successor may start once every CTA here has seen its predecessor complete:
// clear_kernel relies on that.
__global__ void __launch_bounds__(kSortThreads) sort_kernel(const __grid_constant__ SortArgs a) {
  wait_for_predecessor();
  let_successor_start();
  extern __shared__ __align__(16) unsigned char smem[];
  SortShared* sh = reinterpret_cast<SortShared*>(smem);
  uint32_t* place = reinterpret_cast<uint32_t*>(sh + 1);
  for (int p = 0; p < a.passes; ++p) sort_pass(a, p, sh, place);
}

// Few tokens are sorted by counting instead: an entry's place is the number of
// entries before it in the order of (token, position), which one 32-bit word holds
// where both fit. Every CTA reads all the tokens and places kRankItems of them,
// its warps counting over a part of the sequence each: N^2 comparisons, spread over
// the whole GPU, and no exchange between CTAs. (The gradient of 1000 tokens at K=1024,
// added to a table, 8.9 us against 15.0 us by the radix sort; of 4000, 20.8 against
// 17.4 us.)
constexpr int kRankItems = 32;
constexpr int kRankThreads = 512;
constexpr int kRankWarps = kRankThreads / 32;
constexpr int kMaxRankTokens = 2048;

struct RankArgs {
  Ids tokens;
  int N, vocab;
  int pos_bits;
  uint32_t* key;
  int* pos;
};

__global__ void __launch_bounds__(kRankThreads) rank_kernel(const __grid_constant__ RankArgs a) {
  wait_for_predecessor();
  let_successor_start();
  __shared__ uint4 words[kMaxRankTokens / 4];
  __shared__ int part[kRankWarps][kRankItems];
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  uint32_t* const word = reinterpret_cast<uint32_t*>(words);
  const int padded = (int)round_up(a.N, 4);
  constexpr int kLoads = 8;  // tokens of a thread whose loads are in flight at once
  for (int i0 = threadIdx.x; i0 < padded; i0 += kLoads * kRankThreads) {
    long long id[kLoads];
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int i = i0 + j * kRankThreads;
      id[j] = i < a.N ? load_id(a.tokens, (size_t)i) : 0;
    }
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int i = i0 + j * kRankThreads;
      const uint32_t key = (uint32_t)(id[j] >= 0 && id[j] < a.vocab ? id[j] : a.vocab);
      // The padding comes after every entry.
      if (i < padded) word[i] = i < a.N ? key << a.pos_bits | (uint32_t)i : 0xffffffffu;
    }
  }
  __syncthreads();
  const int item = (int)blockIdx.x * kRankItems + lane;
  const uint32_t mine = item < a.N ? word[item] : 0;
  const int quads = padded / 4;
  const int per = (quads + kRankWarps - 1) / kRankWarps;
  const int end = (warp + 1) * per < quads ? (warp + 1) * per : quads;
  int before = 0;
#pragma unroll 4
  for (int q = warp * per; q < end; ++q) {
    const uint4 w = words[q];
    before += (w.x < mine) + (w.y < mine) + (w.z < mine) + (w.w < mine);
  }
  part[warp][lane] = before;
  __syncthreads();
  if (warp || item >= a.N) return;
  int to = 0;
#pragma unroll
  for (int w = 0; w < kRankWarps; ++w) to += part[w][lane];
  a.key[to] = mine >> a.pos_bits;
  a.pos[to] = item;
}

// ---- zeros where no token points ----------------------------------------------

struct ClearArgs {
  Table table;
  size_t bytes;  // of a shard
  int blocks;    // CTAs of one shard
};

constexpr int kClearWords = 8;  // of a thread (128 MB: 18 us, 7.1 TB/s)

// Clears the table beside the sort, whose successor it is on the stream: it
// starts when the sort has started, hence after everything before the sort, and
// needs nothing of it. It waits for the sort before it ends, so that what waits
// for this kernel finds both done.
__global__ void __launch_bounds__(kThreads) clear_kernel(const __grid_constant__ ClearArgs a) {
  let_successor_start();
  const int r = (int)blockIdx.x / a.blocks;
  const int block = (int)blockIdx.x - r * a.blocks;
  unsigned char* const p = static_cast<unsigned char*>(a.table.shard[r]);
  // 16-byte words from the first aligned address on; the ends in 16-bit words.
  size_t head = (16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15;
  if (head > a.bytes) head = a.bytes;
  const size_t words = (a.bytes - head) / 16;
  uint4* const body = reinterpret_cast<uint4*>(p + head);
  const size_t first = (size_t)block * (kThreads * kClearWords) + threadIdx.x;
#pragma unroll
  for (int j = 0; j < kClearWords; ++j)
    if (first + j * kThreads < words) __stcs(body + first + j * kThreads, make_uint4(0, 0, 0, 0));
  if (block == 0 && threadIdx.x < 16) {
    const size_t at = threadIdx.x < 8 ? threadIdx.x * 2 : head + words * 16 + (threadIdx.x - 8) * 2;
    if (at < (threadIdx.x < 8 ? head : a.bytes)) *reinterpret_cast<uint16_t*>(p + at) = 0;
  }
  wait_for_predecessor();
}

// ---- sums over the sorted sequence -------------------------------------------

struct SumArgs {
  Table table;
  const uint32_t* key;
  const int* pos;
  int N, K, W, vocab;
  int run_rows;  // rows of a chunk
  int chunks;
  int slices;  // units of columns of one chunk
  const void* grad;
  size_t ld;
  float scale;
  float* runs;
};

// One lane's columns: U accesses of E elements, 32 accesses apart.
template <typename T, int E, int U>
struct Columns {
  alignas(4 * E) float v[U * E];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < U * E; ++i) v[i] = 0.f;
  }
};

// Load where `on`, without a branch; elsewhere the value is undefined. Between the
// loads of a batch a branch cost more than the loads (the tied table's 8192
// rows: 230 us of sums, against 90 us without the prefetch of the rows added to).
template <typename P>
__device__ __forceinline__ P load_if(const P* p, bool on) {
  P x;
  if constexpr (sizeof(P) == 16) {
    uint4 w;
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.b32 q, %5, 0;\n"
        " @q ld.global.v4.u32 {%0, %1, %2, %3}, [%4];\n}"
        : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
        : "l"(p), "r"((int)on));
    *reinterpret_cast<uint4*>(&x) = w;
  } else if constexpr (sizeof(P) == 4) {
    uint32_t w;
    asm volatile("{\n .reg .pred q;\n setp.ne.b32 q, %2, 0;\n @q ld.global.u32 %0, [%1];\n}"
                 : "=r"(w)
                 : "l"(p), "r"((int)on));
    *reinterpret_cast<uint32_t*>(&x) = w;
  } else {
    uint16_t w;
    asm volatile("{\n .reg .pred q;\n setp.ne.b32 q, %2, 0;\n @q ld.global.u16 %0, [%1];\n}"
                 : "=h"(w)
                 : "l"(p), "r"((int)on));
    *reinterpret_cast<uint16_t*>(&x) = w;
  }
  return x;
}

template <typename P>
__device__ __forceinline__ P* shfl_pointer(P* p, int lane) {
  return reinterpret_cast<P*>(
      __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(p), lane));
}

// `old`: what the row holds, where it is added to.
template <bool ADD, typename T, int E, int U>
__device__ __forceinline__ void write_row(Pack<T, E>* row, float scale, int first, int accesses,
                                          const Columns<T, E, U>& c, const Pack<T, E> (&old)[U]) {
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = first + u * 32;
    if (i >= accesses) continue;
    Pack<T, E> x;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float v = c.v[u * E + e];
      x.v[e] = Elem<T>::down(ADD ? fmaf(scale, v, Elem<T>::up(old[u].v[e])) : scale * v);
    }
    row[i] = x;
  }
}

template <typename T, int E, int U>
__device__ __forceinline__ float* run_slot(const SumArgs& a, long long chunk, int slot) {
  return a.runs + ((size_t)chunk * 2 + slot) * a.K;
}

// Sums of the chunks. The resident CTAs per SM are bounds on the registers: with
// the rows added to in flight as well, 6 (8192 rows at K=7168: 64 us, against 70 us
// with 5 or 8), else 8.
template <typename T, int E, int U, bool ADD>
__global__ void __launch_bounds__(kThreads, U > 1 ? 4 : ADD ? 6 : 8)
    sum_kernel(const __grid_constant__ SumArgs a) {
  wait_for_predecessor();
  let_successor_start();
  constexpr int kBatch = 4;  // rows whose loads are in flight at once
  using P = Pack<T, E>;
  const int lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const long long chunk = unit / a.slices;
  if (chunk >= a.chunks) return;
  const int accesses = a.K / E;
  const int first = (int)(unit - chunk * a.slices) * (32 * U) + lane;
  const long long at = chunk * a.run_rows;
  const int rows = (int)(a.N - at < a.run_rows ? a.N - at : a.run_rows);
  // Lane l holds row l of the chunk; the keys on either side of it.
  const uint32_t none = 0xffffffffu;
  const uint32_t my_key = lane < rows ? a.key[at + lane] : none;
  const uint32_t prev = at > 0 ? a.key[at - 1] : none;
  const uint32_t next = at + rows < a.N ? a.key[at + rows] : none;
  const bool real = lane < rows && my_key < (uint32_t)a.vocab;
  const P* const my_src = reinterpret_cast<const P*>(
      static_cast<const T*>(a.grad) + (size_t)(real ? a.pos[at + lane] : 0) * a.ld);
  P* const my_dst =
      reinterpret_cast<P*>(table_row<T>(a.table, real ? my_key : 0, a.W, a.K));

  Columns<T, E, U> sum;
  sum.clear();
  bool continued = prev == __shfl_sync(0xffffffffu, my_key, 0);
  // Rows that end a run, and those of them that finish it here: not the last of a
  // run that goes on, nor that of one that began earlier.
  const uint32_t my_next = __shfl_down_sync(0xffffffffu, my_key, 1);
  const bool last = lane == rows - 1;
  const int reals = __popc(__ballot_sync(0xffffffffu, real));  // padding sorts to the end
  const unsigned ends = __ballot_sync(0xffffffffu, real && (last || my_next != my_key));
  unsigned finishes = __ballot_sync(0xffffffffu, real && (last ? next : my_next) != my_key);
  if (continued && finishes) finishes &= ~(ends & (0u - ends));
  // Loads go unguarded: past the columns or the rows they repeat the last one.
  int column[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    column[u] = first + u * 32 < accesses ? first + u * 32 : accesses - 1;
  for (int i0 = 0; i0 < reals; i0 += kBatch) {
    P x[kBatch][U], old[kBatch][U];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int i = i0 + b < reals ? i0 + b : reals - 1;
      const P* src = shfl_pointer(my_src, i);
#pragma unroll
      for (int u = 0; u < U; ++u) x[b][u] = src[column[u]];
      if (ADD) {
        const P* dst = shfl_pointer(my_dst, i);
#pragma unroll
        for (int u = 0; u < U; ++u) old[b][u] = load_if(dst + column[u], finishes >> i & 1);
      }
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int i = i0 + b;
      if (i >= reals) break;
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < E; ++e) sum.v[u * E + e] += Elem<T>::up(x[b][u].v[e]);
      if (!(ends >> i & 1)) continue;
      if (finishes >> i & 1) {
        write_row<ADD, T, E, U>(shfl_pointer(my_dst, i), a.scale, first, accesses, sum, old[b]);
      } else {
        float* slot = run_slot<T, E, U>(a, chunk, continued ? 0 : 1);
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (first + u * 32 < accesses) {
            reinterpret_cast<Pack<float, E>*>(slot)[first + u * 32] =
                *reinterpret_cast<const Pack<float, E>*>(&sum.v[u * E]);
          }
      }
      sum.clear();
      continued = false;
    }
  }
}

// Joins the runs that cross a chunk's end: the warp of the chunk a run starts
// in adds that chunk's slot 1 and slot 0 of the chunks after it, in order.
template <typename T, int E, int U, bool ADD>
__global__ void __launch_bounds__(kThreads) join_kernel(const __grid_constant__ SumArgs a) {
  wait_for_predecessor();
  let_successor_start();
  constexpr int kBatch = 4;
  const int lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const long long chunk = unit / a.slices;
  if (chunk + 1 >= a.chunks) return;
  const int accesses = a.K / E;
  const int first = (int)(unit - chunk * a.slices) * (32 * U) + lane;
  const long long at = chunk * a.run_rows;
  const uint32_t key = a.key[at + a.run_rows - 1];
  if (key >= (uint32_t)a.vocab || a.key[at + a.run_rows] != key) return;    // does not go on
  if (a.key[at] == key && at > 0 && a.key[at - 1] == key) return;  // starts earlier
  // Last chunk of the run: the first whose own last row is not of the run, or
  // whose last row ends it.
  long long last = chunk + 1;
  for (;; last += 32) {
    const long long c = last + lane;
    const bool ends = c + 1 >= a.chunks || a.key[(c + 1) * a.run_rows] != key;
    const unsigned m = __ballot_sync(0xffffffffu, ends);
    if (m) {
      last += __ffs(m) - 1;
      break;
    }
  }
  Pack<T, E>* const row = reinterpret_cast<Pack<T, E>*>(table_row<T>(a.table, key, a.W, a.K));
  Pack<T, E> old[U];
  if (ADD) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (first + u * 32 < accesses) old[u] = row[first + u * 32];
  }
  Columns<T, E, U> sum;
  const Pack<float, E>* src =
      reinterpret_cast<const Pack<float, E>*>(run_slot<T, E, U>(a, chunk, 1));
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (first + u * 32 < accesses)
      *reinterpret_cast<Pack<float, E>*>(&sum.v[u * E]) = src[first + u * 32];
  for (long long c0 = chunk + 1; c0 <= last; c0 += kBatch) {
    Pack<float, E> x[kBatch][U];
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (c0 + b <= last && first + u * 32 < accesses)
          x[b][u] = reinterpret_cast<const Pack<float, E>*>(
              run_slot<T, E, U>(a, c0 + b, 0))[first + u * 32];
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (c0 + b <= last && first + u * 32 < accesses) {
#pragma unroll
          for (int e = 0; e < E; ++e) sum.v[u * E + e] += x[b][u].v[e];
        }
  }
  write_row<ADD, T, E, U>(row, a.scale, first, accesses, sum, old);
}

// Widest access that every row of the matrices allows: 16 bytes, 4, or an element.
int access_bytes(int K, size_t ld, const void* p, const Table& t, int tp, size_t elem) {
  size_t bits = (size_t)K * elem | ld * elem | reinterpret_cast<uintptr_t>(p);
  for (int r = 0; r < tp; ++r) bits |= reinterpret_cast<uintptr_t>(t.shard[r]);
  return bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : (int)elem;
}

template <typename T, int E, int A>
cudaError_t embed_as(const EmbedArgs& args, cudaStream_t stream) {
  EmbedArgs a = args;
  a.units_per_row = (int)div_up(a.K / E, A * 32);
  const long long blocks = div_up((long long)a.N * a.units_per_row, kLookupThreads / 32);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_dependent(embed_kernel<T, E, A>, a, (unsigned)blocks, kLookupThreads, 0, 1, stream);
}

template <typename T, int E, int U, bool ADD>
cudaError_t sum_as(const SumArgs& args, cudaStream_t stream) {
  SumArgs a = args;
  a.slices = (int)div_up(a.K / E, 32 * U);
  const long long blocks = div_up((long long)a.chunks * a.slices, kWarps);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  const cudaError_t e =
      launch_dependent(sum_kernel<T, E, U, ADD>, a, (unsigned)blocks, kThreads, 0, 1, stream);
  if (e != cudaSuccess || a.chunks == 1) return e;
  return launch_dependent(join_kernel<T, E, U, ADD>, a, (unsigned)blocks, kThreads, 0, 1, stream);
}

template <typename T, int E, int U>
cudaError_t sum_for(const SumArgs& a, bool accumulate, cudaStream_t stream) {
  return accumulate ? sum_as<T, E, U, true>(a, stream) : sum_as<T, E, U, false>(a, stream);
}

// Sorts the positions by token into buffer *sorted.
cudaError_t sort(const hg_vocab& h, const Ids& tokens, int N, int* sorted, cudaStream_t stream) {
  SortArgs a = {};
  a.tokens = tokens;
  a.N = N;
  a.vocab = h.vocab;
  int bits = 1;
  while ((1ll << bits) <= h.vocab) ++bits;  // keys 0 .. vocab
  int pos_bits = 1;
  while ((1ll << pos_bits) < N) ++pos_bits;
  // The largest word, (vocab, N - 1), stays below the padding's 0xffffffff.
  if (N > 0 && N <= kMaxRankTokens &&
      ((unsigned long long)h.vocab << pos_bits | (unsigned)(N - 1)) < 0xffffffffull) {
    RankArgs r = {};
    r.tokens = tokens;
    r.N = N;
    r.vocab = h.vocab;
    r.pos_bits = pos_bits;
    r.key = h.key[0];
    r.pos = h.pos[0];
    *sorted = 0;
    return launch_dependent(rank_kernel, r, (unsigned)div_up(N, kRankItems), kRankThreads, 0, 1,
                            stream);
  }
  a.passes = (bits + kMaxDigitBits - 1) / kMaxDigitBits;
  a.digit_bits = (bits + a.passes - 1) / a.passes;
  for (int i = 0; i < 2; ++i) {
    a.key[i] = h.key[i];
    a.pos[i] = h.pos[i];
  }
  *sorted = (a.passes + 1) & 1;
  return launch_dependent(sort_kernel, a, kSortCtas, kSortThreads, sort_smem(a.digit_bits),
                          kSortCtas, stream);
}

cudaError_t clear(const hg_vocab& h, const Table& table, cudaStream_t stream) {
  ClearArgs a = {};
  a.table = table;
  a.bytes = (size_t)h.W * h.K * elem_bytes(h.dtype);
  const long long blocks = div_up((long long)a.bytes, kThreads * kClearWords * 16);
  if (blocks * h.tp > 0x7fffffffLL) return cudaErrorInvalidValue;
  a.blocks = (int)blocks;
  return launch_dependent(clear_kernel, a, (unsigned)(blocks * h.tp), kThreads, 0, 1, stream);
}

// Rows of a chunk: kRunRows, but fewer where that leaves too few warps to hide
// the loads' latency (at 3001 rows of 1001 fp32 the sums took 15 us).
// The fewest rows are one chunk, and need no join.
int run_rows(const hg_vocab& h, int N) {
  if (N <= 2 * kFewRunRows) return 2 * kFewRunRows;
  const long long slices = div_up(h.K, 128);
  const long long enough = 16ll * h.sms;
  return div_up(N, kRunRows) * slices >= enough ? kRunRows : kFewRunRows;
}

}  // namespace

cudaError_t embed(const hg_vocab& h, const Ids& tokens, int N, const void* const* table,
                  float scale, void* out, size_t ld_out, cudaStream_t stream) {
  EmbedArgs a = {};
  for (int r = 0; r < h.tp; ++r) a.table.shard[r] = const_cast<void*>(table[r]);
  a.tokens = tokens;
  a.N = N;
  a.K = h.K;
  a.W = h.W;
  a.vocab = h.vocab;
  a.scale = scale;
  a.out = out;
  a.ld = ld_out;
  const int bytes = access_bytes(h.K, ld_out, out, a.table, h.tp, elem_bytes(h.dtype));
  switch (h.dtype) {
    case HG_BF16:
      return bytes == 16  ? embed_as<__nv_bfloat16, 8, 4>(a, stream)
             : bytes == 4 ? embed_as<__nv_bfloat16, 2, 8>(a, stream)
                          : embed_as<__nv_bfloat16, 1, 16>(a, stream);
    case HG_FP16:
      return bytes == 16  ? embed_as<__half, 8, 4>(a, stream)
             : bytes == 4 ? embed_as<__half, 2, 8>(a, stream)
                          : embed_as<__half, 1, 16>(a, stream);
    default:
      return bytes == 16 ? embed_as<float, 4, 4>(a, stream) : embed_as<float, 1, 8>(a, stream);
  }
}

cudaError_t embed_prepare() {
  return cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)sort_smem(kMaxDigitBits));
}

long long embed_grad_chunks(const hg_vocab& h) {
  // Short chunks are the most just before long ones take over.
  const long long all = div_up(h.max_rows, run_rows(h, h.max_rows));
  long long n = 16ll * h.sms / div_up(h.K, 128) * kRunRows + kRunRows;
  if (n > h.max_rows) n = h.max_rows;
  const long long most = div_up(n, kFewRunRows);
  return all > most ? all : most;
}

cudaError_t embed_grad(const hg_vocab& h, const Ids& tokens, int N, const void* grad,
                       size_t ld_grad, void* const* table, float scale, bool accumulate,
                       cudaStream_t stream) {
  SumArgs a = {};
  const size_t e = elem_bytes(h.dtype);
  for (int r = 0; r < h.tp; ++r) a.table.shard[r] = table[r];
  int sorted = 0;
  // The sort runs for no tokens too: the clear starts after it.
  cudaError_t st = sort(h, tokens, N, &sorted, stream);
  if (st == cudaSuccess && !accumulate) st = clear(h, a.table, stream);
  if (st != cudaSuccess || N == 0) return st;
  a.key = h.key[sorted];
  a.pos = h.pos[sorted];
  a.N = N;
  a.K = h.K;
  a.W = h.W;
  a.vocab = h.vocab;
  a.run_rows = run_rows(h, N);
  a.chunks = (int)div_up(N, a.run_rows);
  a.grad = grad;
  a.ld = ld_grad;
  a.scale = scale;
  a.runs = h.runs;
  const int bytes = access_bytes(h.K, ld_grad, grad, a.table, h.tp, e);
  switch (h.dtype) {
    case HG_BF16:
      return bytes == 16  ? sum_for<__nv_bfloat16, 8, 1>(a, accumulate, stream)
             : bytes == 4 ? sum_for<__nv_bfloat16, 2, 8>(a, accumulate, stream)
                          : sum_for<__nv_bfloat16, 1, 8>(a, accumulate, stream);
    case HG_FP16:
      return bytes == 16  ? sum_for<__half, 8, 1>(a, accumulate, stream)
             : bytes == 4 ? sum_for<__half, 2, 8>(a, accumulate, stream)
                          : sum_for<__half, 1, 8>(a, accumulate, stream);
    default:
      return bytes == 16 ? sum_for<float, 4, 1>(a, accumulate, stream)
                         : sum_for<float, 1, 4>(a, accumulate, stream);
  }
}

}  // namespace vocab
}  // namespace hg
