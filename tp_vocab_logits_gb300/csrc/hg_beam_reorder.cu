// States follow their beams, in place.
//
// A thread owns columns of an item's rows, accesses of up to 16 bytes: it reads such a
// column of every row that some other row takes, and then writes it to the rows that move.
// No thread touches another's columns, so a row is read and written once and no barrier
// stands between the two. The reads of a thread's next columns, copied straight into its own
// places in shared memory, are under way while it writes these, and a CTA goes through
// neighbouring columns. Memory bounds it, once the instructions do not: a warp lists an
// item's rows when it comes to it, and a thread moves two columns by that list (32 items
// of 8 beams, 1.49 GB read and written: 243 us, 6.1 TB/s; 284 us with the rows looked up for
// each column, 289 us with four columns a thread, which leaves too few warps).

#include "hg_beam.cuh"

namespace hg {
namespace beam {
namespace {

using vocab::Ids;
using vocab::div_up;
using vocab::launch_dependent;
using vocab::let_successor_start;
using vocab::load_id;
using vocab::wait_for_predecessor;

typedef unsigned long long u64;

constexpr int kMoveThreads = 128;
constexpr int kColumns = 2;      // of a thread at a time
constexpr int kStates = 32;     // states of one launch
constexpr size_t kNarrowMost = 1 << 20;  // bytes of rows in short accesses beside 16-byte ones
constexpr size_t kMoveMost = 136 * 1024;  // shared memory of a CTA's columns
static_assert((size_t)2 * HG_MAX_BEAMS * kColumns * 32 * 16 <= kMoveMost, "at least a warp");
constexpr size_t kSharedOfSm = 228 * 1024;

struct State {
  unsigned char* data;
  size_t outer_stride, row_stride, piece_stride;
  u64 columns;           // accesses of one row
  u64 first_unit;        // units of the states before this one
  u64 chunks;            // units of one item
  u64 pieces, accesses;  // accesses: of one run
  Divisor by_pieces, by_accesses;
  int bytes;             // of an access
};

struct ReorderArgs {
  State state[kStates];
  Ids parents;
  int n_states, beams;
  u64 units, each, more;  // units of a CTA; the first `more` CTAs have one more
};

// What a warp does with an item's rows of a state, as distances in bytes from its first row.
struct Moves {
  u64 from[HG_MAX_BEAMS];  // rows that others take
  u64 to[HG_MAX_BEAMS];    // rows that take another: the one that is in place `place`
  int place[HG_MAX_BEAMS];
  int reads, writes;
};

__device__ __forceinline__ void list_moves(Moves& m, const ReorderArgs& a, const State& s,
                                           size_t item) {
  const int lane = threadIdx.x & 31;
  int of[2];
  uint32_t need[2] = {}, move[2] = {};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int j = h * 32 + lane;
    of[h] = j;
    if (j < a.beams) {
      const long long p = load_id(a.parents, item * a.beams + j);
      if (p >= 0 && p < a.beams) of[h] = (int)p;
    }
    const bool moves = of[h] != j;
    move[h] = __ballot_sync(0xffffffffu, moves);
#pragma unroll
    for (int k = 0; k < 2; ++k)
      need[k] |=
          __reduce_or_sync(0xffffffffu, moves && of[h] / 32 == k ? 1u << of[h] % 32 : 0u);
  }
  auto before = [](const uint32_t (&mask)[2], int b) {
    return b < 32 ? __popc(mask[0] & ((1u << b) - 1))
                  : __popc(mask[0]) + __popc(mask[1] & ((1u << (b - 32)) - 1));
  };
  __syncwarp();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int j = h * 32 + lane;
    if (need[h] >> lane & 1) m.from[before(need, j)] = j * s.row_stride;
    if (move[h] >> lane & 1) {
      const int k = before(move, j);
      m.to[k] = j * s.row_stride;
      m.place[k] = before(need, of[h]);
    }
  }
  if (lane == 0) {
    m.reads = __popc(need[0]) + __popc(need[1]);
    m.writes = __popc(move[0]) + __popc(move[1]);
  }
  __syncwarp();
}

// A thread's columns of a unit, and what is done with them.
struct Columns {
  unsigned char* at[kColumns];  // in the item's first row; null: none
  int bytes;
  int moves;  // which list
};

// Goes through units, one after another, listing an item's moves where it changes.
struct Cursor {
  int i = 0;
  u64 item = 0, chunk = 0;
  int list = 1;

  __device__ __forceinline__ void enter(const ReorderArgs& a, u64 unit, Moves* moves) {
    while (i + 1 < a.n_states && unit >= a.state[i + 1].first_unit) ++i;
    const u64 in = unit - a.state[i].first_unit;
    item = in / a.state[i].chunks;
    chunk = in - item * a.state[i].chunks;
    list ^= 1;
    list_moves(moves[list], a, a.state[i], item);
  }
  __device__ __forceinline__ void step(const ReorderArgs& a, u64 unit, Moves* moves) {
    if (++chunk == a.state[i].chunks) enter(a, unit, moves);
  }
  __device__ __forceinline__ Columns columns(const ReorderArgs& a) const {
    const State& s = a.state[i];
    Columns c;
    c.bytes = s.bytes;
    c.moves = list;
    unsigned char* const first = s.data + item * a.beams * s.row_stride;
    const bool wide = s.columns >> 31;
#pragma unroll
    for (int k = 0; k < kColumns; ++k) {
      const u64 column = (chunk * kColumns + k) * blockDim.x + threadIdx.x;
      u64 run, o;
      if (wide) {
        run = column / s.accesses;
        o = run / s.pieces;
      } else {
        run = (u64)s.by_accesses.divide((int)column);
        o = (u64)s.by_pieces.divide((int)run);
      }
      c.at[k] = column < s.columns
                    ? first + o * s.outer_stride + (run - o * s.pieces) * s.piece_stride +
                          (column - run * s.accesses) * s.bytes
                    : nullptr;
    }
    return c;
  }
};

template <int BYTES>
__device__ __forceinline__ void copy_ahead(void* to, const void* from) {
  const uint32_t at = (uint32_t)__cvta_generic_to_shared(to);
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(at), "l"(from) : "memory");
}

// W: an access. SLOT: a column's place in shared memory. Those too short to be copied ahead are loaded for a few rows at a time.
template <typename W, typename SLOT>
__device__ __forceinline__ void read_as(const Columns& c, const Moves& m, SLOT* held) {
  const int n = m.reads;
  if constexpr (sizeof(W) >= 4) {
    for (int r = 0; r < n; ++r) {
      const u64 from = m.from[r];
#pragma unroll
      for (int k = 0; k < kColumns; ++k)
        if (c.at[k])
          copy_ahead<sizeof(W)>(held + (r * kColumns + k) * blockDim.x, c.at[k] + from);
    }
  } else {
    constexpr int kRows = 8;
    for (int r0 = 0; r0 < n; r0 += kRows) {
      W v[kRows][kColumns];
#pragma unroll
      for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int k = 0; k < kColumns; ++k)
          if (r0 + r < n && c.at[k]) v[r][k] = *reinterpret_cast<const W*>(c.at[k] + m.from[r0 + r]);
#pragma unroll
      for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int k = 0; k < kColumns; ++k)
          if (r0 + r < n && c.at[k])
            *reinterpret_cast<W*>(held + ((r0 + r) * kColumns + k) * blockDim.x) = v[r][k];
    }
  }
}

template <typename W, typename SLOT>
__device__ __forceinline__ void write_as(const Columns& c, const Moves& m, const SLOT* held) {
  const int n = m.writes;
#pragma unroll 2
  for (int w = 0; w < n; ++w) {
    const u64 to = m.to[w];
    const SLOT* from = held + m.place[w] * kColumns * blockDim.x;
    W v[kColumns];
#pragma unroll
    for (int k = 0; k < kColumns; ++k) v[k] = *reinterpret_cast<const W*>(from + k * blockDim.x);
#pragma unroll
    for (int k = 0; k < kColumns; ++k)
      if (c.at[k]) *reinterpret_cast<W*>(c.at[k] + to) = v[k];
  }
}

template <typename SLOT>
__device__ __forceinline__ void read(const Columns& c, const Moves& m, SLOT* held) {
  if constexpr (sizeof(SLOT) == 16)
    if (c.bytes == 16) return read_as<uint4>(c, m, held);
  if (c.bytes == 4)
    read_as<uint32_t>(c, m, held);
  else if (c.bytes == 2)
    read_as<uint16_t>(c, m, held);
  else
    read_as<unsigned char>(c, m, held);
}
template <typename SLOT>
__device__ __forceinline__ void write(const Columns& c, const Moves& m, const SLOT* held) {
  if constexpr (sizeof(SLOT) == 16)
    if (c.bytes == 16) return write_as<uint4>(c, m, held);
  if (c.bytes == 4)
    write_as<uint32_t>(c, m, held);
  else if (c.bytes == 2)
    write_as<uint16_t>(c, m, held);
  else
    write_as<unsigned char>(c, m, held);
}

// SLOT of 32 bits: of accesses of 4 bytes and less, which leave most of 16 bytes unused and with
// them the room for threads (9 items of 28 beams, 85 MB in 2-byte accesses: 669 and 50 us).
template <typename SLOT>
__global__ void __launch_bounds__(kMoveThreads)
    reorder_kernel(const __grid_constant__ ReorderArgs a) {
  extern __shared__ uint4 smem[];  // [2][beams][kColumns][threads] of SLOT
  __shared__ Moves lists[kMoveThreads / 32][2];  // of this unit and of the next
  wait_for_predecessor();
  let_successor_start();
  Moves* const moves = lists[threadIdx.x >> 5];
  SLOT* const slots = reinterpret_cast<SLOT*>(smem) + threadIdx.x;
  SLOT* const held[2] = {slots, slots + a.beams * kColumns * blockDim.x};
  const u64 cta = blockIdx.x;
  u64 unit = cta * a.each + min(cta, a.more);
  const u64 last = unit + a.each + (cta < a.more ? 1 : 0) - 1;
  Cursor cursor;
  cursor.enter(a, unit, moves);
  Columns columns = cursor.columns(a);
  read(columns, moves[columns.moves], held[0]);
  asm volatile("cp.async.commit_group;" ::: "memory");
  for (int side = 0;; side ^= 1) {
    Columns next = columns;
    if (unit < last) {
      cursor.step(a, unit + 1, moves);
      next.moves = cursor.list;
      if (moves[cursor.list].writes > 0) {
        next = cursor.columns(a);
        read(next, moves[next.moves], held[side ^ 1]);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    write(columns, moves[columns.moves], held[side]);
    if (unit++ == last) break;
    columns = next;
  }
}

}  // namespace

namespace {

// Bytes of a state's accesses; 0: there is nothing in it.
int access_of(const hg_beam_state& s) {
  if (s.outer == 0 || s.pieces == 0 || s.piece_bytes == 0) return 0;
  size_t bits = reinterpret_cast<uintptr_t>(s.data) | s.piece_bytes | s.row_stride;
  if (s.outer > 1) bits |= s.outer_stride;
  if (s.pieces > 1) bits |= s.piece_stride;
  return bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : bits % 2 == 0 ? 2 : 1;
}

// The states whose accesses are of `least` to `widest` bytes, 32 a launch.
template <typename SLOT>
cudaError_t reorder_as(int least, int widest, const hg_beam& h, const void* parents, int id_bytes, int items,
                       const hg_beam_state* states, int n_states, cudaStream_t stream) {
  // As many threads as the shared memory of their columns allows, and CTAs to fill an SM.
  int threads = kMoveThreads;
  while ((size_t)2 * h.beams * kColumns * threads * sizeof(SLOT) > kMoveMost) threads /= 2;
  const size_t smem = (size_t)2 * h.beams * kColumns * threads * sizeof(SLOT);
  const u64 room = kSharedOfSm / (smem + sizeof(Moves) * 2 * kMoveThreads / 32 + 1024);
  const u64 per_sm = room < (u64)(2048 / threads) ? room : (u64)(2048 / threads);
  for (int next = 0; next < n_states;) {
    ReorderArgs a = {};
    a.parents = Ids{parents, id_bytes};
    a.beams = h.beams;
    for (; next < n_states && a.n_states < kStates; ++next) {
      const hg_beam_state& in = states[next];
      const int bytes = access_of(in);
      if (bytes < least || bytes > widest) continue;
      State& s = a.state[a.n_states];
      s.data = static_cast<unsigned char*>(in.data);
      s.outer_stride = in.outer_stride;
      s.row_stride = in.row_stride;
      s.piece_stride = in.piece_stride;
      s.bytes = bytes;
      s.pieces = in.pieces;
      s.accesses = in.piece_bytes / s.bytes;
      s.columns = in.outer * in.pieces * s.accesses;
      if (!(s.columns >> 31)) {
        s.by_pieces = Divisor((uint32_t)s.pieces);
        s.by_accesses = Divisor((uint32_t)s.accesses);
      }
      s.chunks = (u64)div_up((long long)s.columns, (long long)threads * kColumns);
      s.first_unit = a.units;
      a.units += s.chunks * items;
      ++a.n_states;
    }
    if (a.units == 0) continue;
    const u64 most = (u64)h.sms * per_sm;
    const unsigned grid = (unsigned)(a.units < most ? a.units : most);
    a.each = a.units / grid;
    a.more = a.units % grid;
    const cudaError_t e =
        launch_dependent(reorder_kernel<SLOT>, a, grid, (unsigned)threads, smem, 1, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t reorder(const hg_beam& h, const void* parents, int id_bytes, int items,
                    const hg_beam_state* states, int n_states, cudaStream_t stream) {
  if (h.beams == 1) return cudaSuccess;  // no row has another to take
  // Short accesses have a launch of their own where they are many, or alone: it takes 1.5 us.
  size_t narrow = 0;
  bool wide = false;
  for (int i = 0; i < n_states; ++i) {
    const hg_beam_state& s = states[i];
    const int bytes = access_of(s);
    if (bytes == 16) wide = true;
    if (bytes > 0 && bytes < 16) narrow += s.outer * s.pieces * s.piece_bytes * items * h.beams;
  }
  const int least = !wide || narrow > kNarrowMost ? 16 : 1;
  const cudaError_t e =
      wide ? reorder_as<uint4>(least, 16, h, parents, id_bytes, items, states, n_states, stream)
           : cudaSuccess;
  return e == cudaSuccess && least == 16 && narrow > 0
             ? reorder_as<uint32_t>(1, 4, h, parents, id_bytes, items, states, n_states, stream)
             : e;
}

cudaError_t reorder_prepare() {
  const cudaError_t e = cudaFuncSetAttribute(
      reorder_kernel<uint4>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMoveMost);
  return e == cudaSuccess ? cudaFuncSetAttribute(reorder_kernel<uint32_t>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 (int)kMoveMost)
                          : e;
}

}  // namespace beam
}  // namespace hg
