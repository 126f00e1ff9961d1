// States follow their beams, in place.
//
// A thread owns one column of an item's rows, an access of up to 16 bytes: it reads
// that column of every row that some other row takes, and then writes it to
// the rows that move. No thread touches another's columns, so nothing is copied
// twice and no barrier stands between the reads and the writes. Memory bounds it.

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

constexpr int kMoveThreads = 128;
constexpr int kInFlight = 8;  // loads of a thread that are under way at once
constexpr int kStates = 32;   // states of one launch

struct State {
  unsigned char* data;
  size_t outer_stride, row_stride, piece_stride;
  unsigned long long columns;     // accesses of one row
  unsigned long long first_unit;  // units of the states before this one
  unsigned long long chunks;      // units of one item
  unsigned long long pieces, accesses;  // accesses: of one run
  int bytes;                      // of an access
};

struct ReorderArgs {
  State state[kStates];
  Ids parents;
  int n_states, beams;
  unsigned long long units;
};

__device__ __forceinline__ unsigned long long quotient(unsigned long long a,
                                                       unsigned long long b) {
  return (a | b) >> 32 ? a / b : (uint32_t)a / (uint32_t)b;
}

template <typename W>
__device__ __forceinline__ void move(const State& s, size_t row0, unsigned long long column,
                                     unsigned long long needed, unsigned long long moved,
                                     const int* parent, W* held) {
  if (column >= s.columns) return;
  const unsigned long long run = quotient(column, s.accesses);
  const unsigned long long o = quotient(run, s.pieces);
  unsigned char* at = s.data + row0 * s.row_stride + o * s.outer_stride +
                      (run - o * s.pieces) * s.piece_stride +
                      (column - run * s.accesses) * sizeof(W);
  while (needed) {
    W v[kInFlight];
    int b[kInFlight];
#pragma unroll
    for (int i = 0; i < kInFlight; ++i) {
      b[i] = __ffsll((long long)needed) - 1;
      if (b[i] >= 0) {
        needed &= needed - 1;
        v[i] = *reinterpret_cast<const W*>(at + b[i] * s.row_stride);
      }
    }
#pragma unroll
    for (int i = 0; i < kInFlight; ++i)
      if (b[i] >= 0) held[b[i] * kMoveThreads] = v[i];
  }
  for (; moved; moved &= moved - 1) {
    const int j = __ffsll((long long)moved) - 1;
    *reinterpret_cast<W*>(at + j * s.row_stride) = held[parent[j] * kMoveThreads];
  }
}

__global__ void __launch_bounds__(kMoveThreads) reorder_kernel(const __grid_constant__ ReorderArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ int parent[HG_MAX_BEAMS];
  wait_for_predecessor();
  let_successor_start();
  int i = 0;
  for (unsigned long long unit = blockIdx.x; unit < a.units; unit += gridDim.x) {
    while (i + 1 < a.n_states && unit >= a.state[i + 1].first_unit) ++i;
    const State& s = a.state[i];
    const unsigned long long at = unit - s.first_unit;
    const unsigned long long item = at / s.chunks;
    const size_t row0 = item * a.beams;
    __syncthreads();
    if (threadIdx.x < a.beams) {
      const long long p = load_id(a.parents, row0 + threadIdx.x);
      parent[threadIdx.x] = p >= 0 && p < a.beams ? (int)p : (int)threadIdx.x;
    }
    __syncthreads();
    unsigned long long needed = 0, moved = 0;
    for (int j = 0; j < a.beams; ++j)
      if (parent[j] != j) {
        needed |= 1ull << parent[j];
        moved |= 1ull << j;
      }
    const unsigned long long column = (at - item * s.chunks) * kMoveThreads + threadIdx.x;
    switch (s.bytes) {
      case 16:
        move(s, row0, column, needed, moved, parent, reinterpret_cast<uint4*>(smem) + threadIdx.x);
        break;
      case 4:
        move(s, row0, column, needed, moved, parent,
             reinterpret_cast<uint32_t*>(smem) + threadIdx.x);
        break;
      case 2:
        move(s, row0, column, needed, moved, parent,
             reinterpret_cast<uint16_t*>(smem) + threadIdx.x);
        break;
      default:
        move(s, row0, column, needed, moved, parent, smem + threadIdx.x);
    }
  }
}

}  // namespace

cudaError_t reorder(const hg_beam& h, const void* parents, int id_bytes, int items,
                    const hg_beam_state* states, int n_states, cudaStream_t stream) {
  const size_t smem = (size_t)h.beams * kMoveThreads * 16;
  for (int next = 0; next < n_states;) {
    ReorderArgs a = {};
    a.parents = Ids{parents, id_bytes};
    a.beams = h.beams;
    for (; next < n_states && a.n_states < kStates; ++next) {
      const hg_beam_state& in = states[next];
      if (in.outer == 0 || in.pieces == 0 || in.piece_bytes == 0) continue;
      State& s = a.state[a.n_states];
      s.data = static_cast<unsigned char*>(in.data);
      s.outer_stride = in.outer_stride;
      s.row_stride = in.row_stride;
      s.piece_stride = in.piece_stride;
      size_t bits = reinterpret_cast<uintptr_t>(in.data) | in.piece_bytes | in.row_stride;
      if (in.outer > 1) bits |= in.outer_stride;
      if (in.pieces > 1) bits |= in.piece_stride;
      s.bytes = bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : bits % 2 == 0 ? 2 : 1;
      s.pieces = in.pieces;
      s.accesses = in.piece_bytes / s.bytes;
      s.columns = in.outer * in.pieces * s.accesses;
      s.chunks = (unsigned long long)div_up((long long)s.columns, kMoveThreads);
      s.first_unit = a.units;
      a.units += s.chunks * items;
      ++a.n_states;
    }
    if (a.units == 0) continue;
    const unsigned long long most = (unsigned long long)h.sms * 16;
    const unsigned grid = (unsigned)(a.units < most ? a.units : most);
    const cudaError_t e = launch_dependent(reorder_kernel, a, grid, kMoveThreads, smem, 1, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t reorder_prepare() {
  return cudaFuncSetAttribute(reorder_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              HG_MAX_BEAMS * kMoveThreads * 16);
}

}  // namespace beam
}  // namespace hg
