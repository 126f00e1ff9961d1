// Host side of the beam search declared in include/hg.h: the handle, its workspace
// and the argument checks.

#include <algorithm>
#include <climits>
#include <functional>
#include <new>

#include "hg_beam.cuh"
#include "hg_overlap.cuh"

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool ids_ok(const void* p, int id_bytes) {
  return (id_bytes == 4 || id_bytes == 8) && p && aligned(p, (size_t)id_bytes);
}

int as_status(cudaError_t e) { return e == cudaSuccess ? HG_OK : HG_ERR_CUDA; }

// The handle's workspace and the caller's tensors are of one device: with another
// one current, the kernels would start there, on pointers it cannot reach.
int check_device(const hg_beam* h) {
  int current = -1;
  if (cudaGetDevice(&current) != cudaSuccess) {
    cudaGetLastError();
    return HG_ERR_CUDA;
  }
  return current == h->device ? HG_OK : HG_ERR_ARG;
}

// The runs of a state do not overlap: taken from the shortest stride to the longest,
// each dimension steps over all that the ones before it span.
bool state_ok(const hg_beam_state& s, size_t rows) {
  if (s.outer == 0 || s.pieces == 0 || s.piece_bytes == 0) return true;  // nothing in it
  if (!s.data) return false;
  struct Dim {
    size_t count, stride;
  } dim[3] = {{s.outer, s.outer_stride}, {rows, s.row_stride}, {s.pieces, s.piece_stride}};
  std::sort(dim, dim + 3, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
  constexpr size_t kMost = (size_t)1 << 60;
  size_t span = s.piece_bytes;
  if (span > kMost) return false;
  for (const Dim& d : dim) {
    if (d.count == 1) continue;
    if (d.stride < span || d.stride > kMost / d.count) return false;
    span += d.stride * (d.count - 1);
    if (span > kMost) return false;
  }
  return true;
}

// Whether [from, to), as a distance in bytes from the state's data, holds a part of its runs. A
// dimension of a larger stride steps over all that those of smaller ones span.
bool state_holds(const hg_beam_state& s, size_t rows, long long from, long long to) {
  struct Dim {
    long long count, stride;
  } dim[3] = {{(long long)s.outer, (long long)s.outer_stride},
              {(long long)rows, (long long)s.row_stride},
              {(long long)s.pieces, (long long)s.piece_stride}};
  long long span[4] = {(long long)s.piece_bytes};
  for (Dim& d : dim)
    if (d.count == 1) d.stride = 0;
  std::sort(dim, dim + 3, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
  for (int k = 0; k < 3; ++k) span[k + 1] = span[k] + dim[k].stride * (dim[k].count - 1);
  // What `level` dimensions span, from `at` on. A part that lies inside whole holds a run; at most
  // two of a dimension's parts lie inside in part.
  auto inside = [&](auto& self, int level, long long at) -> bool {
    if (at >= to || at + span[level] <= from) return false;
    if (level == 0 || (from <= at && at + span[level] <= to)) return true;
    const Dim& d = dim[level - 1];
    if (d.stride == 0) return self(self, level - 1, at);
    const long long before = from - at - span[level - 1];  // a part that begins here ends before
    for (long long i = before < 0 ? 0 : before / d.stride + 1; i < d.count; ++i) {
      if (at + i * d.stride >= to) return false;
      if (self(self, level - 1, at + i * d.stride)) return true;
    }
    return false;
  };
  return inside(inside, 3, 0);
}

// The parents lie outside the states, whose rows move while others read them.
bool parents_ok(const void* parents, size_t bytes, const hg_beam_state& s, size_t rows) {
  if (s.outer == 0 || s.pieces == 0 || s.piece_bytes == 0) return true;
  const long long from =
      (long long)(reinterpret_cast<uintptr_t>(parents) - reinterpret_cast<uintptr_t>(s.data));
  return !state_holds(s, rows, from, from + (long long)bytes);
}

// No state is listed twice: both would be moved at once.
bool states_differ(const hg_beam_state* states, int n) {
  const void* data[HG_MAX_STATES];
  int some = 0;
  for (int i = 0; i < n; ++i)
    if (states[i].outer && states[i].pieces && states[i].piece_bytes) data[some++] = states[i].data;
  std::sort(data, data + some, std::less<const void*>());
  return std::adjacent_find(data, data + some) == data + some;
}

}  // namespace

extern "C" {

int hg_beam_create(int max_items, int beams, int vocab, int picks, int dtype, hg_beam** out) {
  if (!out) return HG_ERR_ARG;
  *out = nullptr;
  if (max_items < 1 || beams < 1 || beams > HG_MAX_BEAMS || vocab < 1 || picks < 1 ||
      picks > HG_MAX_PICKS || (dtype != HG_BF16 && dtype != HG_FP16 && dtype != HG_FP32))
    return HG_ERR_ARG;
  // Rows, columns and picks are indexed with int.
  if ((long long)max_items * std::max(beams, picks) > INT_MAX / 2 || vocab > INT_MAX / 2 ||
      picks > (long long)beams * vocab)
    return HG_ERR_ARG;
  hg_beam* h = new (std::nothrow) hg_beam;
  if (!h) return HG_ERR_CUDA;
  h->max_items = max_items;
  h->beams = beams;
  h->vocab = vocab;
  h->picks = picks;
  h->dtype = dtype;
  if (cudaGetDevice(&h->device) != cudaSuccess ||
      cudaDeviceGetAttribute(&h->sms, cudaDevAttrMultiProcessorCount, h->device) != cudaSuccess ||
      hg::beam::select_prepare(*h) != cudaSuccess || hg::beam::reorder_prepare() != cudaSuccess) {
    cudaGetLastError();
    delete h;
    return HG_ERR_CUDA;
  }
  const size_t slots = (size_t)hg::beam::part_slots(*h), rows = (size_t)max_items * beams;
  h->bytes = slots * (hg::beam::kThreads * sizeof(*h->maxima) +
                      hg::beam::kWarps * sizeof(*h->stats) + sizeof(*h->beam_of)) +
             rows * picks * sizeof(*h->list);
  void* p = nullptr;
  if (cudaMalloc(&p, h->bytes) != cudaSuccess) {
    cudaGetLastError();  // leave no sticky allocation error behind
    delete h;
    return HG_ERR_CUDA;
  }
  h->base = static_cast<unsigned char*>(p);
  // The most aligned first.
  h->maxima = static_cast<float*>(p);
  h->stats = reinterpret_cast<float2*>(h->maxima + slots * hg::beam::kThreads);
  h->list = reinterpret_cast<unsigned long long*>(h->stats + slots * hg::beam::kWarps);
  h->beam_of = reinterpret_cast<int*>(h->list + rows * picks);
  *out = h;
  return HG_OK;
}

int hg_beam_destroy(hg_beam* h) {
  if (!h) return HG_OK;
  // A handle goes whatever device is current (a collector calls this too), but the
  // device to wait for is its own.
  int current = -1;
  bool ok = cudaGetDevice(&current) == cudaSuccess;
  const bool away = ok && current != h->device;
  if (away) ok = cudaSetDevice(h->device) == cudaSuccess;
  ok = ok && cudaDeviceSynchronize() == cudaSuccess;
  if (cudaFree(h->base) != cudaSuccess) ok = false;
  if (away && cudaSetDevice(current) != cudaSuccess) ok = false;
  delete h;
  return ok ? HG_OK : HG_ERR_CUDA;
}

size_t hg_beam_workspace_bytes(const hg_beam* h) { return h ? h->bytes : 0; }

int hg_beam_select(hg_beam* h, const void* logits, size_t ld_logits, const float* lse,
                   size_t lse_stride, const float* scores, const uint8_t* finished, int end,
                   int items, void* tokens, void* parents, int id_bytes, float* picked,
                   uint8_t* picked_finished, hg_stream_t stream) {
  if (!h || items < 0 || end < -1 || end >= h->vocab || (finished && end < 0)) return HG_ERR_ARG;
  if (items > 0) {
    const size_t e = hg::vocab::elem_bytes(h->dtype);
    const size_t rows = (size_t)items * h->beams;
    if (!logits || !aligned(logits, e) || ld_logits < (size_t)h->vocab ||
        ld_logits > (size_t)LLONG_MAX / 8 / rows || !aligned(lse, 4) ||
        (lse && (lse_stride < 1 || lse_stride > (size_t)LLONG_MAX / 8 / rows)) || !scores ||
        !aligned(scores, 4) || !ids_ok(tokens, id_bytes) || !ids_ok(parents, id_bytes) || !picked ||
        !aligned(picked, 4))
      return HG_ERR_ARG;
    const size_t picks = (size_t)items * h->picks;
    if (!hg::apart<7>({{tokens, picks * id_bytes}, {parents, picks * id_bytes}, {picked, picks * 4},
                       {picked_finished, picks}, {scores, rows * 4}, {finished, rows},
                       {logits, rows, ld_logits * e, h->vocab * e}}, 4))
      return HG_ERR_ARG;
  }
  if (items > h->max_items) return HG_ERR_ROWS;
  const int st = check_device(h);
  if (st != HG_OK || items == 0) return st;
  hg::beam::SelectCall c;
  c.items = items;
  c.logits = logits;
  c.ld = ld_logits;
  c.lse = lse;
  c.lse_stride = lse_stride;
  c.scores = scores;
  c.finished = finished;
  c.end = end;
  c.tokens = tokens;
  c.parents = parents;
  c.id_bytes = id_bytes;
  c.picked = picked;
  c.picked_finished = picked_finished;
  return as_status(hg::beam::select(*h, c, stream));
}

int hg_beam_reorder(hg_beam* h, const void* parents, int id_bytes, int items,
                    const hg_beam_state* states, int n_states, hg_stream_t stream) {
  if (!h || items < 0 || n_states < 0 || n_states > HG_MAX_STATES || (n_states > 0 && !states))
    return HG_ERR_ARG;
  if (items > 0 && !ids_ok(parents, id_bytes)) return HG_ERR_ARG;
  if (items > h->max_items) return HG_ERR_ROWS;
  if (items > 0) {
    const size_t rows = (size_t)items * h->beams;
    for (int i = 0; i < n_states; ++i)
      if (!state_ok(states[i], rows) || !parents_ok(parents, rows * id_bytes, states[i], rows))
        return HG_ERR_ARG;
    if (!states_differ(states, n_states)) return HG_ERR_ARG;
  }
  const int st = check_device(h);
  if (st != HG_OK || items == 0 || n_states == 0) return st;
  return as_status(hg::beam::reorder(*h, parents, id_bytes, items, states, n_states, stream));
}

}  // extern "C"
