// Host side of the vocabulary operators declared in include/hg.h: the handle,
// its workspace (one allocation, made at creation) and the argument checks.

#include <climits>
#include <new>

#include "hg_vocab.cuh"

namespace {

using hg::vocab::Ids;

constexpr size_t kDefaultPieceBytes = (size_t)512 << 20;
constexpr int kAllOps = HG_VOCAB_EMBED | HG_VOCAB_EMBED_GRAD | HG_VOCAB_LOSS | HG_VOCAB_LOSS_GRAD;
constexpr int kStatusBytes = 256;  // status words, row count and scale of a call

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Places the parts of the workspace one after another, 256-byte aligned; with a
// null base it only counts.
struct Layout {
  unsigned char* base;
  size_t used = 0;
  template <typename T>
  void take(T*& p, size_t n, size_t elem = sizeof(T)) {
    p = base ? reinterpret_cast<T*>(base + used) : nullptr;
    used += (n * elem + 255) / 256 * 256;
  }
  void take(void*& p, size_t bytes) {
    p = base ? base + used : nullptr;
    used += (bytes + 255) / 256 * 256;
  }
};

size_t lay_out(hg_vocab* h, unsigned char* base) {
  Layout l{base};
  const size_t n = (size_t)h->max_rows;
  const size_t e = hg::vocab::elem_bytes(h->dtype);
  l.take(h->status, kStatusBytes / sizeof(int));
  if (base) {
    h->count = h->status + 16;
    h->unscale = reinterpret_cast<float*>(h->status + 32);
  }
  if (h->ops & (HG_VOCAB_LOSS | HG_VOCAB_LOSS_GRAD)) {
    const size_t pad = (size_t)hg::vocab::loss_rows_pad(h->max_rows);
    l.take(h->row_of, n);
    l.take(h->target, n);
    l.take(h->packed, pad * h->pitch * e);
    if (h->ops & HG_VOCAB_LOSS) {
      l.take(h->hit, n);
      l.take(h->partial, (size_t)hg::vocab::loss_partials(*h));
    }
    if (h->ops & HG_VOCAB_LOSS_GRAD) {
      l.take(h->row_scale, n);
      l.take(h->row_lse, n);
      l.take(h->prob, pad * h->tp * (size_t)h->piece_cols * e);
      l.take(h->accum, (size_t)hg::vocab::loss_accum_rows(*h) * h->pitch);
    }
  }
  if (h->ops & HG_VOCAB_EMBED_GRAD) {
    for (int i = 0; i < 2; ++i) {
      l.take(h->key[i], n);
      l.take(h->pos[i], n);
    }
    l.take(h->runs, (size_t)hg::vocab::embed_grad_chunks(*h) * 2 * h->K);
  }
  return l.used;
}

bool shards_ok(const hg_vocab* h, const void* const* p, size_t align) {
  if (!p) return false;
  for (int r = 0; r < h->tp; ++r)
    if (!p[r] || !aligned(p[r], align)) return false;
  return true;
}

bool ids_ok(const void* p, int id_bytes, int N) {
  return (id_bytes == 4 || id_bytes == 8) && (N == 0 || (p && aligned(p, (size_t)id_bytes)));
}

// The token-side matrix of N rows: present, aligned, rows at least K apart.
bool matrix_ok(const hg_vocab* h, const void* p, size_t ld, size_t align, size_t ld_step, int N) {
  return N == 0 || (p && aligned(p, align) && ld >= (size_t)h->K && ld % ld_step == 0 &&
                    ld <= (size_t)LLONG_MAX / 8 / (size_t)(N + 1));
}

bool floats_ok(const float* p, int N) { return N == 0 || (p && aligned(p, 4)); }

int as_status(cudaError_t e) { return e == cudaSuccess ? HG_OK : HG_ERR_CUDA; }

// The handle's workspace and the caller's tensors are of one device: with another
// one current, the kernels would start there, on pointers it cannot reach.
int check_device(const hg_vocab* h) {
  int current = -1;
  if (cudaGetDevice(&current) != cudaSuccess) {
    cudaGetLastError();
    return HG_ERR_CUDA;
  }
  return current == h->device ? HG_OK : HG_ERR_ARG;
}

// Checks that hg_vocab_loss and its gradient share.
int check_loss(const hg_vocab* h, int op, const void* hidden, size_t ld,
               const void* const* weight, const void* targets, int id_bytes, int N) {
  if (!h || N < 0 || !(h->ops & op) || !shards_ok(h, weight, 16) || !ids_ok(targets, id_bytes, N) ||
      !matrix_ok(h, hidden, ld, 16, 8, N))
    return HG_ERR_ARG;
  return N > h->max_rows ? HG_ERR_ROWS : check_device(h);
}

}  // namespace

extern "C" {

int hg_vocab_create(int tp, int shard_cols, int vocab, int hidden, int max_rows, int dtype,
                    int ops, size_t piece_bytes, hg_vocab** out) {
  if (!out) return HG_ERR_ARG;
  *out = nullptr;
  if (tp < 1 || tp > HG_MAX_TP || shard_cols < 1 || hidden < 1 || max_rows < 1 || vocab < 0 ||
      (dtype != HG_BF16 && dtype != HG_FP16 && dtype != HG_FP32) || (ops & ~kAllOps) || ops == 0)
    return HG_ERR_ARG;
  // Sizes that the kernels index with int: columns, rows and tiles, each with
  // room for the last partial tile.
  const long long total = (long long)tp * shard_cols;
  if (total > INT_MAX / 2 || max_rows > INT_MAX / 2 || hidden > INT_MAX / 8 || vocab > total)
    return HG_ERR_ARG;
  const bool loss = (ops & (HG_VOCAB_LOSS | HG_VOCAB_LOSS_GRAD)) != 0;
  if (loss && (dtype == HG_FP32 || hidden % 8 != 0)) return HG_ERR_ARG;

  hg_vocab* h = new (std::nothrow) hg_vocab;
  if (!h) return HG_ERR_CUDA;
  h->tp = tp;
  h->W = shard_cols;
  h->vocab = vocab ? vocab : (int)total;
  h->K = hidden;
  h->pitch = (int)hg::vocab::round_up(hidden, 64);
  h->max_rows = max_rows;
  h->dtype = dtype;
  h->ops = ops;
  if (cudaGetDevice(&h->device) != cudaSuccess ||
      cudaDeviceGetAttribute(&h->sms, cudaDevAttrMultiProcessorCount, h->device) != cudaSuccess ||
      ((ops & HG_VOCAB_EMBED_GRAD) && hg::vocab::embed_prepare() != cudaSuccess) ||
      (loss && hg::vocab::loss_prepare(*h) != cudaSuccess)) {
    delete h;
    return HG_ERR_CUDA;
  }
  if (ops & HG_VOCAB_LOSS_GRAD) {
    const size_t budget = piece_bytes ? piece_bytes : kDefaultPieceBytes;
    const size_t per_col = (size_t)hg::vocab::loss_rows_pad(max_rows) * tp * 2;
    long long cols = (long long)(budget / per_col) / 256 * 256;
    const long long most = hg::vocab::round_up(shard_cols, 256);
    if (cols > most) cols = most;
    if (cols < 256) cols = 256;
    h->piece_cols = (int)cols;
  }
  h->bytes = lay_out(h, nullptr);
  void* p = nullptr;
  if (cudaMalloc(&p, h->bytes) != cudaSuccess) {
    cudaGetLastError();  // leave no sticky allocation error behind
    delete h;
    return HG_ERR_CUDA;
  }
  h->base = static_cast<unsigned char*>(p);
  if (cudaMemset(p, 0, kStatusBytes) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) {
    cudaFree(p);
    delete h;
    return HG_ERR_CUDA;
  }
  lay_out(h, h->base);
  *out = h;
  return HG_OK;
}

int hg_vocab_destroy(hg_vocab* h) {
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

size_t hg_vocab_workspace_bytes(const hg_vocab* h) { return h ? h->bytes : 0; }

int hg_vocab_sync(hg_vocab* h, hg_stream_t stream) {
  if (!h) return HG_ERR_ARG;
  int st = check_device(h);
  if (st != HG_OK) return st;
  if (cudaMemcpyAsync(&st, h->status, sizeof st, cudaMemcpyDeviceToHost, stream) != cudaSuccess ||
      cudaStreamSynchronize(stream) != cudaSuccess)
    return HG_ERR_CUDA;
  if (st == 0) return HG_OK;
  if (cudaMemsetAsync(h->status, 0, sizeof st, stream) != cudaSuccess) return HG_ERR_CUDA;
  return HG_ERR_TIMEOUT;
}

int hg_vocab_embed(hg_vocab* h, const void* tokens, int id_bytes, int N,
                   const void* const* table_ptrs, float scale, void* out, size_t ld_out,
                   hg_stream_t stream) {
  if (!h || N < 0 || !ids_ok(tokens, id_bytes, N)) return HG_ERR_ARG;
  const size_t e = hg::vocab::elem_bytes(h->dtype);
  if (!shards_ok(h, table_ptrs, e) || !matrix_ok(h, out, ld_out, e, 1, N)) return HG_ERR_ARG;
  if (N > h->max_rows) return HG_ERR_ROWS;
  const int st = check_device(h);
  if (st != HG_OK || N == 0) return st;
  return as_status(hg::vocab::embed(*h, Ids{tokens, id_bytes}, N, table_ptrs, scale, out, ld_out,
                                    stream));
}

int hg_vocab_embed_grad(hg_vocab* h, const void* tokens, int id_bytes, int N,
                        const void* grad_out, size_t ld_grad_out, void* const* grad_table_ptrs,
                        float scale, int accumulate, hg_stream_t stream) {
  if (!h || N < 0 || !(h->ops & HG_VOCAB_EMBED_GRAD) || !ids_ok(tokens, id_bytes, N))
    return HG_ERR_ARG;
  const size_t e = hg::vocab::elem_bytes(h->dtype);
  if (!shards_ok(h, grad_table_ptrs, e) || !matrix_ok(h, grad_out, ld_grad_out, e, 1, N))
    return HG_ERR_ARG;
  if (N > h->max_rows) return HG_ERR_ROWS;
  const int st = check_device(h);
  if (st != HG_OK || (N == 0 && accumulate)) return st;
  return as_status(hg::vocab::embed_grad(*h, Ids{tokens, id_bytes}, N, grad_out, ld_grad_out,
                                         grad_table_ptrs, scale, accumulate != 0, stream));
}

int hg_vocab_loss(hg_vocab* h, const void* hidden, size_t ld_hidden,
                  const void* const* weight_ptrs, const void* targets, int id_bytes, int N,
                  float logit_scale, float* loss, float* lse, hg_stream_t stream) {
  const int st = check_loss(h, HG_VOCAB_LOSS, hidden, ld_hidden, weight_ptrs, targets, id_bytes, N);
  if (st != HG_OK) return st;
  if (!floats_ok(loss, N) || !floats_ok(lse, N)) return HG_ERR_ARG;
  if (N == 0) return HG_OK;
  hg::vocab::LossCall c;
  c.hidden = hidden;
  c.ld = ld_hidden;
  c.weight = weight_ptrs;
  c.targets = Ids{targets, id_bytes};
  c.N = N;
  c.logit_scale = logit_scale;
  c.loss = loss;
  c.lse_out = lse;
  return as_status(hg::vocab::loss(*h, c, stream));
}

int hg_vocab_loss_grad(hg_vocab* h, const void* hidden, size_t ld_hidden,
                       const void* const* weight_ptrs, const void* targets, int id_bytes,
                       const float* lse, const float* grad_loss, int N, float logit_scale,
                       void* grad_hidden, size_t ld_grad_hidden, void* const* grad_weight_ptrs,
                       int accumulate, hg_stream_t stream) {
  const int st =
      check_loss(h, HG_VOCAB_LOSS_GRAD, hidden, ld_hidden, weight_ptrs, targets, id_bytes, N);
  if (st != HG_OK) return st;
  if (!floats_ok(lse, N) || !floats_ok(grad_loss, N) || (!grad_hidden && !grad_weight_ptrs) ||
      (grad_hidden && !matrix_ok(h, grad_hidden, ld_grad_hidden, 16, 8, N)) ||
      (grad_weight_ptrs && !shards_ok(h, grad_weight_ptrs, 16)))
    return HG_ERR_ARG;
  if (N == 0 && (!grad_weight_ptrs || accumulate)) return HG_OK;
  hg::vocab::LossCall c;
  c.hidden = hidden;
  c.ld = ld_hidden;
  c.weight = weight_ptrs;
  c.targets = Ids{targets, id_bytes};
  c.N = N;
  c.logit_scale = logit_scale;
  c.lse = lse;
  c.grad_loss = grad_loss;
  c.grad_hidden = grad_hidden;
  c.ld_grad = ld_grad_hidden;
  c.grad_weight = grad_weight_ptrs;
  c.accumulate = accumulate != 0;
  return as_status(hg::vocab::loss_grad(*h, c, stream));
}

}  // extern "C"
