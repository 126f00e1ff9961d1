// Host side of the norm declared in include/hg.h: the handle, its workspace and
// the argument checks.

#include <climits>
#include <cmath>
#include <new>

#include "hg_norm.cuh"
#include "hg_overlap.cuh"

namespace {

using hg::Block;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// A matrix of N rows: present, aligned to its element, rows at least K apart.
bool matrix_ok(const hg_norm* h, const void* p, size_t ld, size_t elem, int N) {
  return N == 0 || (p && aligned(p, elem) && ld >= (size_t)h->K &&
                    ld <= (size_t)LLONG_MAX / 8 / (size_t)(N + 1));
}

Block rows_block(const hg_norm* h, const void* p, size_t ld, size_t elem, int N) {
  return Block(p, (size_t)N, ld * elem, (size_t)h->K * elem);
}

// An output that may be an input's own rows, row by row, and overlaps them in no other way.
bool in_place_ok(const Block& out, const Block& in) {
  return (out.p == in.p && (out.distance == in.distance || out.rows <= 1)) || !hg::overlap(out, in);
}

int as_status(cudaError_t e) { return e == cudaSuccess ? HG_OK : HG_ERR_CUDA; }

// The handle's workspace and the caller's tensors are of one device: with another
// one current, the kernels would start there, on pointers it cannot reach.
int check_device(const hg_norm* h) {
  int current = -1;
  if (cudaGetDevice(&current) != cudaSuccess) {
    cudaGetLastError();
    return HG_ERR_CUDA;
  }
  return current == h->device ? HG_OK : HG_ERR_ARG;
}

}  // namespace

extern "C" {

int hg_norm_create(int hidden, int max_rows, int dtype, hg_norm** out) {
  if (!out) return HG_ERR_ARG;
  *out = nullptr;
  if (hidden < 1 || hidden > INT_MAX / 8 || max_rows < 1 || max_rows > INT_MAX / 2 ||
      (dtype != HG_BF16 && dtype != HG_FP16 && dtype != HG_FP32))
    return HG_ERR_ARG;
  hg_norm* h = new (std::nothrow) hg_norm;
  if (!h) return HG_ERR_CUDA;
  h->K = hidden;
  h->max_rows = max_rows;
  h->dtype = dtype;
  if (cudaGetDevice(&h->device) != cudaSuccess ||
      cudaDeviceGetAttribute(&h->sms, cudaDevAttrMultiProcessorCount, h->device) != cudaSuccess ||
      hg::norm::prepare(*h) != cudaSuccess) {
    cudaGetLastError();
    delete h;
    return HG_ERR_CUDA;
  }
  h->bytes = (size_t)hg::norm::grad_parts(*h) * hidden * sizeof(float);
  void* p = nullptr;
  if (cudaMalloc(&p, h->bytes) != cudaSuccess) {
    cudaGetLastError();  // leave no sticky allocation error behind
    delete h;
    return HG_ERR_CUDA;
  }
  h->base = static_cast<unsigned char*>(p);
  h->partial = static_cast<float*>(p);
  *out = h;
  return HG_OK;
}

int hg_norm_destroy(hg_norm* h) {
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

size_t hg_norm_workspace_bytes(const hg_norm* h) { return h ? h->bytes : 0; }

int hg_norm_rows(hg_norm* h, const void* x, size_t ld_x, const void* residual,
                 size_t ld_residual, void* sum, size_t ld_sum, const void* gain, float eps, int N,
                 void* out, size_t ld_out, int out_type, float* scales, int scale_block,
                 float* rstd, hg_stream_t stream) {
  if (!h || N < 0 || !(eps >= 0.f) || std::isinf(eps) ||
      (out_type != h->dtype && out_type != HG_E4M3))
    return HG_ERR_ARG;
  const size_t e = hg::vocab::elem_bytes(h->dtype);
  const bool e4m3 = out_type == HG_E4M3;
  if (!matrix_ok(h, x, ld_x, e, N) || !matrix_ok(h, out, ld_out, e4m3 ? 1 : e, N) ||
      (residual && !matrix_ok(h, residual, ld_residual, e, N)) ||
      (sum && !matrix_ok(h, sum, ld_sum, e, N)) || !gain || !aligned(gain, e) ||
      (rstd && !aligned(rstd, 4)))
    return HG_ERR_ARG;
  if (e4m3 ? (N > 0 && !scales) || !aligned(scales, 4) || (scale_block != 0 && scale_block != 128)
           : scales || scale_block != 0)
    return HG_ERR_ARG;
  if (N > h->max_rows) return HG_ERR_ROWS;
  const size_t n = N, blocks = scale_block ? (h->K + 127) / 128 : 1;
  const Block of_x = rows_block(h, x, ld_x, e, N), of_res = rows_block(h, residual, ld_residual, e, N);
  const Block of_sum = rows_block(h, sum, ld_sum, e, N);
  const Block of_out = rows_block(h, out, ld_out, e4m3 ? 1 : e, N), of_rstd(rstd, n * 4);
  const Block of_scales(scales, n * blocks * 4), of_gain(gain, h->K * e);
  if (hg::overlap(of_sum, of_out) || !in_place_ok(of_sum, of_x) || !in_place_ok(of_sum, of_res) ||
      (e4m3 ? hg::overlap(of_out, of_x) || hg::overlap(of_out, of_res)
            : !in_place_ok(of_out, of_x) || !in_place_ok(of_out, of_res)) ||
      !hg::apart<6>({of_rstd, of_scales, of_x, of_res, of_sum, of_out}, 2) ||
      !hg::apart<4>({of_sum, of_out, of_rstd, of_gain}, 3))
    return HG_ERR_ARG;
  const int st = check_device(h);
  if (st != HG_OK || N == 0) return st;
  hg::norm::NormCall c;
  c.N = N;
  c.x = {x, ld_x};
  if (residual) c.residual = {residual, ld_residual};
  if (sum) c.sum = {sum, ld_sum};
  c.out = {out, ld_out};
  c.gain = gain;
  c.eps = eps;
  c.e4m3 = e4m3;
  c.scales = scales;
  c.scale_block = scale_block;
  c.rstd = rstd;
  return as_status(hg::norm::rows(*h, c, stream));
}

int hg_norm_rows_grad(hg_norm* h, const void* s, size_t ld_s, const void* gain, const float* rstd,
                      const void* grad_out, size_t ld_grad_out, const void* grad_sum,
                      size_t ld_grad_sum, int N, void* grad_x, size_t ld_grad_x, void* grad_gain,
                      int accumulate, hg_stream_t stream) {
  if (!h || N < 0 || (!grad_x && !grad_gain)) return HG_ERR_ARG;
  const size_t e = hg::vocab::elem_bytes(h->dtype);
  if (!matrix_ok(h, s, ld_s, e, N) || !matrix_ok(h, grad_out, ld_grad_out, e, N) ||
      (grad_sum && !matrix_ok(h, grad_sum, ld_grad_sum, e, N)) ||
      (grad_x && !matrix_ok(h, grad_x, ld_grad_x, e, N)) || !gain || !aligned(gain, e) ||
      (N > 0 && (!rstd || !aligned(rstd, 4))) || !aligned(grad_gain, e) || grad_gain == gain)
    return HG_ERR_ARG;
  if (N > h->max_rows) return HG_ERR_ROWS;
  const Block of_s = rows_block(h, s, ld_s, e, N), of_x = rows_block(h, grad_x, ld_grad_x, e, N);
  const Block of_up = rows_block(h, grad_out, ld_grad_out, e, N);
  const Block of_more = rows_block(h, grad_sum, ld_grad_sum, e, N);
  const Block of_rstd(rstd, (size_t)N * 4), of_gain(gain, h->K * e), of_sums(grad_gain, h->K * e);
  if (!in_place_ok(of_x, of_up) || !in_place_ok(of_x, of_more) ||
      !hg::apart<5>({of_x, of_sums, of_s, of_rstd, of_gain}, 2) ||
      !hg::apart<3>({of_sums, of_up, of_more}, 1))
    return HG_ERR_ARG;
  const int st = check_device(h);
  if (st != HG_OK || (N == 0 && (!grad_gain || accumulate))) return st;
  hg::norm::GradCall c;
  c.N = N;
  c.s = {s, ld_s};
  c.grad_out = {grad_out, ld_grad_out};
  if (grad_sum) c.grad_sum = {grad_sum, ld_grad_sum};
  c.gain = gain;
  c.rstd = rstd;
  if (grad_x) c.grad_x = {grad_x, ld_grad_x};
  c.grad_gain = grad_gain;
  c.accumulate = accumulate != 0;
  return as_status(hg::norm::rows_grad(*h, c, stream));
}

}  // extern "C"
