// Internal declarations of the norm: the handle, what a call works on, and the
// launches.
#pragma once

#include "hg_vocab.cuh"

struct hg_norm {
  int device = -1;
  int sms = 0;
  int K = 0;
  int max_rows = 0;
  int dtype = HG_BF16;
  unsigned char* base = nullptr;
  size_t bytes = 0;
  float* partial = nullptr;  // [grad_parts][K] sums of grad_gain over some rows
};

namespace hg {
namespace norm {

// The rows of one matrix.
struct Rows {
  const void* p = nullptr;
  size_t ld = 0;
};
struct RowsOut {
  void* p = nullptr;
  size_t ld = 0;
};

struct NormCall {
  int N = 0;
  Rows x, residual;
  RowsOut sum, out;
  const void* gain = nullptr;
  float eps = 0.f;
  bool e4m3 = false;
  float* scales = nullptr;
  int scale_block = 0;
  float* rstd = nullptr;
};

struct GradCall {
  int N = 0;
  Rows s, grad_out, grad_sum;
  const void* gain = nullptr;
  const float* rstd = nullptr;
  RowsOut grad_x;
  void* grad_gain = nullptr;
  bool accumulate = false;
};

cudaError_t rows(const hg_norm& h, const NormCall& c, cudaStream_t stream);
cudaError_t rows_grad(const hg_norm& h, const GradCall& c, cudaStream_t stream);

// Kernel attributes that the calls need on the current device, set when a handle is made.
cudaError_t prepare(const hg_norm& h);

// The most partial sums of grad_gain that a call writes.
int grad_parts(const hg_norm& h);

// Widest access that all of these allow: 16 bytes, 4, or an element.
struct Access {
  size_t bits = 0;
  void rows(const void* p, size_t ld, int N, size_t elem) {
    if (!p) return;
    bits |= reinterpret_cast<uintptr_t>(p);
    if (N > 1) bits |= ld * elem;
  }
  int bytes(size_t elem) const { return bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : (int)elem; }
};

}  // namespace norm
}  // namespace hg
