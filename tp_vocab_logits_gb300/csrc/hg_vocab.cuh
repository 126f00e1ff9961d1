// Internal declarations of the vocabulary operators (embedding, loss and their
// gradients): the handle, its workspace, and the launches of each translation
// unit.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "hg.h"

struct hg_vocab {
  int device = -1;
  int sms = 0;
  int tp = 0;
  int W = 0;      // matrix rows per shard
  int vocab = 0;  // real vocabulary
  int K = 0;
  int max_rows = 0;
  int dtype = HG_BF16;
  int ops = 0;
  int piece_cols = 0;  // columns of one shard in a piece of the gradient's logits
  unsigned char* base = nullptr;
  size_t bytes = 0;
  // Parts of the workspace.
  int* status = nullptr;     // device status words; [0] != 0: a bounded wait gave up
  int* count = nullptr;      // packed rows of the call
  float* unscale = nullptr;  // factor that takes the call's products back to scale
  int* row_of = nullptr;     // [max_rows] packed row -> row
  int* target = nullptr;     // [max_rows] packed row's target, -1: outside the vocabulary
  float* row_scale = nullptr;  // [max_rows] packed row's upstream gradient, scaled
  float* row_lse = nullptr;    // [max_rows] packed row's logsumexp in base 2
  float* hit = nullptr;        // [max_rows] packed row's target logit in base 2
  float2* partial = nullptr;   // [max_rows][vocab tiles] maximum and sum of a tile
  int pitch = 0;  // elements between rows of packed and accum: K up to whole 128-byte lines
  void* packed = nullptr;      // [rows_pad][pitch] unmasked rows of hidden
  void* prob = nullptr;        // [rows_pad][tp * piece_cols] piece of the logits' gradient
  float* accum = nullptr;      // [splits][rows_pad][pitch] grad_hidden before rounding
  uint32_t* key[2] = {};       // [max_rows] sorted tokens, and the sort's other buffer
  int* pos[2] = {};            // [max_rows] their positions
  float* runs = nullptr;       // [chunks][2][K] sums of runs that cross a chunk's ends
};

namespace hg {
namespace vocab {

inline size_t elem_bytes(int dtype) { return dtype == HG_FP32 ? 4 : 2; }
__host__ __device__ constexpr long long div_up(long long a, long long b) { return (a + b - 1) / b; }
__host__ __device__ constexpr long long round_up(long long a, long long b) {
  return div_up(a, b) * b;
}

// Token ids as the caller holds them.
struct Ids {
  const void* p;
  int bytes;  // 4 or 8
};

__device__ __forceinline__ long long load_id(const Ids& ids, size_t i) {
  return ids.bytes == 8 ? static_cast<const long long*>(ids.p)[i]
                        : (long long)static_cast<const int*>(ids.p)[i];
}

// Conversions of the matrix types to and from fp32 (round to nearest even).
template <typename T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ float up(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 down(float v) { return __float2bfloat16_rn(v); }
  static __device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
    return w;
  }
  static __device__ __forceinline__ float2 unpack2(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
};
template <>
struct Elem<__half> {
  static __device__ __forceinline__ float up(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half down(float v) { return __float2half_rn(v); }
  static __device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t w;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
    return w;
  }
  static __device__ __forceinline__ float2 unpack2(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
};
template <>
struct Elem<float> {
  static __device__ __forceinline__ float up(float v) { return v; }
  static __device__ __forceinline__ float down(float v) { return v; }
};

// E elements moved as one access.
template <typename T, int E>
struct alignas(sizeof(T) * E) Pack {
  T v[E];
};

// Programmatic dependent launch: a kernel launched so may start while its
// predecessor on the stream still runs, and waits for it (and all its writes)
// here, before its first access to global memory.
__device__ __forceinline__ void wait_for_predecessor() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Lets the next kernel on the stream start (and get as far as its own wait).
__device__ __forceinline__ void let_successor_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Launch as a dependent of the kernel before it, in clusters of `cluster` CTAs.
template <typename Args>
cudaError_t launch_dependent(void (*kernel)(Args), const Args& args, unsigned grid, unsigned block,
                             size_t smem, unsigned cluster, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args);
}

// Sorted rows that embed_grad sums as one sequence, and where there are few of them.
constexpr int kRunRows = 32;
constexpr int kFewRunRows = 8;

// Kernel attributes that the calls need on the current device (the shared memory
// limits), set once, when a handle is made.
cudaError_t embed_prepare();
cudaError_t loss_prepare(const hg_vocab& h);

cudaError_t embed(const hg_vocab& h, const Ids& tokens, int N, const void* const* table,
                  float scale, void* out, size_t ld_out, cudaStream_t stream);
cudaError_t embed_grad(const hg_vocab& h, const Ids& tokens, int N, const void* grad,
                       size_t ld_grad, void* const* table, float scale, bool accumulate,
                       cudaStream_t stream);

// Sequences of the largest call (workspace).
long long embed_grad_chunks(const hg_vocab& h);

// What one call of the loss or its gradient works on.
struct LossCall {
  const void* hidden;
  size_t ld;
  const void* const* weight;
  Ids targets;
  int N;
  float logit_scale;
  float* loss = nullptr;  // the loss's outputs
  float* lse_out = nullptr;
  const float* lse = nullptr;  // the gradient's inputs
  const float* grad_loss = nullptr;
  void* grad_hidden = nullptr;  // and outputs
  size_t ld_grad = 0;
  void* const* grad_weight = nullptr;
  bool accumulate = false;
};

cudaError_t loss(const hg_vocab& h, const LossCall& c, cudaStream_t stream);
cudaError_t loss_grad(const hg_vocab& h, const LossCall& c, cudaStream_t stream);

// Sizes of the loss's workspace: statistics of the tiles, rows of the packed
// matrices, slabs x rows of the gradient's accumulator.
long long loss_partials(const hg_vocab& h);
long long loss_rows_pad(long long rows);
long long loss_accum_rows(const hg_vocab& h);

}  // namespace vocab
}  // namespace hg
