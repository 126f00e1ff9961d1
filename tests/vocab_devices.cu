// The host side of the vocabulary operators on a fake CUDA runtime of two devices:
// prints, one event a line, what the library asks of it. No device is touched.
#include <cuda_runtime.h>

#include <cstdio>
#include <cstdlib>

static int g_current = 0;

static cudaError_t fakeGetDevice(int* d) {
  *d = g_current;
  return cudaSuccess;
}
static cudaError_t fakeSetDevice(int d) {
  if (d < 0 || d > 1) return cudaErrorInvalidDevice;
  g_current = d;
  return cudaSuccess;
}
static cudaError_t fakeSynchronize() {
  std::printf("wait for device %d\n", g_current);
  return cudaSuccess;
}
static cudaError_t fakeAttribute(int* v, cudaDeviceAttr, int) {
  *v = 152;
  return cudaSuccess;
}
static cudaError_t fakeMalloc(void** p, size_t) {
  *p = std::malloc(1 << 20);
  return cudaSuccess;
}
static cudaError_t fakeFree(void* p) {
  std::printf("free\n");
  std::free(p);
  return cudaSuccess;
}
static cudaError_t fakeMemset(void*, int, size_t) { return cudaSuccess; }

#define cudaGetDevice fakeGetDevice
#define cudaSetDevice fakeSetDevice
#define cudaDeviceSynchronize fakeSynchronize
#define cudaDeviceGetAttribute fakeAttribute
#define cudaMalloc fakeMalloc
#define cudaFree fakeFree
#define cudaMemset fakeMemset
#include "hg_vocab_lib.cu"

namespace hg {
namespace vocab {
static cudaError_t launched(const char* what) {
  std::printf("%s on device %d\n", what, g_current);
  return cudaSuccess;
}
cudaError_t embed_prepare() { return cudaSuccess; }
cudaError_t loss_prepare(const hg_vocab&) { return cudaSuccess; }
cudaError_t embed(const hg_vocab&, const Ids&, int, const void* const*, float, void*, size_t,
                  cudaStream_t) {
  return launched("embed");
}
cudaError_t embed_grad(const hg_vocab&, const Ids&, int, const void*, size_t, void* const*, float,
                       bool, cudaStream_t) {
  return launched("embed_grad");
}
cudaError_t loss(const hg_vocab&, const LossCall&, cudaStream_t) { return launched("loss"); }
cudaError_t loss_grad(const hg_vocab&, const LossCall&, cudaStream_t) {
  return launched("loss_grad");
}
long long embed_grad_chunks(const hg_vocab&) { return 1; }
long long loss_partials(const hg_vocab&) { return 1; }
long long loss_rows_pad(long long rows) { return rows; }
long long loss_accum_rows(const hg_vocab&) { return 1; }
}  // namespace vocab
}  // namespace hg

int main() {
  alignas(16) static unsigned char memory[4096];
  void* shard[1] = {memory};
  float* floats = reinterpret_cast<float*>(memory);
  hg_vocab* h = nullptr;
  fakeSetDevice(1);
  std::printf("create %d\n", hg_vocab_create(1, 4, 0, 8, 4, HG_BF16, 15, 0, &h));
  for (int device = 0; device < 2; ++device) {
    fakeSetDevice(device);
    std::printf("current %d\n", device);
    int st = hg_vocab_embed(h, memory, 8, 1, shard, 1.f, memory, 8, nullptr);
    std::printf("embed %d\n", st);
    st = hg_vocab_embed_grad(h, memory, 8, 1, memory, 8, shard, 1.f, 0, nullptr);
    std::printf("embed_grad %d\n", st);
    st = hg_vocab_loss(h, memory, 8, shard, memory, 8, 1, 1.f, floats, floats, nullptr);
    std::printf("loss %d\n", st);
    st = hg_vocab_loss_grad(h, memory, 8, shard, memory, 8, floats, floats, 1, 1.f, memory, 8,
                            shard, 0, nullptr);
    std::printf("loss_grad %d\n", st);
  }
  fakeSetDevice(0);
  std::printf("destroy %d\n", hg_vocab_destroy(h));
  std::printf("current %d\n", g_current);
  return 0;
}
