// The host side of the norm (or, with BEAM defined, the beam search) on a fake CUDA
// runtime of two devices: prints, one line each, what the entry points answer and
// what the library asks of the runtime. No device is touched.
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

static cudaError_t launched(const char* what) {
  std::printf("%s on device %d\n", what, g_current);
  return cudaSuccess;
}

static void show(const char* what, int st) { std::printf("%s %d\n", what, st); }

alignas(256) static unsigned char a[4096], b[4096], c[4096], d[4096];

#ifdef BEAM
#include "hg_beam_lib.cu"

namespace hg {
namespace beam {
cudaError_t select(const hg_beam&, const SelectCall&, cudaStream_t) { return launched("select"); }
cudaError_t reorder(const hg_beam&, const void*, int, int, const hg_beam_state*, int,
                    cudaStream_t) {
  return launched("reorder");
}

cudaError_t select_prepare(const hg_beam&) { return cudaSuccess; }
cudaError_t reorder_prepare() { return cudaSuccess; }
long long part_slots(const hg_beam&) { return 1; }
}  // namespace beam
}  // namespace hg

int main() {
  hg_beam* h = nullptr;
  fakeSetDevice(1);
  show("create", hg_beam_create(2, 3, 50, 4, HG_BF16, &h));
  float* f = reinterpret_cast<float*>(b);
  auto select = [&](const char* what, const void* logits, size_t ld, const float* lse,
                    size_t stride, const uint8_t* finished, int end, int items, void* tokens,
                    int id_bytes) {
    show(what, hg_beam_select(h, logits, ld, lse, stride, f, finished, end, items, tokens, d,
                              id_bytes, f + 16, nullptr, nullptr));
  };
  auto reorder = [&](const char* what, hg_beam_state s) {
    show(what, hg_beam_reorder(h, d, 8, 2, &s, 1, nullptr));
  };
  for (int device = 0; device < 2; ++device) {
    fakeSetDevice(device);
    std::printf("current %d\n", device);
    select("select", a, 50, nullptr, 0, nullptr, -1, 2, c, 8);
    reorder("reorder", {a, 1, 0, 8, 1, 0, 8});
  }
  std::printf("refused\n");
  select("no logits", nullptr, 50, nullptr, 0, nullptr, -1, 2, c, 8);
  select("odd address", a + 1, 50, nullptr, 0, nullptr, -1, 2, c, 8);
  select("short rows", a, 49, nullptr, 0, nullptr, -1, 2, c, 8);
  select("rows beyond 64 bits", a, (size_t)1 << 60, nullptr, 0, nullptr, -1, 2, c, 8);
  select("no stride of lse", a, 50, f, 0, nullptr, -1, 2, c, 8);
  select("finished without end", a, 50, nullptr, 0, a, -1, 2, c, 8);
  select("end beyond the vocabulary", a, 50, nullptr, 0, nullptr, 50, 2, c, 8);
  select("negative end", a, 50, nullptr, 0, nullptr, -2, 2, c, 8);
  select("negative items", a, 50, nullptr, 0, nullptr, -1, -1, c, 8);
  select("no tokens", a, 50, nullptr, 0, nullptr, -1, 2, nullptr, 8);
  select("ids of 2 bytes", a, 50, nullptr, 0, nullptr, -1, 2, c, 2);
  select("ids not aligned", a, 50, nullptr, 0, nullptr, -1, 2, c + 4, 8);
  auto overlap = [&](const char* what, void* tokens, void* parents, float* picked, uint8_t* done) {
    show(what, hg_beam_select(h, a, 50, nullptr, 0, f, b + 40, 3, 2, tokens, parents, 8, picked,
                              done, nullptr));
  };
  overlap("totals over scores", c, d, f, nullptr);
  overlap("totals over the last score", c, d, f + 5, nullptr);
  overlap("flags over flags", c, d, f + 24, b + 45);
  overlap("tokens over parents", c + 8, c, f + 12, nullptr);
  overlap("parents over totals", c, d, reinterpret_cast<float*>(d + 60), nullptr);
  reorder("no data", {nullptr, 1, 0, 8, 1, 0, 8});
  reorder("rows overlap", {a, 1, 0, 7, 1, 0, 8});
  reorder("pieces overlap", {a, 1, 0, 64, 4, 4, 8});
  reorder("rows over pieces", {a, 1, 0, 31, 4, 8, 8});
  reorder("outer over rows", {a, 2, 47, 8, 1, 0, 8});
  reorder("bytes beyond 64 bits", {a, 1, 0, (size_t)1 << 61, 1, 0, (size_t)1 << 61});
  reorder("steps beyond 64 bits", {a, (size_t)1 << 40, (size_t)1 << 40, 8, 1, 0, 8});
  const hg_beam_state twice[3] = {{a, 1, 0, 8, 1, 0, 8}, {b, 1, 0, 8, 1, 0, 8}, {a, 1, 0, 8, 1, 0, 8}};
  show("a state twice", hg_beam_reorder(h, d, 8, 2, twice, 3, nullptr));
  show("states missing", hg_beam_reorder(h, d, 8, 2, nullptr, 1, nullptr));
  show("too many states", hg_beam_reorder(h, d, 8, 2, nullptr, HG_MAX_STATES + 1, nullptr));
  show("no parents", hg_beam_reorder(h, nullptr, 8, 2, nullptr, 0, nullptr));
  std::printf("too many items\n");
  select("select", a, 50, nullptr, 0, nullptr, -1, 3, c, 8);
  show("reorder", hg_beam_reorder(h, d, 8, 3, nullptr, 0, nullptr));
  std::printf("served\n");
  select("no items", nullptr, 0, nullptr, 0, nullptr, -1, 0, nullptr, 8);
  select("all", a, 50, f, 4, a, 49, 2, c + 4, 4);
  reorder("rows outside the layers", {a, 2, 8, 16, 1, 0, 8});
  reorder("nothing in it", {nullptr, 1, 0, 0, 0, 0, 8});
  show("no states", hg_beam_reorder(h, d, 8, 2, nullptr, 0, nullptr));
  // The workspace's arrays, where odd counts come before them.
  std::printf("workspaces\n");
  for (int items = 1; items < 4; ++items)
    for (int picks = 1; picks < 4; ++picks) {
      hg_beam* w = nullptr;
      hg_beam_create(items, 3, 50, picks, HG_BF16, &w);
      auto off = [&](const void* p) { return (uintptr_t)p - (uintptr_t)w->base; };
      const bool ok = off(w->maxima) % 16 == 0 && off(w->stats) % 8 == 0 && off(w->list) % 8 == 0 &&
                      off(w->beam_of) % 4 == 0 &&
                      off(w->beam_of + hg::beam::part_slots(*w)) == w->bytes;
      show("aligned", ok);
      w->base = nullptr;  // not freed: the lines below are compared
      delete w;
    }
  std::printf("end\n");
  fakeSetDevice(0);
  show("destroy", hg_beam_destroy(h));
  std::printf("current %d\n", g_current);
  return 0;
}
#else
#include "hg_norm_lib.cu"

namespace hg {
namespace norm {
cudaError_t rows(const hg_norm&, const NormCall&, cudaStream_t) { return launched("rows"); }
cudaError_t rows_grad(const hg_norm&, const GradCall&, cudaStream_t) { return launched("grad"); }
cudaError_t prepare(const hg_norm&) { return cudaSuccess; }
int grad_parts(const hg_norm&) { return 1; }
}  // namespace norm
}  // namespace hg

int main() {
  hg_norm* h = nullptr;
  fakeSetDevice(1);
  show("create", hg_norm_create(16, 2, HG_BF16, &h));
  float* f = reinterpret_cast<float*>(d);
  struct Rows {
    const void* x = a;
    size_t ld_x = 16;
    const void* res = nullptr;
    size_t ld_res = 0;
    void* sum = nullptr;
    size_t ld_sum = 0;
    const void* gain = d;
    float eps = 1e-6f;
    int N = 2;
    void* out = b;
    size_t ld_out = 16;
    int type = HG_BF16;
    float* scales = nullptr;
    int block = 0;
    float* rstd = nullptr;
  };
  auto rows = [&](const char* what, Rows r) {
    show(what, hg_norm_rows(h, r.x, r.ld_x, r.res, r.ld_res, r.sum, r.ld_sum, r.gain, r.eps, r.N,
                            r.out, r.ld_out, r.type, r.scales, r.block, r.rstd, nullptr));
  };
  struct Grad {
    const void* s = a;
    size_t ld_s = 16;
    const void* gain = d;
    const float* rstd = reinterpret_cast<const float*>(d);
    const void* up = b;
    size_t ld_up = 16;
    const void* more = nullptr;
    size_t ld_more = 0;
    int N = 2;
    void* x = c;
    size_t ld_x = 16;
    void* gain_out = nullptr;
  };
  auto grad = [&](const char* what, Grad g) {
    show(what, hg_norm_rows_grad(h, g.s, g.ld_s, g.gain, g.rstd, g.up, g.ld_up, g.more, g.ld_more,
                                 g.N, g.x, g.ld_x, g.gain_out, 0, nullptr));
  };
  for (int device = 0; device < 2; ++device) {
    fakeSetDevice(device);
    std::printf("current %d\n", device);
    rows("rows", {});
    grad("grad", {});
  }
  std::printf("refused\n");
  rows("no x", {.x = nullptr});
  rows("odd address", {.x = a + 1});
  rows("short rows", {.ld_x = 15});
  rows("rows beyond 64 bits", {.ld_x = (size_t)1 << 62});
  rows("short residual", {.res = c, .ld_res = 15});
  rows("short sum", {.sum = c, .ld_sum = 15});
  rows("no gain", {.gain = nullptr});
  rows("negative eps", {.eps = -1.f});
  rows("NaN eps", {.eps = NAN});
  rows("infinite eps", {.eps = INFINITY});
  rows("negative rows", {.N = -1});
  rows("no out", {.out = nullptr});
  rows("another type", {.type = HG_FP32});
  rows("scales of 16 bits", {.scales = f});
  rows("a block of 16 bits", {.block = 128});
  rows("no scales", {.type = HG_E4M3});
  rows("another block", {.type = HG_E4M3, .scales = f, .block = 64});
  rows("8 bits in place", {.out = a, .type = HG_E4M3, .scales = f});
  rows("out and sum", {.res = c, .ld_res = 16, .sum = b, .ld_sum = 16});
  rows("in place, other distance", {.out = a, .ld_out = 24});
  rows("sum in place, other distance", {.res = c, .ld_res = 16, .sum = c, .ld_sum = 24});
  rows("rstd not aligned", {.rstd = reinterpret_cast<float*>(d + 2)});
  grad("no gradient", {.x = nullptr});
  grad("no s", {.s = nullptr});
  grad("no rstd", {.rstd = nullptr});
  grad("no grad_out", {.up = nullptr});
  grad("short grad_sum", {.more = d, .ld_more = 15});
  grad("over s", {.x = a});
  grad("in place, other distance", {.x = b, .ld_x = 24});
  grad("odd grad_gain", {.gain_out = d + 1});
  grad("over the gain", {.gain_out = d});
  std::printf("too many rows\n");
  rows("rows", {.N = 3});
  grad("grad", {.N = 3});
  std::printf("served\n");
  rows("no rows", {.x = nullptr, .N = 0, .out = nullptr});
  grad("no rows", {.s = nullptr, .rstd = nullptr, .up = nullptr, .N = 0, .x = nullptr,
                   .gain_out = d + 512});
  rows("in place", {.res = c, .ld_res = 16, .sum = c, .ld_sum = 16, .out = a});
  rows("one row, other distance", {.N = 1, .out = a, .ld_out = 24});
  rows("8 bits", {.type = HG_E4M3, .scales = f, .block = 128});
  grad("in place", {.more = c, .ld_more = 16, .gain_out = d + 512});
  std::printf("end\n");
  fakeSetDevice(0);
  show("destroy", hg_norm_destroy(h));
  std::printf("current %d\n", g_current);
  return 0;
}
#endif
