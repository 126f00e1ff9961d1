// Which overlaps of a call's arrays are refused, on the fake CUDA runtime of step_calls.cu, and
// the tests for them against sets of bytes. Prints what is wrong, and "done".
#define main calls_main
#include "step_calls.cu"
#undef main

#include <cstring>
#include <random>
#include <vector>

#ifndef BEAM
static void blocks() {
  std::mt19937 gen(5);
  auto below = [&](int n) { return (int)(gen() % n); };
  alignas(64) static unsigned char memory[4096];
  int seen[2] = {};
  for (int i = 0; i < 200000; ++i) {
    hg::Block block[2];
    std::vector<char> set[2];
    for (int k = 0; k < 2; ++k) {
      const size_t rows = below(6), width = below(9);
      const size_t distance = k && below(2) ? block[0].distance : width + below(20);
      if (distance < width) continue;
      unsigned char* p = memory + below(k && below(2) ? 40 : 150);
      block[k] = hg::Block(p, rows, distance, width);
      set[k].assign(512, 0);
      for (size_t r = 0; r < rows; ++r)
        for (size_t w = 0; w < width; ++w) set[k][(size_t)(p - memory) + r * distance + w] = 1;
    }
    bool want = false;
    if (!set[0].empty() && !set[1].empty())
      for (int j = 0; j < 512; ++j) want |= set[0][j] && set[1][j];
    ++seen[want];
    if (hg::overlap(block[0], block[1]) != want || hg::overlap(block[1], block[0]) != want)
      std::printf("blocks %d\n", i);
  }
  if (seen[0] < 20000 || seen[1] < 20000) std::printf("too few kinds of blocks\n");
}

int main() {
  blocks();
  hg_norm* h = nullptr;
  fakeSetDevice(1);
  hg_norm_create(16, 4, HG_BF16, &h);
  // Rows of 16 elements, 32 bytes, 4 of them in 128 bytes; the gain and small arrays apart.
  alignas(256) static unsigned char more[4096];
  float* const f = reinterpret_cast<float*>(more);
  void* const gain = more + 1024;
  auto expect = [](const char* what, int want, int got) {
    if (got != want) std::printf("%s: %d, not %d\n", what, got, want);
  };
  auto rows = [&](const char* what, int want, const void* x, const void* res, size_t ld, void* sum,
                  void* out, size_t ld_out, float* rstd, float* scales = nullptr) {
    expect(what, want,
           hg_norm_rows(h, x, 16, res, ld, sum, ld, gain, 1e-6f, 4, out, ld_out,
                        scales ? (int)HG_E4M3 : (int)HG_BF16, scales, 0, rstd, nullptr));
  };
  const int no = HG_ERR_ARG, yes = HG_OK;
  rows("apart", yes, a, b, 16, c, d, 16, f);
  rows("out one row into x", no, a, nullptr, 16, nullptr, a + 32, 16, nullptr);
  rows("x one row into out", no, a + 32, nullptr, 16, nullptr, a, 16, nullptr);
  rows("out on x's last element", no, a, nullptr, 16, nullptr, a + 126, 16, nullptr);
  rows("out behind x", yes, a, nullptr, 16, nullptr, a + 128, 16, nullptr);
  rows("out is x", yes, a, nullptr, 16, nullptr, a, 16, nullptr);
  rows("out is x, other distance", no, a, nullptr, 16, nullptr, a, 24, nullptr);
  rows("sum is the residual, out is x", yes, a, b, 16, b, a, 16, f);
  rows("sum one row into the residual", no, a, b, 16, b + 32, c, 16, nullptr);
  rows("sum over out", no, a, b, 16, c, c + 64, 16, nullptr);
  rows("sum beside out", yes, a, b, 32, c, c + 32, 32, nullptr);
  rows("sum half over out", no, a, b, 32, c, c + 30, 32, nullptr);
  rows("out between the residual's rows", yes, a, b, 48, nullptr, b + 32, 96, nullptr);
  rows("out over a later row of the residual", no, a, b, 40, nullptr, b + 32, 24, nullptr);
  rows("rstd over x", no, a, nullptr, 16, nullptr, b, 16, reinterpret_cast<float*>(a + 124));
  rows("rstd over out", no, a, nullptr, 16, nullptr, b, 16, reinterpret_cast<float*>(b));
  rows("rstd over the gain", no, a, nullptr, 16, nullptr, b, 16, reinterpret_cast<float*>(gain));
  rows("out over the gain", no, a, nullptr, 16, nullptr, more + 1000, 16, nullptr);
  rows("8 bits", yes, a, nullptr, 16, nullptr, b, 16, f, f + 4);
  rows("8 bits over x", no, a, nullptr, 16, nullptr, a + 100, 16, f, f + 4);
  rows("8 bits behind x", yes, a, nullptr, 16, nullptr, a + 128, 16, f, f + 4);
  rows("scales over rstd", no, a, nullptr, 16, nullptr, b, 16, f, f + 3);
  rows("scales over out", no, a, nullptr, 16, nullptr, b, 16, f, reinterpret_cast<float*>(b + 60));
  rows("scales behind out", yes, a, nullptr, 16, nullptr, b, 16, f,
       reinterpret_cast<float*>(b + 64));
  auto grad = [&](const char* what, int want, void* x, size_t ld_x, void* sums, const void* up,
                  const void* rest) {
    expect(what, want,
           hg_norm_rows_grad(h, a, 16, gain, f, up, 16, rest, 16, 4, x, ld_x, sums, 0, nullptr));
  };
  grad("apart", yes, c, 16, d, b, nullptr);
  grad("grad_x is grad_out", yes, b, 16, d, b, nullptr);
  grad("grad_x is grad_sum", yes, c, 16, d, b, c);
  grad("grad_x one row into grad_out", no, b + 32, 16, d, b, nullptr);
  grad("grad_x one row into grad_sum", no, c + 32, 16, d, b, c);
  grad("grad_x over s", no, a + 96, 16, d, b, nullptr);
  grad("grad_x over rstd", no, more, 16, d, b, nullptr);
  grad("grad_gain over grad_x", no, c, 16, c + 100, b, nullptr);
  grad("grad_gain over grad_out", no, c, 16, b + 100, b, nullptr);
  grad("grad_gain over grad_sum", no, c, 16, d + 2, b, d);
  grad("grad_gain over s", no, nullptr, 0, a, b, nullptr);
  grad("grad_gain over rstd", no, c, 16, f + 2, b, nullptr);
  grad("grad_gain over half of the gain", no, c, 16, more + 1040, b, nullptr);
  hg_norm_destroy(h);
  std::printf("done\n");
  return 0;
}
#else
static void states() {
  std::mt19937 gen(6);
  auto below = [&](int n) { return (size_t)(gen() % n); };
  constexpr size_t kMost = 4096;
  int seen[2] = {};
  for (int i = 0; i < 100000; ++i) {
    hg_beam_state s = {a, 1 + below(3), 0, 0, 1 + below(3), 0, 1 + below(8)};
    const size_t rows = 1 + below(3);
    // Strides in a random order of the dimensions.
    size_t* stride[3] = {&s.outer_stride, &s.row_stride, &s.piece_stride};
    const size_t count[3] = {s.outer, rows, s.pieces};
    int order[3] = {0, 1, 2};
    std::shuffle(order, order + 3, gen);
    size_t span = s.piece_bytes;
    for (int k : order) {
      *stride[k] = count[k] == 1 ? below(50) : span + below(12);
      span += count[k] == 1 ? 0 : *stride[k] * (count[k] - 1);
    }
    if (span > kMost) continue;
    if (!state_ok(s, rows)) std::printf("state %d\n", i);
    std::vector<char> set(kMost + 64);
    for (size_t o = 0; o < s.outer; ++o)
      for (size_t r = 0; r < rows; ++r)
        for (size_t p = 0; p < s.pieces; ++p)
          for (size_t w = 0; w < s.piece_bytes; ++w)
            set[o * s.outer_stride + r * s.row_stride + p * s.piece_stride + w] = 1;
    const long long from = (long long)below((int)span + 20) - 10, to = from + 1 + (long long)below(12);
    bool want = false;
    for (long long x = from < 0 ? 0 : from; x < to; ++x) want |= set[x];
    ++seen[want];
    if (state_holds(s, rows, from, to) != want) std::printf("parents %d\n", i);
  }
  if (seen[0] < 10000 || seen[1] < 10000) std::printf("too few kinds of states\n");
}

int main() {
  states();
  hg_beam* h = nullptr;
  fakeSetDevice(1);
  hg_beam_create(2, 3, 50, 4, HG_BF16, &h);
  auto expect = [](const char* what, int want, int got) {
    if (got != want) std::printf("%s: %d, not %d\n", what, got, want);
  };
  const int no = HG_ERR_ARG, yes = HG_OK;
  float* const f = reinterpret_cast<float*>(b);
  // Rows of 50 elements, 100 bytes, 6 of them.
  auto select = [&](const char* what, int want, size_t ld, void* tokens, float* picked) {
    expect(what, want, hg_beam_select(h, a, ld, nullptr, 0, f, nullptr, -1, 2, tokens, d, 8, picked,
                                      nullptr, nullptr));
  };
  select("apart", yes, 50, c, f + 16);
  select("tokens over the first row", no, 50, a, f + 16);
  select("tokens over the last row", no, 50, a + 592, f + 16);
  select("tokens behind the logits", yes, 50, a + 600, f + 16);
  select("totals over a row in the middle", no, 50, c, reinterpret_cast<float*>(a + 300));
  select("totals between two rows", yes, 66, c, reinterpret_cast<float*>(a + 100));
  select("totals over the next row", no, 65, c, reinterpret_cast<float*>(a + 100));
  auto reorder = [&](const char* what, int want, void* parents, hg_beam_state s) {
    expect(what, want, hg_beam_reorder(h, parents, 8, 2, &s, 1, nullptr));
  };
  reorder("apart", yes, d, {a, 1, 0, 8, 1, 0, 8});
  reorder("the parents themselves", no, d, {d, 1, 0, 8, 1, 0, 8});
  reorder("parents over the last row", no, a + 40, {a, 1, 0, 8, 1, 0, 8});
  reorder("parents behind the rows", yes, a + 48, {a, 1, 0, 8, 1, 0, 8});
  reorder("parents between two runs", yes, a + 8, {a, 1, 0, 56, 1, 0, 8});
  reorder("parents over the second run", no, a + 16, {a, 1, 0, 56, 1, 0, 8});
  reorder("nothing in it", yes, d, {d, 1, 0, 8, 0, 0, 8});
  hg_beam_destroy(h);
  std::printf("done\n");
  return 0;
}
#endif
