// Internal declarations of the beam search's step: the handle, what a call works
// on, and the launches.
#pragma once

#include "hg_vocab.cuh"

struct hg_beam {
  int device = -1;
  int sms = 0;
  int max_items = 0;
  int beams = 0;
  int vocab = 0;
  int picks = 0;
  int dtype = HG_BF16;
  unsigned char* base = nullptr;
  size_t bytes = 0;
  // Parts of the workspace.
  unsigned long long* list = nullptr;  // [max_items * beams][picks]
  float2* stats = nullptr;             // [part_slots][warps] maximum and sum of exponentials
  float* maxima = nullptr;             // [part_slots][threads]
  int* beam_of = nullptr;              // [part_slots] whose part it is
};

namespace hg {
namespace beam {

// The threads of a CTA that searches logits.
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Division of numbers below 2^31 by one that is known when the kernel is launched.
struct Divisor {
  uint32_t by = 1, factor = 0;
  int shift = 0;
  Divisor() = default;
  explicit Divisor(uint32_t d) : by(d) {
    while ((1ull << shift) < d) ++shift;
    factor = (uint32_t)((1ull << (31 + shift)) / d + 1);
    shift += 31;
  }
  __device__ int divide(int n) const {
    return by == 1 ? n : (int)((unsigned long long)(uint32_t)n * factor >> shift);
  }
};

struct SelectCall {
  int items = 0;
  const void* logits = nullptr;
  size_t ld = 0;
  const float* lse = nullptr;
  size_t lse_stride = 0;
  const float* scores = nullptr;
  const uint8_t* finished = nullptr;
  int end = -1;
  void *tokens = nullptr, *parents = nullptr;
  int id_bytes = 8;
  float* picked = nullptr;
  uint8_t* picked_finished = nullptr;
};

cudaError_t select(const hg_beam& h, const SelectCall& c, cudaStream_t stream);
cudaError_t reorder(const hg_beam& h, const void* parents, int id_bytes, int items,
                    const hg_beam_state* states, int n_states, cudaStream_t stream);

// Kernel attributes that the calls need on the current device, set when a handle is made.
cudaError_t select_prepare(const hg_beam& h);
cudaError_t reorder_prepare();

// Parts of rows that any call of the handle has at most (workspace).
long long part_slots(const hg_beam& h);

}  // namespace beam
}  // namespace hg
