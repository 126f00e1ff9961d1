// Counts, on the host, what calls of the vocabulary operators need of the parts of
// a handle's workspace beside what the handle allocates for them. Reads lines of
//   tp W K max_rows piece_cols sms
// and prints for each: statistics allocated, the most a call writes, rows of the
// accumulator allocated, the most a call writes (or, with EMBED defined, chunks
// allocated and the most a call cuts).
#ifdef EMBED
#include "hg_embed.cu"
#else
#include "hg_loss.cu"
#endif

#include <cstdio>
#include <vector>

using namespace hg::vocab;

// Row counts around every place where a rule on rows can change, and between.
static std::vector<long long> row_counts(long long most) {
  std::vector<long long> n;
  for (long long i = 1; i <= 1024 && i <= most; ++i) n.push_back(i);
  for (long long i = 1024; i <= most; i += i / 16)
    for (long long j = i / 256 * 256 - 1; j <= i / 256 * 256 + 1; ++j)
      if (j <= most) n.push_back(j);
  n.push_back(most);
  return n;
}

int main() {
  hg_vocab h;
  while (std::scanf("%d %d %d %d %d %d", &h.tp, &h.W, &h.K, &h.max_rows, &h.piece_cols, &h.sms) ==
         6) {
    h.vocab = h.tp * h.W;
    long long need[2] = {};
    for (const long long n : row_counts(h.max_rows)) {
      const int N = (int)n;
#ifdef EMBED
      const long long a = div_up(n, run_rows(h, N)), b = 0;
#else
      const long long a = n * 2 * real_shards(h) * div_up(h.W, tile_width(h, N, h.W, 32));
      const long long b = (long long)dx_splits(h, N) * slab_rows(N);
#endif
      if (a > need[0]) need[0] = a;
      if (b > need[1]) need[1] = b;
    }
#ifdef EMBED
    std::printf("%lld %lld\n", embed_grad_chunks(h), need[0]);
#else
    std::printf("%lld %lld %lld %lld\n", loss_partials(h), need[0], loss_accum_rows(h), need[1]);
#endif
  }
  return 0;
}
