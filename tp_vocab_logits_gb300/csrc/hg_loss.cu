// LM head with softmax cross entropy, and its gradient, without the logits.
//
// With z[n][v] = s * x_n . w_v over the real vocabulary (s = logit_scale):
//   loss_n = lse_n - z[n][t_n],  lse_n = log sum_v exp z[n][v]
//   d[n][v] = g_n * s * (exp(z[n][v] - lse_n) - [v = t_n])
//   grad_hidden = d W,  grad_weight = d^T X
//
// Four matrix products on the tensor cores, one kernel template (Kind):
//   kLoss  z = X W^T, a tile of which is reduced to a maximum and a sum of
//          exponentials per row where it leaves the tensor memory; merge_kernel
//          joins the tiles' statistics. The logits are never written.
//   kProb  z again, turned into d in the matrix's type, for a piece of the
//          vocabulary (the columns [c0, c0 + wcols) of every shard)
//   kDx    grad_hidden += d W over the piece, in fp32 (accum)
//   kDw    grad_weight = d^T X for the rows of the piece
// pack_kernel first copies the unmasked rows of hidden together, so that masked
// rows cost nothing and what they hold (NaN too) reaches no product; all
// later kernels read the number of packed rows from device memory.
//
// Everything in the exponent is kept in base 2: y = z * log2(e), ex2(y - lse2).
//
// What bounds them. For many rows the tensor cores: the pipe is busy 89-92 % of the
// time (1536 rows, V=32768, K=2048; gradient of 2048 rows, V=16384, K=4096), and over
// milliseconds the power limit sets the clock: the loss of 8192 rows at V=163840, K=7168
// takes 11.1-12.2 ms (1570-1740 TFLOP/s; a library GEMM sustains 1714), the gradient of
// 4096 rows 16.3-17.6 ms. Hence 256 x 256 tiles of a CTA pair, which read the fewest bytes
// from L2 per product, and two accumulators, so that a tile's epilogue runs beside
// the next one's products. For few rows reading the weights: the loss of one row
// 325-345 us for 2.35 GB (6.8-7.2 TB/s), the gradient of 16 rows 1107-1125 us for the
// weights twice and grad_weight once. Hence one CTA per tile, stages that hold only the
// rows there are, and tile widths that leave every SM the same share of the weights. In
// between, where K is short, the epilogues: 4096 rows at V=32768, K=1024 take 150-154 us
// (1785-1830 TFLOP/s); at K=80 the tensor pipe is busy an eighth of the time.

#include <cfloat>

#include "hg_tcgen05.cuh"
#include "hg_vocab.cuh"

namespace hg {
namespace vocab {
namespace {

enum Kind { kLoss, kProb, kDx, kDw };

constexpr int kTileM = 128;   // rows of a CTA's tile: TMEM lanes
constexpr int kTileN = 256;   // columns of a tile: fp32 TMEM columns
constexpr int kBlockK = 64;   // K per stage: one 128-byte swizzle atom of 16-bit elements
constexpr int kMmaK = 16;     // K per tcgen05.mma of kind::f16
constexpr int kMaxStages = 12;
constexpr uint32_t kBox = 64 * 128;  // a [64 x 64] box of 16-bit elements
constexpr uint32_t kTmemCols = 2 * kTileN;  // two accumulators
constexpr int kEpilogueWarps = 8;
// Warp 0 copies A and warp 2 copies B: one thread for both kept the tensor cores
// waiting (V=49999, K=1544: kDw's four copies a stage took a tenth longer when the
// loop around them was not unrolled). Warp 1 issues the MMAs.
constexpr int kFirstEpilogueWarp = 3;
constexpr int kThreads = 32 * (kFirstEpilogueWarp + kEpilogueWarps);
constexpr uint32_t kStageOut = 32 * 128;  // a warp's staged [32 rows x 128 bytes]
constexpr size_t kMaxSmem = 227 * 1024;
constexpr size_t kFixedSmem = 1024 + 256;  // alignment of the stages, barriers

// K blocks that are summed in the tensor core before the epilogue adds them up in
// registers: the tensor core drops the low bits of every step's sum, always
// downwards, and fp32 additions round them. In long sums of one sign that shows:
// without segments the logsumexp was 1e-6 off at K = 7168 (448 steps); every term of
// d 1.6e-3 (logits of one sign, 16 rows at V=4096, K=7168, fp16; with kProb cut as
// kLoss is, the gradient has the loss's own logits); the mean of grad_hidden
// 4.2e-4 over 65536 columns and of grad_weight 4.0e-4 over 65536 rows, in fp16, whose
// rounding is 4.9e-4 at most. Now 1e-5. The gradient of 4096 rows at V=163840, K=7168
// takes 16.3-16.4 ms for it against 16.3 ms, of 2048 rows at V=16384, K=4096 526-529
// against 515-526 us.
constexpr int kSegment = 16;
// Row tiles that go through the column tiles together, so that both operands of a
// round of tiles come from L2 (gradient of 4096 rows: 17.65 ms, 17.96 with 4 and
// 17.94 with 32).
constexpr int kGroupM = 8;
constexpr int kSmallRows = 128;  // up to here a tile of one CTA holds all rows
// Up to here d is kept as the sum of two rounded terms, the second's rows
// kSplitRows below the first's in prob and packed: they fill rows of a tile that would
// be empty. A row of grad_hidden or grad_weight is mostly one term of d then, and
// over few rows the roundings of those few terms do not average out (16 rows:
// 0.0028 off in bf16, against 0.0017 for the rounding of the result alone). Above, a
// second term would double the work of both products, for less and less: the
// gradient of 600 rows in fp16 is 2.8e-4 off, where the rounding of the result is 2.1e-4.
constexpr int kSplitRows = 64;
constexpr int kOneTileRows = 256;  // and a pair's: packing leaves no tile out
constexpr int kNarrowRounds = 8;  // rounds of tiles up to which narrower ones are tried
constexpr int kMaxSplits = 16;
constexpr int kMinPartBlocks = 8;  // K blocks of a part: fewer, and joining the parts costs more
constexpr unsigned long long kTimeoutNs = 4000000000ull;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct GemmArgs {
  CUtensorMap shard[HG_MAX_TP];  // the weights; kDw: grad_weight (stores)
  CUtensorMap x;                 // hidden, packed or where it lies
  CUtensorMap p;                 // loads from prob
  CUtensorMap out;               // stores: prob (kProb), accum (kDx)
  int* status;
  const int* count;  // packed rows, on the device (nullptr: `rows`)
  int rows;
  int tp, W, vocab, K;
  int c0, wc, wcols;  // the piece: first column, its width in prob, its columns
  int bn;             // columns of a tile
  int stages;         // K blocks in flight
  uint32_t a_bytes;   // of one stage in shared memory
  uint32_t b_bytes;
  uint32_t load_bytes;  // of one stage that the copies of one CTA bring
  uint32_t idesc;
  float c1;           // logit_scale * log2(e)
  Ids targets;        // of the packed rows, or of all
  const float* row_scale;
  const float* row_lse;
  float2* partial;
  int tiles;          // row length of partial: two halves of each vocabulary tile
  float* hit;
  int splits;         // kDx: parts of the sum over the vocabulary
  int accum_rows;     // rows of one part's slab
  int used_rows;      // rows of a tile that can hold any of the call's
  int split;          // d in two terms (kSplitRows)
  int add;            // kDx: add to accum; kDw: add to grad_weight
  const float* unscale;
};

struct Shared {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t acc_full[2];
  uint64_t acc_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
};
static_assert(sizeof(Shared) <= 256, "barriers must fit the 256 bytes kept for them");

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// One bounded try: the thread sleeps until the phase completes or about 20 us
// pass. Without that hint the waiting warps' polls cost the loss of 8192 rows a tenth
// (12.5 against 11.4 ms).
__device__ __forceinline__ bool try_phase(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n"
      " .reg .pred p;\n"
      " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000;\n"
      " selp.u32 %0, 1, 0, p;\n"
      "}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Wait for a phase, bounded in time: on expiry the status word is set and the
// kernel's roles stop issuing work.
__device__ bool wait_phase(uint64_t* bar, uint32_t parity, int* status) {
  if (try_phase(bar, parity)) return true;
  const unsigned long long t0 = globaltimer_ns();
  while (!try_phase(bar, parity)) {
    if (globaltimer_ns() - t0 > kTimeoutNs) {
      atomicExch(status, 1);
      return false;
    }
  }
  return true;
}

// Operand whose M (or N) dimension is contiguous: 64 elements of it to a
// 128-byte row, one row per k, boxes of [64 k][64 elements] one after another.
// Leading byte offset: to the next 64 elements (a box); stride byte offset: to
// the next 8 k.
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(kBox >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

template <int CTAS>
__device__ __forceinline__ void mma_f16(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t accumulate) {
  if constexpr (CTAS == 1)
    asm volatile(
        "{\n"
        " .reg .pred p;\n"
        " setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n"
        "}\n" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n"
        " .reg .pred p;\n"
        " setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n"
        "}\n" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrives on the barrier (in both CTAs of a pair) when the MMAs issued so far are done.
template <int CTAS>
__device__ __forceinline__ void commit(uint64_t* bar) {
  if constexpr (CTAS == 1)
    mma_commit(bar);
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}

// One lane of the converged warp, the same one every time: commits track the MMAs
// that the same thread issued.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// The same shared-memory object in the pair's first CTA.
__device__ __forceinline__ uint32_t in_first_cta(const void* p) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(p)));
  return a;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A copy of a CTA pair: into this CTA's shared memory, counted on the first CTA's barrier.
__device__ __forceinline__ void tma_load_pair(void* dst, const CUtensorMap* tm, int x, int y,
                                              uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2.L2::cache_hint [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(bar), "l"(policy)
      : "memory");
}

__device__ __forceinline__ void tmem_ld_x32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// 64 columns of this warp's 32 lanes, in one load.
__device__ __forceinline__ void tmem_ld_x64(uint32_t taddr, uint32_t (&lo)[32],
                                            uint32_t (&hi)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
      "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(lo[0]), "=r"(lo[1]), "=r"(lo[2]), "=r"(lo[3]), "=r"(lo[4]), "=r"(lo[5]),
        "=r"(lo[6]), "=r"(lo[7]), "=r"(lo[8]), "=r"(lo[9]), "=r"(lo[10]), "=r"(lo[11]),
        "=r"(lo[12]), "=r"(lo[13]), "=r"(lo[14]), "=r"(lo[15]), "=r"(lo[16]), "=r"(lo[17]),
        "=r"(lo[18]), "=r"(lo[19]), "=r"(lo[20]), "=r"(lo[21]), "=r"(lo[22]), "=r"(lo[23]),
        "=r"(lo[24]), "=r"(lo[25]), "=r"(lo[26]), "=r"(lo[27]), "=r"(lo[28]), "=r"(lo[29]),
        "=r"(lo[30]), "=r"(lo[31]), "=r"(hi[0]), "=r"(hi[1]), "=r"(hi[2]), "=r"(hi[3]),
        "=r"(hi[4]), "=r"(hi[5]), "=r"(hi[6]), "=r"(hi[7]), "=r"(hi[8]), "=r"(hi[9]),
        "=r"(hi[10]), "=r"(hi[11]), "=r"(hi[12]), "=r"(hi[13]), "=r"(hi[14]), "=r"(hi[15]),
        "=r"(hi[16]), "=r"(hi[17]), "=r"(hi[18]), "=r"(hi[19]), "=r"(hi[20]), "=r"(hi[21]),
        "=r"(hi[22]), "=r"(hi[23]), "=r"(hi[24]), "=r"(hi[25]), "=r"(hi[26]), "=r"(hi[27]),
        "=r"(hi[28]), "=r"(hi[29]), "=r"(hi[30]), "=r"(hi[31])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* tm, int x, int y,
                                             const void* src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(tm)),
               "r"(x), "r"(y), "r"(smem_u32(src))
               : "memory");
}

__device__ __forceinline__ void tma_add_2d(const CUtensorMap* tm, int x, int y, const void* src) {
  asm volatile(
      "cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2}], "
      "[%3];" ::"l"(reinterpret_cast<uint64_t>(tm)),
      "r"(x), "r"(y), "r"(smem_u32(src))
      : "memory");
}

// One tile of the output and the K blocks [kb0, kb1) that are summed into it.
struct Tile {
  int m;      // row tile (kDw: tile of the shard's rows)
  int n;      // column tile; kLoss, kProb: tile within the shard
  int r;      // shard (kDx: part of the sum)
  int index;  // kLoss: vocabulary tile
  int kb0, kb1;
  // Parts of the sum that the epilogue adds up.
  __device__ __forceinline__ int segments() const {
    return (kb1 - kb0 + kSegment - 1) / kSegment;
  }
};

template <int KIND, int CTAS>
struct Work {
  static constexpr int kRows = kTileM * CTAS;  // rows of a tile of the pair
  int mt, nt, total, kb, per_shard;
  __device__ __forceinline__ Work(const GemmArgs& a, int rows) {
    const int row_tiles = (rows + kRows - 1) / kRows;
    const int k_tiles = (a.K + kTileN - 1) / kTileN;
    if (KIND == kLoss || KIND == kProb) {
      per_shard = (a.wcols + a.bn - 1) / a.bn;
      mt = row_tiles;
      nt = a.tp * per_shard;
      kb = (a.K + kBlockK - 1) / kBlockK;
      total = mt * nt;
    } else if (KIND == kDx) {
      per_shard = (a.wcols + kBlockK - 1) / kBlockK;  // K blocks of a shard
      mt = row_tiles;
      nt = k_tiles;
      kb = a.tp * per_shard;
      total = mt * nt * a.splits;
    } else {
      per_shard = (a.wcols + kRows - 1) / kRows;
      mt = a.tp * per_shard;
      nt = k_tiles;
      kb = (rows + kBlockK - 1) / kBlockK;
      total = mt * nt;
    }
  }
  __device__ __forceinline__ Tile at(const GemmArgs& a, int i) const {
    Tile t;
    int part = 0;
    if (KIND == kDx) {
      part = i / (mt * nt);
      i -= part * (mt * nt);
    }
    const int group = i / (kGroupM * nt);
    const int rem = i - group * (kGroupM * nt);
    const int left = mt - group * kGroupM;
    const int rows = left < kGroupM ? left : kGroupM;
    t.m = group * kGroupM + rem % rows;
    t.n = rem / rows;
    t.index = t.n;
    t.kb0 = 0;
    t.kb1 = kb;
    t.r = part;
    if (KIND == kLoss || KIND == kProb) {
      t.r = t.n / per_shard;
      t.n -= t.r * per_shard;
    } else if (KIND == kDx) {
      t.kb0 = (int)((long long)part * kb / a.splits);
      t.kb1 = (int)((long long)(part + 1) * kb / a.splits);
    } else {
      t.r = t.m / per_shard;
      t.m -= t.r * per_shard;
    }
    return t;
  }
};

// One CTA (CTAS 1) or a pair (CTAS 2) takes tiles i, i + units, ... A pair's tile
// is 256 x 256: each CTA holds 128 rows of A and 128 columns of B, one thread
// of the first issues MMAs that read both, and each CTA's tensor memory holds
// its 128 rows of the sum. LONG: tiles of more than one segment, which are gathered in
// registers first. With one, the accumulator is read and stored a few columns at a
// time (the gradient of 28 rows at V=3391, K=184, fp16: 23.7 us, d gathered first 25.6).
template <int KIND, int CTAS, typename T, bool LONG>
__device__ __forceinline__ void gemm_body(const GemmArgs& a, int unit, int units) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* base = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t stage_bytes = a.a_bytes + a.b_bytes;
  unsigned char* sOut = base + (size_t)a.stages * stage_bytes;
  Shared* sh = reinterpret_cast<Shared*>(sOut + (KIND == kLoss ? 0 : kEpilogueWarps * kStageOut));
  const int warp = (int)threadIdx.x >> 5;
  const int lane = (int)threadIdx.x & 31;
  const int rank = CTAS == 2 ? (int)cta_rank() : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(&sh->full[s], 1);
      mbar_init(&sh->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh->acc_full[b], 1);
      mbar_init(&sh->acc_empty[b], kEpilogueWarps * CTAS);
    }
    mbar_init(&sh->drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    if constexpr (CTAS == 1) {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_u32(&sh->tmem_base)),
                   "r"(kTmemCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_u32(&sh->tmem_base)),
                   "r"(kTmemCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (CTAS == 2) cluster_sync();
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;

  wait_for_predecessor();
  let_successor_start();
  const int packed = a.count ? *a.count : a.rows;  // rows that count
  // At least one row tile is made, so that a piece without rows comes out as zeros.
  const Work<KIND, CTAS> work(
      a, KIND == kDw && a.split ? 2 * kSplitRows : packed > 0 ? packed : 1);
  const int row0 = rank * kTileM;             // of this CTA in a tile
  const int cols = a.bn / CTAS;              // columns of B in this CTA

  // The warps of the two roles below run whole, on values that are the same in
  // every lane, and one elected lane issues: what copies and MMAs take as operands
  // then stays in uniform registers (V=2908, K=4544, 1 row, bound by the 71 K blocks'
  // issue: 23.0 -> 21.5 us).
  if (warp == 0 || warp == 2) {
    // The loss of few rows reads the weights once (evict-first: 1 row at V=163840,
    // K=7168 342 us, against 359 us with the default policy); every other
    // operand is read again by other tiles.
    const uint64_t policy = KIND == kLoss && CTAS == 1 && warp == 2 ? policy_evict_first()
                                                                    : policy_evict_normal();
    const uint32_t first_full = CTAS == 2 ? in_first_cta(sh->full) : 0;
    int stage = 0, issued = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int i = unit; i < work.total && ok; i += units) {
      const Tile t = work.at(a, i);
      // Coordinates of the tile's rows of A or columns of B; kDx walks the shards.
      const int at = warp == 0 ? t.m * work.kRows + row0 : t.n * a.bn + rank * cols;
      int r = KIND == kDx ? t.kb0 / work.per_shard : t.r;
      int b = KIND == kDx ? t.kb0 - r * work.per_shard : 0;
      for (int kb = t.kb0; kb < t.kb1; ++kb) {
        ok = __all_sync(0xffffffffu, wait_phase(&sh->empty[stage], phase ^ 1u, a.status));
        if (!ok) break;
        if (elect_one()) {
          uint64_t* bar = &sh->full[stage];
          unsigned char* dst = base + (size_t)stage * stage_bytes + (warp == 0 ? 0 : a.a_bytes);
          auto load = [&](int box, const CUtensorMap* tm, int x, int y) {
            if constexpr (CTAS == 1)
              tma_load_2d(dst + box * kBox, tm, x, y, bar, policy);
            else
              tma_load_pair(dst + box * kBox, tm, x, y, first_full + (uint32_t)stage * 8, policy);
          };
          if (warp == 0) {
            if (rank == 0) mbar_expect_tx(bar, a.load_bytes * CTAS);
            if (KIND == kLoss || KIND == kProb) {
              load(0, &a.x, kb * kBlockK, at);
            } else if (KIND == kDx) {
              load(0, &a.p, r * a.wc + b * kBlockK, at);
            } else {
#pragma unroll
              for (int j = 0; j < kTileM / 64; ++j)
                load(j, &a.p, r * a.wc + at + j * 64, kb * kBlockK);
            }
          } else {
            if (KIND == kLoss || KIND == kProb) {
              load(0, &a.shard[r], kb * kBlockK, a.c0 + at);
            } else {
#pragma unroll
              for (int j = 0; j < kTileN / CTAS / 64; ++j)
                load(j, KIND == kDx ? &a.shard[r] : &a.x, at + j * 64,
                     KIND == kDx ? a.c0 + b * kBlockK : kb * kBlockK);
            }
          }
        }
        if (KIND == kDx && ++b == work.per_shard) { b = 0; ++r; }
        ++issued;
        if (++stage == a.stages) { stage = 0; phase ^= 1u; }
      }
    }
    // Every copy issued must land before the CTA's shared memory goes: fill j
    // completes the phase of parity (j / stages) & 1 of stage j % stages (of a
    // pair, on the first CTA's barriers; the second waits for it at the end).
    const int last = rank == 0 ? issued - 1 : -1;
    for (int s = 0; s < a.stages && s <= last; ++s) {
      const int j = last - (last - s) % a.stages;
      wait_phase(&sh->full[s], (uint32_t)((j / a.stages) & 1), a.status);
    }
  } else if (warp == 1) {
    if (rank == 0) {
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      const uint32_t A0 = smem_u32(base), B0 = A0 + a.a_bytes;
      const uint64_t da0 = KIND == kDw ? smem_desc_mn(A0) : smem_desc_sw128(A0);
      const uint64_t db0 = KIND == kDw || KIND == kDx ? smem_desc_mn(B0) : smem_desc_sw128(B0);
      for (int i = unit; i < work.total && ok; i += units) {
        const Tile t = work.at(a, i);
        int kb = t.kb0;
        while (kb < t.kb1) {
          const int end = kb + kSegment < t.kb1 ? kb + kSegment : t.kb1;
          ok = __all_sync(0xffffffffu, wait_phase(&sh->acc_empty[acc], acc_phase ^ 1u, a.status));
          if (!ok) break;
          tc_fence_after();
          const uint32_t d = tmem + (uint32_t)(acc * kTileN);
          for (uint32_t accumulate = 0; kb < end; ++kb) {
            ok = __all_sync(0xffffffffu, wait_phase(&sh->full[stage], phase, a.status));
            if (!ok) break;
            tc_fence_after();
            const uint64_t da = da0 + (uint64_t)((uint32_t)stage * (stage_bytes >> 4));
            const uint64_t db = db0 + (uint64_t)((uint32_t)stage * (stage_bytes >> 4));
            // A step of 16 k: 32 bytes along a K-contiguous row, or 16 rows of 128
            // bytes of an operand with one row per k (the address field counts 16).
            constexpr uint64_t step_a = KIND == kDw ? 128 : 2;
            constexpr uint64_t step_b = KIND == kDw || KIND == kDx ? 128 : 2;
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < kBlockK / kMmaK; ++k)
                mma_f16<CTAS>(d, da + step_a * k, db + step_b * k, a.idesc, k ? 1u : accumulate);
              commit<CTAS>(&sh->empty[stage]);
            }
            accumulate = 1;
            if (++stage == a.stages) { stage = 0; phase ^= 1u; }
          }
          if (!ok) break;
          if (elect_one()) commit<CTAS>(&sh->acc_full[acc]);
          if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
        }
      }
      // Every MMA issued must complete before the tensor memory is freed.
      if (elect_one()) commit<CTAS>(&sh->drain);
      wait_phase(&sh->drain, 0, a.status);
    }
  } else {
    // Warps w and w + 4 share 32 rows and take half of the columns each.
    const int quarter = warp & 3;
    const int half = (warp - kFirstEpilogueWarp) >> 2;
    const int first = half * (kTileN / 2);
    const int row = row0 + quarter * 32 + lane;  // in the tile
    unsigned char* const stage_out = sOut + (size_t)(warp - kFirstEpilogueWarp) * kStageOut;
    int acc = 0;
    uint32_t acc_phase = 0;
    const float unscale = KIND == kDw ? *a.unscale : 1.f;
    // Staged stores: the warp's 32 rows of 128 bytes, 16-byte column c of row r
    // at c ^ (r & 7), the 128-byte swizzle of the tensor map.
    auto store_begin = [&]() {
      if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
      __syncwarp();
      return stage_out + (size_t)lane * 128;
    };
    auto store_end = [&](const CUtensorMap* tm, int x, int y, bool add) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        if (add)
          tma_add_2d(tm, x, y, stage_out);
        else
          tma_store_2d(tm, x, y, stage_out);
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      }
    };
    auto acquire = [&]() {
      const bool ready = wait_phase(&sh->acc_full[acc], acc_phase, a.status);
      if (!__all_sync(0xffffffffu, ready)) return false;
      tc_fence_after();
      return true;
    };
    auto acc_at = [&](int column) {
      return tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(acc * kTileN + column);
    };
    auto release = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (CTAS == 1)
          mbar_arrive(&sh->acc_empty[acc]);
        else
          asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                           in_first_cta(&sh->acc_empty[acc]))
                       : "memory");
      }
      if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
    };
    // A tile's sums in this warp's columns, its segments added up in registers.
    auto gather = [&](float (&v)[2][2][32], int segments) {
      for (int seg = 0; seg < segments; ++seg) {
        if (!acquire()) return false;
        if (seg == 0 && first + kTileN / 2 <= a.bn) {
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            uint32_t r[2][32];
            tmem_ld_x64(acc_at(first + s * 64), r[0], r[1]);
#pragma unroll
            for (int j = 0; j < 64; ++j) v[s][j >> 5][j & 31] = __uint_as_float(r[j >> 5][j & 31]);
          }
        } else {
          // Sixteen columns at a time: with 32 the registers spilled (loss of 4096 rows
          // at V=32768, K=1024: 160 against 151 us).
#pragma unroll
          for (int g = 0; g < 8; ++g) {
            if (first + g * 16 >= a.bn) continue;
            uint32_t r[16];
            tmem_ld_32x32b_x16(acc_at(first + g * 16), r);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              float& sum = v[g >> 2][g >> 1 & 1][(g & 1) * 16 + j];
              sum = seg ? sum + __uint_as_float(r[j]) : __uint_as_float(r[j]);
            }
          }
        }
        release();
      }
      return true;
    };
    for (int i = unit; i < work.total; i += units) {
      const Tile t = work.at(a, i);
      if (KIND == kLoss || KIND == kProb) {
        const int n = t.m * work.kRows + row;
        const bool on = n < packed;
        // Columns of the tile in the real vocabulary, and the row's target in it.
        const int col0 = a.c0 + t.n * a.bn;  // within the shard
        int valid = a.vocab - t.r * a.W;
        if (valid > a.W) valid = a.W;
        valid -= col0;
        long long id = -1;
        if (on) id = load_id(a.targets, (size_t)n) - ((long long)t.r * a.W + col0);
        const int at = id >= 0 && id < valid ? (int)id : -1;
        if (KIND == kLoss) {
          float v[2][2][32];
          if (!gather(v, t.segments())) break;
          float top = -INFINITY, sum = 0.f;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int c = first + q * 32;
            if (c >= a.bn) continue;
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < 32; ++j) v[q >> 1][q & 1][j] *= a.c1;
            if (c + 32 > valid) {  // the shard's or the vocabulary's last columns
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (c + j >= valid) v[q >> 1][q & 1][j] = -INFINITY;
            }
#pragma unroll
            for (int j = 0; j < 32; ++j) mx = fmaxf(mx, v[q >> 1][q & 1][j]);
            const float now = fmaxf(top, mx);
            // Nothing above -inf yet: ex2(-inf - 0) = 0 adds nothing, and a NaN still shows.
            const float ref = now == -INFINITY ? 0.f : now;
            float part = 0.f;
#pragma unroll
            for (int j = 0; j < 32; ++j) part += ex2(v[q >> 1][q & 1][j] - ref);
            sum = sum * ex2(top - ref) + part;
            top = now;
            if (at >= c && at < c + 32) {
              float z = 0.f;
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (at == c + j) z = v[q >> 1][q & 1][j];
              a.hit[n] = z;
            }
          }
          if (on && n < a.rows)
            a.partial[(size_t)n * a.tiles + t.index * 2 + half] = make_float2(top, sum);
        } else {
          const float scale = on ? a.row_scale[n] : 0.f;
          const float lse = on ? a.row_lse[n] : 0.f;
          const bool rows_full = __all_sync(0xffffffffu, on);
          // 64 columns from c on: the logits in v become d, and are stored.
          auto emit = [&](int c, float (&v)[2][32]) {
            if (t.n * a.bn + c >= a.wc) return;  // beyond the piece's place in prob
            if (a.split && quarter * 32 >= kSplitRows) return;
            const int x = t.r * a.wc + t.n * a.bn + c;
            const int y = t.m * work.kRows + row0 + quarter * 32;
            auto store = [&](int term) {
              unsigned char* dst = store_begin();
#pragma unroll
              for (int q = 0; q < 8; ++q) {
                uint32_t w[4];
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                  const int j = q * 8 + h * 2;
                  float& lo = v[j >> 5][j & 31];
                  float& hi = v[j >> 5][(j & 31) + 1];
                  w[h] = Elem<T>::pack2(lo, hi);
                  if (CTAS == 1 && term == 0) {  // what the rounding left
                    const float2 kept = Elem<T>::unpack2(w[h]);
                    lo -= kept.x;
                    hi -= kept.y;
                  }
                }
                *reinterpret_cast<uint4*>(dst + ((q ^ (lane & 7)) << 4)) =
                    make_uint4(w[0], w[1], w[2], w[3]);
              }
              store_end(&a.out, x, y + term * kSplitRows, false);
            };
            // Four instructions an element where nothing is masked; the target, in one
            // chunk of a row's hundreds, on its own.
#pragma unroll
            for (int j = 0; j < 64; ++j)
              v[j >> 5][j & 31] = ex2(fmaf(v[j >> 5][j & 31], a.c1, -lse)) * scale;
            if (at >= c && at < c + 64) {
#pragma unroll
              for (int j = 0; j < 64; ++j)
                if (at == c + j) v[j >> 5][j & 31] -= scale;
            }
            if (!rows_full || c + 64 > valid) {
#pragma unroll
              for (int j = 0; j < 64; ++j)
                if (!on || c + j >= valid) v[j >> 5][j & 31] = 0.f;
            }
            store(0);
            if (CTAS == 1 && a.split) store(1);
          };
          if constexpr (LONG) {
            float v[2][2][32];
            if (!gather(v, t.segments())) break;
#pragma unroll
            for (int s = 0; s < 2; ++s)
              if (first + s * 64 < a.bn) emit(first + s * 64, v[s]);
          } else {
            if (!acquire()) break;
            if (first >= a.bn) release();
            for (int c = first; c < a.bn && c < first + kTileN / 2; c += 64) {
              uint32_t r[2][32];
              tmem_ld_x64(acc_at(c), r[0], r[1]);
              if (c + 64 >= a.bn || c + 64 == first + kTileN / 2) release();
              float v[2][32];
#pragma unroll
              for (int j = 0; j < 64; ++j) v[j >> 5][j & 31] = __uint_as_float(r[j >> 5][j & 31]);
              emit(c, v);
            }
          }
        }
      } else if (KIND == kDx) {
        auto emit = [&](int c, uint32_t (&v)[32]) {
          // Nobody reads the tile's other rows.
          if (t.n * kTileN + c >= a.K || (CTAS == 1 && quarter * 32 >= a.used_rows)) return;
          unsigned char* dst = store_begin();
#pragma unroll
          for (int q = 0; q < 8; ++q)
            *reinterpret_cast<uint4*>(dst + ((q ^ (lane & 7)) << 4)) =
                make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
          const int y = t.r * a.accum_rows + t.m * work.kRows + row0 + quarter * 32;
          store_end(&a.out, t.n * kTileN + c, y, a.add != 0);
        };
        if constexpr (LONG) {
          float v[2][2][32];
          if (!gather(v, t.segments())) break;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t r[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(v[q >> 1][q & 1][j]);
            emit(first + q * 32, r);
          }
        } else {
          if (!acquire()) break;
          for (int c = first; c < first + kTileN / 2; c += 32) {
            uint32_t r[32];
            tmem_ld_x32(acc_at(c), r);
            if (c + 32 == first + kTileN / 2) release();
            emit(c, r);
          }
        }
      } else {
        auto emit = [&](int c, float (&v)[2][32]) {
          const int y = a.c0 + t.m * work.kRows + row0 + quarter * 32;
          if (t.n * kTileN + c >= a.K || y >= a.W) return;
          unsigned char* dst = store_begin();
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            uint32_t w[4];
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              const int j = q * 8 + h * 2;
              w[h] = Elem<T>::pack2(v[j >> 5][j & 31] * unscale, v[j >> 5][(j & 31) + 1] * unscale);
            }
            *reinterpret_cast<uint4*>(dst + ((q ^ (lane & 7)) << 4)) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
          // Added to what is there by the copy engine, in the matrix's type: one
          // rounding of the gradient and one of the sum, and nothing read back.
          store_end(&a.shard[t.r], t.n * kTileN + c, y, a.add != 0);
        };
        if constexpr (LONG) {
          float v[2][2][32];
          if (!gather(v, t.segments())) break;
#pragma unroll
          for (int s = 0; s < 2; ++s) emit(first + s * 64, v[s]);
        } else {
          if (!acquire()) break;
          for (int c = first; c < first + kTileN / 2; c += 64) {
            uint32_t r[2][32];
            tmem_ld_x64(acc_at(c), r[0], r[1]);
            if (c + 64 == first + kTileN / 2) release();
            float v[2][32];
#pragma unroll
            for (int j = 0; j < 64; ++j) v[j >> 5][j & 31] = __uint_as_float(r[j >> 5][j & 31]);
            emit(c, v);
          }
        }
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }

  // A pair leaves together: copies, MMAs and arrivals of one CTA reach into the other.
  tc_fence_before();
  __syncthreads();
  if constexpr (CTAS == 2) cluster_sync();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    if constexpr (CTAS == 1)
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                   "r"(kTmemCols)
                   : "memory");
    else
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                   "r"(kTmemCols)
                   : "memory");
  }
}

template <int KIND, int CTAS, typename T, bool LONG>
__global__ void __launch_bounds__(kThreads, 1) gemm_kernel(const __grid_constant__ GemmArgs a) {
  gemm_body<KIND, CTAS, T, LONG>(a, (int)blockIdx.x / CTAS, (int)gridDim.x / CTAS);
}

// Both gradients of a small piece in one launch, the CTAs shared out between them:
// each alone leaves most of the time to the start and the end of a kernel (28
// rows at V=3391, K=184: 24 us for the gradient, against 29 us with two launches).
struct BothArgs {
  GemmArgs dx, dw;
  int dx_units;
};

template <int CTAS, typename T, bool LONG>
__global__ void __launch_bounds__(kThreads, 1) both_kernel(const __grid_constant__ BothArgs a) {
  const int unit = (int)blockIdx.x / CTAS;
  const int units = (int)gridDim.x / CTAS;
  if (unit < a.dx_units)
    gemm_body<kDx, CTAS, T, LONG>(a.dx, unit, a.dx_units);
  else
    gemm_body<kDw, CTAS, T, LONG>(a.dw, unit - a.dx_units, units - a.dx_units);
}

// ---- rows ----------------------------------------------------------------------

constexpr int kPackThreads = 512;
constexpr int kPackWarps = kPackThreads / 32;

struct PackArgs {
  const void* hidden;
  size_t ld;
  Ids targets;
  int N, K, vocab;
  int grad;  // for the gradient (targets outside the vocabulary are masked too)
  float logit_scale;
  const float* lse;
  const float* grad_loss;
  float* loss;     // zeros in masked rows
  float* lse_out;
  void* grad_hidden;
  size_t ld_grad;
  float headroom;  // the largest |row_scale| is made this
  int split;       // every row once more, kSplitRows further on
  void* packed;
  int pitch;
  int* count;
  float* unscale;
  int* row_of;
  int* target;
  float* row_scale;
  float* row_lse;
};

__device__ __forceinline__ bool unmasked(const PackArgs& a, long long id) {
  return id >= 0 && (!a.grad || id < a.vocab);
}

// Copies the unmasked rows of hidden together, in order, each to the start of a
// 128-byte line: rows that start inside a 32-byte sector slow TMA down (at V=49999,
// K=1000 the loss of 512 rows took 82 us with the rows as they lay and 69 us
// with them packed so, against 57 us at K=1024). CTA b has the rows
// [b * N / G, (b + 1) * N / G); each CTA counts the unmasked rows before its own
// from the targets (a few bytes per row from L2, against K elements copied), so
// the CTAs need nothing from one another. The rows up to the next multiple of
// 64 are filled with zeros: kDw sums 64 rows at a time. Of few rows (`split`)
// there are two such blocks.
__global__ void __launch_bounds__(kPackThreads) pack_kernel(const __grid_constant__ PackArgs a) {
  __shared__ int warp_sum[2][kPackWarps];
  __shared__ int kept[kPackWarps];
  __shared__ float warp_max[kPackWarps];
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  wait_for_predecessor();
  let_successor_start();
  const long long G = gridDim.x;
  const int lo = (int)(blockIdx.x * (long long)a.N / G);
  const int hi = (int)((blockIdx.x + 1) * (long long)a.N / G);
  int before = 0, all = 0;
  float most = 0.f;
  for (int n = threadIdx.x; n < a.N; n += kPackThreads) {
    if (!unmasked(a, load_id(a.targets, n))) continue;
    ++all;
    if (n < lo) ++before;
    if (a.grad) most = fmaxf(most, fabsf(a.grad_loss[n] * a.logit_scale));
  }
  for (int o = 16; o; o >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, o);
    all += __shfl_xor_sync(0xffffffffu, all, o);
    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  }
  if (lane == 0) {
    warp_sum[0][warp] = before;
    warp_sum[1][warp] = all;
    warp_max[warp] = most;
  }
  __syncthreads();
  before = all = 0;
  most = 0.f;
  for (int w = 0; w < kPackWarps; ++w) {
    before += warp_sum[0][w];
    all += warp_sum[1][w];
    most = fmaxf(most, warp_max[w]);
  }
  // The largest row_scale becomes `headroom`, so that equal upstream gradients (a
  // mean's) give factors that are exact, and d's largest terms (-1 of the target)
  // with them.
  const bool rescale = a.grad && most > 1e-30f && most <= FLT_MAX;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *a.count = all;
    *a.unscale = rescale ? most / a.headroom : 1.f;
  }

  const uint4 zero = make_uint4(0, 0, 0, 0);
  const int vecs = a.K / 8;
  uint4* const packed = static_cast<uint4*>(a.packed);
  // Rows go in rounds of `rows`; the warps share them out evenly, several to a
  // row where a CTA has few.
  int per_row = 1;
  while (per_row < kPackWarps && (hi - lo) * per_row * 2 <= kPackWarps) per_row *= 2;
  const int rows = kPackWarps / per_row;
  const int slot = warp / per_row;
  const int part = (warp - slot * per_row) * 32 + lane;
  const int step = per_row * 32;
  int at = before;
  for (int n0 = lo; n0 < hi; n0 += rows) {
    // Row n0 + slot; its place follows the unmasked rows of the slots before it.
    const int n = n0 + slot;
    const long long id = n < hi ? load_id(a.targets, n) : -1;
    const bool keep = n < hi && unmasked(a, id);
    __syncthreads();  // the flags of the last round have been read
    if (part == 0) kept[slot] = keep;
    __syncthreads();
    int to = at;
    for (int w = 0; w < rows; ++w) {
      const int f = kept[w];
      at += f;
      if (w < slot) to += f;
    }
    if (n >= hi) continue;
    if (keep) {
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.hidden) +
                                                        (size_t)n * a.ld);
      uint4* dst = packed + (size_t)to * (a.pitch / 8);
      for (int v = part; v < vecs; v += 4 * step) {
        uint4 x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (v + step * j < vecs) x[j] = src[v + step * j];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (v + step * j < vecs) dst[v + step * j] = x[j];
        if (a.split)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (v + step * j < vecs) dst[kSplitRows * (a.pitch / 8) + v + step * j] = x[j];
      }
      if (part == 0) {
        a.row_of[to] = n;
        a.target[to] = id < a.vocab ? (int)id : -1;
        if (a.grad) {
          const float g = a.grad_loss[n] * a.logit_scale;
          a.row_scale[to] = rescale ? g / most * a.headroom : g;
          a.row_lse[to] = a.lse[n] * kLog2e;
        }
      }
    } else if (a.grad) {
      if (a.grad_hidden) {
        uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.grad_hidden) +
                                              (size_t)n * a.ld_grad);
        for (int v = part; v < vecs; v += step) dst[v] = zero;
      }
    } else if (part == 0) {
      a.loss[n] = 0.f;
      a.lse_out[n] = 0.f;
    }
  }
  const int end = a.split ? 2 * kSplitRows : (int)round_up(all > 0 ? all : 1, 64);
  for (int to = all + (int)blockIdx.x * kPackWarps + warp; to < end; to += (int)G * kPackWarps)
    if (!a.split || to < kSplitRows || to >= kSplitRows + all)
      for (int v = lane; v < vecs; v += 32) packed[(size_t)to * (a.pitch / 8) + v] = zero;
}

struct MergeArgs {
  const float2* partial;
  int tiles;
  const float* hit;
  const int* count;  // packed rows (nullptr: the rows are the caller's own)
  const int* row_of;
  Ids targets;
  int vocab;
  float* loss;
  float* lse;
};

__device__ __forceinline__ void join_stats(float& top, float& sum, float t, float s) {
  const float now = fmaxf(top, t);
  const float ref = now == -INFINITY ? 0.f : now;
  sum = sum * ex2(top - ref) + s * ex2(t - ref);
  top = now;
}

// Joins the tiles' statistics of a row: one CTA per row, so that a single row's
// hundreds of tiles are read at once (about 3 us; a warp took 13 us for the 1472 of
// one row at V=163840).
constexpr int kMergeThreads = 128;

__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const __grid_constant__ MergeArgs a) {
  __shared__ float2 joined[kMergeThreads / 32];
  wait_for_predecessor();
  let_successor_start();
  const int i = blockIdx.x;
  if (a.count && i >= *a.count) return;
  const float2* p = a.partial + (size_t)i * a.tiles;
  float top = -INFINITY, sum = 0.f;
  for (int t0 = threadIdx.x; t0 < a.tiles; t0 += 4 * kMergeThreads) {
    float2 x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = t0 + j * kMergeThreads;
      x[j] = t < a.tiles ? p[t] : make_float2(-INFINITY, 0.f);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) join_stats(top, sum, x[j].x, x[j].y);
  }
  for (int o = 16; o; o >>= 1) {
    const float t = __shfl_xor_sync(0xffffffffu, top, o);
    const float s = __shfl_xor_sync(0xffffffffu, sum, o);
    join_stats(top, sum, t, s);
  }
  if ((threadIdx.x & 31) == 0) joined[threadIdx.x >> 5] = make_float2(top, sum);
  __syncthreads();
  if (threadIdx.x) return;
#pragma unroll
  for (int w = 1; w < kMergeThreads / 32; ++w) join_stats(top, sum, joined[w].x, joined[w].y);
  const long long id = load_id(a.targets, i);
  const int n = a.count ? a.row_of[i] : i;
  const bool masked = !a.count && id < 0;
  const float rest = log2f(sum);
  // The difference to the largest logit first: it is exact where they are near.
  const float loss = id >= 0 && id < a.vocab ? (top - a.hit[i] + rest) * kLn2 : NAN;
  a.loss[n] = masked ? 0.f : loss;
  a.lse[n] = masked ? 0.f : (top + rest) * kLn2;
}

struct FinishArgs {
  const float* accum;
  int splits, accum_rows, K, pitch;
  int split;  // two rows of accum to a row
  const int* count;
  const int* row_of;
  const float* unscale;
  void* grad;
  size_t ld;
};

// grad_hidden: the parts' sums in order, rounded once, to the rows they belong to.
// A thread has four elements; kBatch parts' loads are in flight at once (one
// after another, 16 parts took 8 us).
template <typename T>
__global__ void __launch_bounds__(256) finish_kernel(const __grid_constant__ FinishArgs a) {
  wait_for_predecessor();
  let_successor_start();
  constexpr int kBatch = 8;
  const int quads = a.K / 4;
  const long long total = (long long)*a.count * quads;
  const float unscale = *a.unscale;
  const int halves = a.split ? 2 : 1;
  const int parts = a.splits * halves;
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
    const int row = (int)(i / quads);
    const int v = (int)(i - (long long)row * quads);
    const float* const src = a.accum + (size_t)row * a.pitch + (size_t)v * 4;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p0 = 0; p0 < parts; p0 += kBatch) {
      float4 x[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int p = p0 + j < parts ? p0 + j : parts - 1;
        const int part = p / halves;
        const size_t at = (size_t)part * a.accum_rows + (p - part * halves) * kSplitRows;
        x[j] = *reinterpret_cast<const float4*>(src + at * a.pitch);
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        if (p0 + j >= parts) break;
        s.x += x[j].x;
        s.y += x[j].y;
        s.z += x[j].z;
        s.w += x[j].w;
      }
    }
    uint2 x;
    x.x = Elem<T>::pack2(s.x * unscale, s.y * unscale);
    x.y = Elem<T>::pack2(s.z * unscale, s.w * unscale);
    *reinterpret_cast<uint2*>(static_cast<T*>(a.grad) + (size_t)a.row_of[row] * a.ld +
                              (size_t)v * 4) = x;
  }
}

// ---- host ----------------------------------------------------------------------

// Row-major [rows, cols] matrix, rows `ld` elements apart, box of [box_rows][128 bytes].
bool encode(CUtensorMap* tm, const void* ptr, int dtype, uint64_t rows, uint64_t cols, uint64_t ld,
            uint32_t box_rows) {
  const EncodeTiled fn = tensor_map_encoder();
  if (!fn) return false;
  const uint32_t e = (uint32_t)elem_bytes(dtype);
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {ld * e};
  cuuint32_t box[2] = {128 / e, box_rows};
  cuuint32_t steps[2] = {1, 1};
  const CUtensorMapDataType type = dtype == HG_BF16   ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                   : dtype == HG_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                      : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
  return fn(tm, type, 2, const_cast<void*>(ptr), dims, strides, box, steps,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Real vocabulary rows of shard r.
int shard_rows(const hg_vocab& h, int r) {
  const long long left = (long long)h.vocab - (long long)r * h.W;
  return (int)(left < 0 ? 0 : left < h.W ? left : h.W);
}

// Shards that hold part of the real vocabulary.
int real_shards(const hg_vocab& h) { return (int)div_up(h.vocab, h.W); }

// The weights' maps stop at the real vocabulary: what lies beyond reads as
// zeros. (A shard without any real row keeps one, whose logits kProb masks.)
bool encode_weights(const hg_vocab& h, const void* const* w, uint32_t box_rows, CUtensorMap* tm) {
  for (int r = 0; r < h.tp; ++r) {
    const int rows = shard_rows(h, r);
    if (!encode(&tm[r], w[r], h.dtype, rows > 0 ? rows : 1, h.K, h.K, box_rows)) return false;
  }
  return true;
}

// Instruction descriptor of tcgen05.mma kind::f16: D fp32 (bits 4-5 = 1), A and
// B bf16 (1) or fp16 (0) (bits 7-9, 10-12), A and B transposed (bits 15, 16:
// their M or N dimension is contiguous), N >> 3 in bits 17-22, M >> 4 in bits
// 24-28.
uint32_t instruction(int dtype, bool a_mn, bool b_mn, int m, int n) {
  const uint32_t type = dtype == HG_BF16 ? 1u : 0u;
  return (1u << 4) | (type << 7) | (type << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// How one product is cut: a pair of CTAs or one, the rows of A and columns of B
// that a CTA loads per stage.
struct Shape {
  int ctas = 2;
  int a_rows = kTileM;
  int b_cols = kTileN / 2;
};

template <int KIND, int CTAS, typename T, bool LONG>
cudaError_t launch_as(const GemmArgs& a, int sms, cudaStream_t stream) {
  return launch_dependent(gemm_kernel<KIND, CTAS, T, LONG>, a, (unsigned)(sms / CTAS * CTAS),
                          kThreads, kMaxSmem, CTAS, stream);
}

// Units (CTAs or pairs) for the hidden gradient when a piece's two gradients share
// a launch, in proportion to their K blocks and tiles; 0 where the piece is large enough
// for a launch each. A tile's ends count as kTileEnds blocks: with 0, 3 and 12 the
// gradient of 300 rows at V=30000, K=512 took 73.2, 69.3 and 75.7 us, with 6 69.5
// (K=128: 53.8, 53.8 and 60.1, with 6 53.8; 600 rows at V=4096, K=512: 32.8, 29.5, 29.5
// and 29.5); single CTAs would rather have 0 (16 rows at V=32000, K=1024: 65.4 against
// 72.4 us).
constexpr int kTileEnds = 6;
// Blocks of a unit up to which the launch is shared. Shared against apart: 28 rows at
// V=3391, K=184 22.7 against 29.5 us, 300 rows at V=30000, K=512 69.5 against 75.6, 1000
// rows at V=8192, K=512 43.7 against 49.0. Above 64 it still gains, but less of a longer
// call (1000 rows at V=8192, K=1024: 56.8 against 62.7 us; 2000 rows: 92.3 against 99.0).
constexpr int kBothBlocks = 64;

int both_units(const hg_vocab& h, const GemmArgs& dx, const GemmArgs& dw, int N, int ctas) {
  const long long rows = div_up(N, kTileM * ctas), cols = div_up(h.K, kTileN);
  const long long dx_blocks = dx.tp * div_up(dx.wcols, kBlockK) * rows * cols;
  const long long dx_tiles = rows * cols * dx.splits;
  const long long dw_tiles = dw.tp * div_up(dw.wcols, kTileM * ctas) * cols;
  const long long dw_blocks = dw_tiles * div_up(N, kBlockK);
  const long long dx_cost = dx_blocks + kTileEnds * dx_tiles;
  const long long cost = dx_cost + dw_blocks + kTileEnds * dw_tiles;
  const long long units = h.sms / ctas;
  if (cost > kBothBlocks * units) return 0;
  long long n = (units * dx_cost + cost / 2) / cost;
  if (n > dx_tiles) n = dx_tiles;
  return (int)(n < 1 ? 1 : n < units ? n : units - 1);
}

template <int CTAS, typename T, bool LONG>
cudaError_t launch_both(const BothArgs& a, int sms, cudaStream_t stream) {
  return launch_dependent(both_kernel<CTAS, T, LONG>, a, (unsigned)(sms / CTAS * CTAS), kThreads,
                          kMaxSmem, CTAS, stream);
}

template <int CTAS, typename T>
cudaError_t allow_smem_all() {
  const void* const kernels[] = {
      (const void*)gemm_kernel<kLoss, CTAS, T, true>,
      (const void*)gemm_kernel<kProb, CTAS, T, false>,
      (const void*)gemm_kernel<kProb, CTAS, T, true>,
      (const void*)gemm_kernel<kDx, CTAS, T, false>,
      (const void*)gemm_kernel<kDx, CTAS, T, true>,
      (const void*)gemm_kernel<kDw, CTAS, T, false>,
      (const void*)gemm_kernel<kDw, CTAS, T, true>,
      (const void*)both_kernel<CTAS, T, false>,
      (const void*)both_kernel<CTAS, T, true>};
  for (const void* k : kernels) {
    const cudaError_t e =
        cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSmem);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int KIND>
void stage_layout(const Shape& shape, GemmArgs& a) {
  a.a_bytes = (uint32_t)round_up(shape.a_rows * 128, 1024);
  a.b_bytes = (uint32_t)shape.b_cols * 128;
  a.load_bytes = (uint32_t)(shape.a_rows + shape.b_cols) * 128;
  const size_t room = kMaxSmem - kFixedSmem - (KIND == kLoss ? 0 : kEpilogueWarps * kStageOut);
  const size_t stages = room / (a.a_bytes + a.b_bytes);
  a.stages = (int)(stages < kMaxStages ? stages : kMaxStages);
}

template <int KIND, bool LONG>
cudaError_t launch_cut(const hg_vocab& h, const Shape& shape, GemmArgs& a, cudaStream_t stream) {
  stage_layout<KIND>(shape, a);
  const bool bf16 = h.dtype == HG_BF16;
  if (shape.ctas == 2)
    return bf16 ? launch_as<KIND, 2, __nv_bfloat16, LONG>(a, h.sms, stream)
                : launch_as<KIND, 2, __half, LONG>(a, h.sms, stream);
  return bf16 ? launch_as<KIND, 1, __nv_bfloat16, LONG>(a, h.sms, stream)
              : launch_as<KIND, 1, __half, LONG>(a, h.sms, stream);
}

// `blocks`: K blocks of a tile, at most.
template <int KIND>
cudaError_t launch(const hg_vocab& h, const Shape& shape, GemmArgs& a, long long blocks,
                   cudaStream_t stream) {
  if constexpr (KIND != kLoss)
    if (blocks <= kSegment) return launch_cut<KIND, false>(h, shape, a, stream);
  return launch_cut<KIND, true>(h, shape, a, stream);
}

template <bool LONG>
cudaError_t launch_both_cut(const hg_vocab& h, int ctas, const BothArgs& a, cudaStream_t stream) {
  if (h.dtype == HG_BF16)
    return ctas == 2 ? launch_both<2, __nv_bfloat16, LONG>(a, h.sms, stream)
                     : launch_both<1, __nv_bfloat16, LONG>(a, h.sms, stream);
  return ctas == 2 ? launch_both<2, __half, LONG>(a, h.sms, stream)
                   : launch_both<1, __half, LONG>(a, h.sms, stream);
}

// The shape of a product whose rows are the call's N: for few rows one CTA per
// tile, which then holds all of them, and loads no more of A than there are
// (the tile's other rows keep what shared memory held, and only reach output rows
// nobody reads).
Shape row_shape(int N, int columns) {
  Shape s;
  s.ctas = N > kSmallRows ? 2 : 1;
  s.a_rows = N > kSmallRows ? kTileM : (int)round_up(N > 0 ? N : 1, 8);
  s.b_cols = columns / s.ctas;
  return s;
}

// Width of the vocabulary tiles: the one that leaves the busiest SM the least.
// That is bytes of weights for few rows and MMA columns for many; either way a
// tile has a part that does not shrink with it: the rows it reads from L2, half
// as dear as the weights, or the ends of its pipeline. (333 rows at V=49999,
// K=1000: 224 columns 56 us, 256 columns 60 us.) Where tiles go many times
// round (kNarrowRounds), the widest.
int tile_width(const hg_vocab& h, int N, int cols, int step) {
  const int ctas = row_shape(N, kTileN).ctas;
  const long long row_tiles = div_up(N > 0 ? N : 1, kTileM * ctas);
  const int fixed = ctas == 1 ? (int)round_up(N > 0 ? N : 1, 8) / 2 : 16;
  int best = kTileN;
  if (ctas == 2 && row_tiles * h.tp * div_up(cols, kTileN) > kNarrowRounds * h.sms / 2)
    return best;
  long long least = -1;
  for (int bn = kTileN; bn >= (ctas == 1 ? step : kTileN / 2); bn -= step) {
    const long long tiles = row_tiles * h.tp * div_up(cols, bn);
    const long long cost = div_up(tiles * ctas, h.sms) * (bn + fixed);
    if (least < 0 || cost < least) {
      least = cost;
      best = bn;
    }
  }
  return best;
}

// Rows of one of kDx's slabs: whole tiles.
int slab_rows(int N) {
  return (int)round_up(N > 0 ? N : 1, kTileM * row_shape(N, kTileN).ctas);
}

// Parts of the sum over the vocabulary in kDx. More of them fill the last round of
// tiles better, but each is a slab of fp32 that is written and read again: take
// the least of the two times together, at kBlockNs for a K block of a tile
// and the copy rate for the slabs.
//
// kBlockNs is a pair's time for 256 x 256 x 64 products at the tensor cores' pace. A CTA
// of few rows takes half of that from L2 and twice from HBM, but their slabs are small:
// with a quarter, a half, two and four times of it the hidden gradient of 16 rows
// at V=163840, K=7168 (with its logits) took 706, 705, 726 and 726 us against 706, of 128
// rows 715, 715, 738 and 737 against 715, of 2048 rows at V=16384, K=4096 338, 338, 359
// and 359 against 338, of 2500 rows at V=32768, K=2048 453, 444, 451 and 466 against 443.
constexpr double kBlockNs = 340;

int dx_splits(const hg_vocab& h, int N) {
  const int ctas = row_shape(N, kTileN).ctas;
  const long long tiles = div_up(N > 0 ? N : 1, kTileM * ctas) * div_up(h.K, kTileN);
  const long long units = h.sms / ctas;
  const int cols = h.piece_cols < h.W ? h.piece_cols : h.W;
  const long long kb = real_shards(h) * div_up(cols, kBlockK);
  const double slab_ns = (double)slab_rows(N) * h.K * 8 / 6800;
  int best = 1;
  double least = 0;
  for (int s = 1; s <= kMaxSplits && (s == 1 || s * kMinPartBlocks <= kb); ++s) {
    const double ns = (double)div_up(tiles * s, units) / s * kb * kBlockNs + s * slab_ns;
    if (s == 1 || ns < least) {
      least = ns;
      best = s;
    }
  }
  return best;
}

unsigned row_blocks(const hg_vocab& h, int N) {
  return (unsigned)(N < 1 ? 1 : N < 2 * h.sms ? N : 2 * h.sms);
}

PackArgs pack_args(const hg_vocab& h, const LossCall& c) {
  PackArgs a = {};
  a.hidden = c.hidden;
  a.ld = c.ld;
  a.targets = c.targets;
  a.N = c.N;
  a.K = h.K;
  a.vocab = h.vocab;
  a.logit_scale = c.logit_scale;
  a.lse = c.lse;
  a.grad_loss = c.grad_loss;
  a.loss = c.loss;
  a.lse_out = c.lse_out;
  a.grad_hidden = c.grad_hidden;
  a.ld_grad = c.ld_grad;
  a.packed = h.packed;
  a.pitch = h.pitch;
  a.count = h.count;
  a.unscale = h.unscale;
  a.row_of = h.row_of;
  a.target = h.target;
  a.row_scale = h.row_scale;
  a.row_lse = h.row_lse;
  return a;
}

GemmArgs gemm_args(const hg_vocab& h, const LossCall& c) {
  GemmArgs a = {};
  a.status = h.status;
  a.rows = c.N;
  a.tp = h.tp;
  a.W = h.W;
  a.vocab = h.vocab;
  a.K = h.K;
  a.c1 = c.logit_scale * kLog2e;
  a.row_scale = h.row_scale;
  a.row_lse = h.row_lse;
  a.partial = h.partial;
  a.hit = h.hit;
  a.unscale = h.unscale;
  a.splits = 1;
  a.bn = kTileN;

  return a;
}

}  // namespace

long long loss_partials(const hg_vocab& h) {
  // Few rows may have tiles of 32 columns; many the widest, or half as wide where
  // kNarrowRounds allow no more tiles than that (tile_width).
  const long long rows = h.max_rows;  // rows * tp passes 32 bits in handles that fit the card
  const long long few_rows = rows < kSmallRows ? rows : kSmallRows;
  const long long few = few_rows * h.tp * div_up(h.W, 32);
  const long long many = rows * h.tp * div_up(h.W, kTileN);
  long long narrow = rows * h.tp * div_up(h.W, kTileN / 2);
  const long long most = 2ll * kTileM * 2 * (kNarrowRounds * h.sms / 2 + h.tp);
  if (narrow > most) narrow = most;
  const long long least = few > many ? few : many;
  return 2 * (least > narrow ? least : narrow);
}

long long loss_rows_pad(long long rows) { return round_up(rows, 256); }

long long loss_accum_rows(const hg_vocab& h) {
  long long most = 0;
  for (long long n = kTileM;; n += kTileM) {
    const int N = (int)(n < h.max_rows ? n : h.max_rows);
    const long long rows = (long long)dx_splits(h, N) * slab_rows(N);
    if (rows > most) most = rows;
    if (n >= h.max_rows) return most;
  }
}

cudaError_t loss_prepare(const hg_vocab& h) {
  const bool bf16 = h.dtype == HG_BF16;
  const cudaError_t e = bf16 ? allow_smem_all<1, __nv_bfloat16>() : allow_smem_all<1, __half>();
  if (e != cudaSuccess) return e;
  return bf16 ? allow_smem_all<2, __nv_bfloat16>() : allow_smem_all<2, __half>();
}

cudaError_t loss(const hg_vocab& h, const LossCall& c, cudaStream_t stream) {
  GemmArgs a = gemm_args(h, c);
  // Packing pays where it leaves row tiles out, or where rows are not whole lines.
  const bool lines = (c.ld * 2) % 128 == 0 && reinterpret_cast<uintptr_t>(c.hidden) % 128 == 0;
  const bool pack = c.N > (lines ? kOneTileRows : kSmallRows);
  a.wcols = h.W;
  a.bn = tile_width(h, c.N, h.W, 32);
  const Shape shape = row_shape(c.N, a.bn);
  a.tp = real_shards(h);
  a.tiles = (int)(2 * a.tp * div_up(h.W, a.bn));
  a.idesc = instruction(h.dtype, false, false, kTileM * shape.ctas, a.bn);
  if (!encode_weights(h, c.weight, shape.b_cols, a.shard)) return cudaErrorInvalidValue;
  cudaError_t e = cudaSuccess;
  MergeArgs m = {};
  if (pack) {
    const PackArgs p = pack_args(h, c);
    e = launch_dependent(pack_kernel, p, row_blocks(h, c.N), kPackThreads, 0, 1, stream);
    if (e != cudaSuccess) return e;
    a.count = h.count;
    a.targets = Ids{h.target, 4};
    if (!encode(&a.x, h.packed, h.dtype, loss_rows_pad(c.N), h.K, h.pitch, kTileM))
      return cudaErrorInvalidValue;
    m.count = h.count;
    m.row_of = h.row_of;
  } else {
    a.targets = c.targets;
    if (!encode(&a.x, c.hidden, h.dtype, c.N, h.K, c.ld, shape.a_rows))
      return cudaErrorInvalidValue;
  }
  e = launch<kLoss>(h, shape, a, div_up(h.K, kBlockK), stream);
  if (e != cudaSuccess) return e;
  m.partial = h.partial;
  m.tiles = a.tiles;
  m.hit = h.hit;
  m.targets = a.targets;
  m.vocab = h.vocab;
  m.loss = c.loss;
  m.lse = c.lse_out;
  return launch_dependent(merge_kernel, m, (unsigned)c.N, kMergeThreads, 0, 1, stream);
}

cudaError_t loss_grad(const hg_vocab& h, const LossCall& c, cudaStream_t stream) {
  const long long pad = loss_rows_pad(c.N > 0 ? c.N : 1);
  PackArgs p = pack_args(h, c);
  p.grad = 1;
  p.headroom = h.dtype == HG_FP16 ? 16384.f : 1.f;  // small terms stay off fp16's floor
  p.split = c.N <= kSplitRows;
  cudaError_t e =
      launch_dependent(pack_kernel, p, row_blocks(h, c.N), kPackThreads, 0, 1, stream);
  if (e != cudaSuccess) return e;

  // One argument block per product; only the piece changes between launches.
  GemmArgs prob = gemm_args(h, c);
  prob.count = h.count;
  prob.targets = Ids{h.target, 4};
  prob.wc = h.piece_cols;
  prob.split = p.split;
  GemmArgs dx = prob, dw = prob;
  const uint64_t prob_cols = (uint64_t)h.tp * h.piece_cols;
  const int first = h.piece_cols < h.W ? h.piece_cols : h.W;
  prob.bn = tile_width(h, c.N, first, 64);
  const Shape prob_shape = row_shape(c.N, prob.bn);
  const Shape dx_shape = row_shape(p.split ? kSplitRows + c.N : c.N, kTileN);
  // Of few rows a tile is a K block or two and a store, and the exchange between the
  // CTAs of a pair costs more than sharing B saves: 16 rows at V=163840, K=7168
  // took 382 us by single CTAs, against 480 us.
  Shape dw_shape = row_shape(c.N, kTileN);
  dw_shape.a_rows = kTileM;
  prob.idesc = instruction(h.dtype, false, false, kTileM * prob_shape.ctas, prob.bn);
  if (!encode_weights(h, c.weight, prob_shape.b_cols, prob.shard) ||
      !encode(&prob.x, h.packed, h.dtype, pad, h.K, h.pitch, prob_shape.a_rows) ||
      !encode(&prob.out, h.prob, h.dtype, pad, prob_cols, prob_cols, 32))
    return cudaErrorInvalidValue;
  int splits = 1;
  if (c.grad_hidden) {
    dx.idesc = instruction(h.dtype, false, true, kTileM * dx_shape.ctas, kTileN);
    dx.tp = real_shards(h);  // 0 * NaN of a padding shard must not be summed
    splits = dx_splits(h, c.N);
    dx.used_rows = dx_shape.a_rows;
    dx.accum_rows = slab_rows(c.N);
    if (!encode_weights(h, c.weight, kBlockK, dx.shard) ||
        !encode(&dx.p, h.prob, h.dtype, pad, prob_cols, prob_cols, dx_shape.a_rows) ||
        !encode(&dx.out, h.accum, HG_FP32, (uint64_t)splits * dx.accum_rows, h.K, h.pitch, 32))
      return cudaErrorInvalidValue;
  }
  if (c.grad_weight) {
    dw.idesc = instruction(h.dtype, true, true, kTileM * dw_shape.ctas, kTileN);
    dw.add = c.accumulate;
    for (int r = 0; r < h.tp; ++r)
      if (!encode(&dw.shard[r], c.grad_weight[r], h.dtype, h.W, h.K, h.K, 32))
        return cudaErrorInvalidValue;
    if (!encode(&dw.p, h.prob, h.dtype, pad, prob_cols, prob_cols, kBlockK) ||
        !encode(&dw.x, h.packed, h.dtype, pad, h.K, h.pitch, kBlockK))
      return cudaErrorInvalidValue;
  }
  const long long dw_blocks = div_up(p.split ? 2 * kSplitRows : c.N, kBlockK);
  for (int c0 = 0; c0 < h.W; c0 += h.piece_cols) {
    const int left = h.W - c0;
    prob.c0 = dx.c0 = dw.c0 = c0;
    prob.wcols = dx.wcols = dw.wcols = left < h.piece_cols ? left : h.piece_cols;
    e = launch<kProb>(h, prob_shape, prob, div_up(h.K, kBlockK), stream);
    if (e != cudaSuccess) return e;
    int dx_units = 0;
    long long dx_blocks = 0;  // K blocks of a part
    if (c.grad_hidden) {
      dx.add = c0 > 0;
      // A short last piece may have fewer K blocks than parts: each part has one.
      const int kb = dx.tp * (int)div_up(dx.wcols, kBlockK);
      dx.splits = splits < kb ? splits : kb;
      dx_blocks = div_up(kb, dx.splits);
      if (c.grad_weight && c.N > 0) dx_units = both_units(h, dx, dw, c.N, dx_shape.ctas);
    }
    if (dx_units) {
      BothArgs both;
      stage_layout<kDx>(dx_shape, dx);
      stage_layout<kDw>(dw_shape, dw);
      both.dx = dx;
      both.dw = dw;
      both.dx_units = dx_units;
      e = dx_blocks > kSegment || dw_blocks > kSegment
              ? launch_both_cut<true>(h, dx_shape.ctas, both, stream)
              : launch_both_cut<false>(h, dx_shape.ctas, both, stream);
    } else {
      if (c.grad_hidden) e = launch<kDx>(h, dx_shape, dx, dx_blocks, stream);
      if (e == cudaSuccess && c.grad_weight) e = launch<kDw>(h, dw_shape, dw, dw_blocks, stream);
    }
    if (e != cudaSuccess) return e;
  }
  if (!c.grad_hidden || c.N == 0) return cudaSuccess;
  FinishArgs f = {};
  f.accum = h.accum;
  f.splits = splits;
  f.split = p.split;
  f.accum_rows = dx.accum_rows;
  f.K = h.K;
  f.pitch = h.pitch;
  f.count = h.count;
  f.row_of = h.row_of;
  f.unscale = h.unscale;
  f.grad = c.grad_hidden;
  f.ld = c.ld_grad;
  const long long blocks = div_up((long long)c.N * (h.K / 4), 256);
  const unsigned grid = (unsigned)(blocks < 8ll * h.sms ? blocks : 8ll * h.sms);
  return h.dtype == HG_BF16
             ? launch_dependent(finish_kernel<__nv_bfloat16>, f, grid, 256, 0, 1, stream)
             : launch_dependent(finish_kernel<__half>, f, grid, 256, 0, 1, stream);
}

}  // namespace vocab
}  // namespace hg
