// Dense attention of packed query rows over paged or contiguous caches, on the
// 5th-generation tensor cores: whole prompts and chunks of them (causal), single tokens,
// and the rows of all sequences behind a shared prefix (not causal).
//
// For token row n of sequence b (token number p) and head h of kv group g:
//   o = sum_j e^(s_j - m) v_j / l,  s_j = q.k_j * scale over the keys j <= p (causal) or all
//   keys of the sequence, with the running maximum m and sum l in fp32 over one pass.
//
// Design:
//  * The G query heads of a kv group are rows of the same tile: row r of a 128-row tile is
//    token r / G, head r % G, which is how one TMA box {64, G, 128/G} of q [N, Hq, d] lands
//    in shared memory. A unit is two such tiles (256/G tokens) of one kv head, so a key tile
//    is read once for 256 rows, and a single token still fills G rows. A unit of up to 128
//    rows gives both tiles of tensor memory the same rows and its steps in turn; their
//    results are joined when they are written.
//  * A step is 128 keys (two blocks of the cache). The loader warp copies K and V of a step
//    into a ring of 32 KB stages; one issuing thread runs S = Q K^T into 128 columns of tensor
//    memory and O += P V from them; four softmax warps per tile, a thread a row, turn S into P,
//    written as bf16 over S and handed over by quarters. The two tiles take turns: while one is
//    in its softmax, the other has the tensor cores. P V (j) and S (j + 1) of a tile are issued
//    by the same thread, in order, so S needs no second buffer and the arrival of S (j + 1) says
//    that P V (j) is done.
//    (At d = 64 there is room for a third buffer of scores, and S runs further ahead.)
//  * The running maximum only moves when it grows by more than 8 (log2): O is then rescaled
//    in tensor memory. l sums the fp32 weights, P <= 2^8. P meets V as one bf16 part, off by
//    2^-8 of itself at most (as the output's own rounding is; where one key dominates a row, by
//    that of the result), or as two, in both halves of S's columns, off by 2^-15. Two are half as
//    many products again: a prompt of 32K takes 10.4 ms instead of 7.8, 200 rows behind three
//    prefixes of 64K 460 us instead of 370, but one row each over 32K keys 148 instead of 136,
//    since there the keys' arrival takes the time. V stays bf16, so no value range is lost.
//  * Four more warps write a unit's result from tensor memory while the softmax warps are in
//    the next unit's first steps (with the softmax warps writing it, 10,000 cycles a unit).
//  * Few rows over many keys: a plan (a kernel of one block or, for few tiles, each block for
//    itself) cuts units into splits of the key axis, until the SMs are filled; each writes its
//    O, m and l in fp32 and the merge kernel joins them. Units are handed out longest first.
//    What a row's own tokens gave is joined by whoever writes the row.
//  * Rows of V behind a sequence's end are whatever the page held before: a patch warp
//    zeroes them in shared memory in the step that has the end (0 * NaN is NaN), before the
//    step is handed to the tensor cores. K there may be anything: its scores are replaced.
// Tensor memory: O of tile t at d t, the scores' buffers (then P) of 128 columns from 2 d. Every
// wait is bounded; on a timeout the kernel reports BSA_DEV_TIMEOUT, drains and returns.
#include <algorithm>

#include "tcgen05.cuh"
#include "tokens_common.cuh"
#include "tokens_internal.h"

namespace bsa {
namespace {

constexpr int kThreads = 512;          // warps 0-3 / 4-7: softmax of tile 0 / 1; then one each:
constexpr int kSoftmaxWarps = 8, kWarpLoad = 8, kWarpMma = 9, kWarpPatch = 10, kWarpQ = 11;
constexpr int kWarpOut = 12;           // and 12-15: results
constexpr int kPolyOf = 8;             // see Cfg
// registers a thread of the softmax warps, of the warps 8-11 and of 12-15
constexpr int kRegsSoftmax = 192, kRegsOther = 56, kRegsOut = 72;
static_assert(2 * kRegsSoftmax + kRegsOther + kRegsOut <= 65536 / 128, "registers of the launch");
constexpr uint32_t kTmemCols = 512;
constexpr int kStep = 128;             // keys a step
constexpr int kMaxStages = 11;
constexpr int kRounds = 2;              // units a block may have where it plans for itself
constexpr int kPlanThreads = 1024;
constexpr int kMergeThreads = 256, kMergeBlocks = 4;    // blocks an SM
constexpr int kBuckets = 512, kPlanTiles = 1024, kPlanSeqs = 1024;
// in quarters of a step of two tiles (750 cycles)
constexpr float kUnitCost = 8.f, kMergeCost = 12.f, kRowsCost = 10.f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;            // 64-dim slabs (rows of 128 B)
  static constexpr int kSlab = 128 * 128;           // 128 rows of one slab
  static constexpr int kTile = kHalves * kSlab;     // 128 rows x D: a Q tile, or K or V of a step
  // One more where no unit has two tiles: it takes the place of the second Q tile, before the
  // others. A pair of steps of one tile uses four stages, so that with five the next keys come
  // late: 2,250 cycles a step at d = 128 (keys in L2), 1,650 with six; from HBM 2,970 and 2,760
  // (the loop of steps alone; see step_cost for whole calls).
  static constexpr int kStages = D == 128 ? 5 : 10;
  // Of every kPolyOf pairs of a row's scores, kPoly take their exponentials by polynomial. At
  // d = 128 more cost power, which is the limit there; at d = 64 the loop of steps of two tiles
  // takes 2,650 cycles a step with none, 2,730 with 1, 2,610 with 2 and 3,150 with 3.
  static constexpr int kPoly = D == 128 ? 1 : 2;
  // Buffers of scores: one a tile, or three that the tiles take in turn (see the issuer).
  static constexpr int kRing = D == 128 ? 2 : 3;
  static constexpr int kScores = 2 * D;             // their first column in tensor memory
  static constexpr int kOffKV = 2 * kTile;
  static constexpr int kOffBar = kOffKV + kStages * kTile;
};

struct Unit {
  int u, b, g, row0, ntok, pos0, len, step0, step1, split, nsplit, bad;
  int more;                            // stages besides kStages, the same for all units
};

struct Bars {
  uint64_t info_full[2], info_empty[2];
  uint64_t q_full[2], q_empty[2];
  uint64_t kv_full[kMaxStages], kv_empty[kMaxStages], kv_raw[kMaxStages];
  uint64_t s_full[2][3];               // [tile][buffer]
  uint64_t pv_done[2], o_full[2];      // pv_done: with three buffers
  uint64_t p_ready[3][4];              // [buffer][quarter of the step's keys]
  uint64_t ml_full[2], o_empty[2];     // a unit's (m, l) is written; its O and (m, l) are read
  uint64_t mma_done;
  float2 ml[2][128];                   // [tile][row]
  Unit info[2];
  int4 own[2 * kRounds];               // the block's entries, where it plans for itself
  uint32_t tmem_base;
  int abort_flag;
};

template <int D>
constexpr int smem_bytes() {
  return Cfg<D>::kOffBar + static_cast<int>(sizeof(Bars));
}
static_assert(smem_bytes<128>() <= 232448 && smem_bytes<64>() <= 232448, "shared memory");

BSA_DEVFN bool aborted(Bars* b) { return *reinterpret_cast<volatile int*>(&b->abort_flag) != 0; }
BSA_DEVFN void set_abort(Bars* b, int32_t* status) {
  *reinterpret_cast<volatile int*>(&b->abort_flag) = 1;
  report(status, BSA_DEV_TIMEOUT);
}

BSA_DEVFN bool warp_wait_sleep(uint64_t* bar, uint32_t parity) {
  bool ok = true;
  if ((threadIdx.x & 31) == 0) ok = mbar_wait_sleep(bar, parity);
  return __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
}

// Every lane polls (one broadcast read a try): no shuffle behind the wait. Warp-uniform.
BSA_DEVFN bool warp_wait_all(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity)) != 0;
}

// The same for waits that are long: the warp sleeps instead of polling.
BSA_DEVFN bool warp_sleep_all(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait_sleep(bar, parity)) != 0;
}

BSA_DEVFN float max3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}

// 2^x on the FMA pipes, two lanes at once, for x <= 8: x = n + f with n the nearest integer
// (adding 1.5 * 2^23 rounds it into the low mantissa bits), 2^f by a quartic of least relative
// error on [-1/2, 1/2] among those that are exactly 1 at 0 (Remez exchange, exp2_poly_fit.py:
// 2.8e-6, below 2^-18), n added to the exponent field.
// x is clamped at -127, where that gives exactly 0: masked scores add nothing.
BSA_DEVFN float2 exp2_poly(float2 x) {
  constexpr float kC1 = 0.6931241750717163f, kC2 = 0.24024099111557007f;
  constexpr float kC3 = 0.055906426161527634f, kC4 = 0.009582852944731712f;
  constexpr float kShift = 12582912.0f;  // 1.5 * 2^23
  x.x = fmaxf(x.x, -127.0f);
  x.y = fmaxf(x.y, -127.0f);
  const float2 r = __fadd2_rn(x, make_float2(kShift, kShift));
  const float2 nn = __ffma2_rn(r, make_float2(-1.0f, -1.0f), make_float2(kShift, kShift));  // -n
  const float2 f = __fadd2_rn(x, nn);
  float2 p = __ffma2_rn(make_float2(kC4, kC4), f, make_float2(kC3, kC3));
  p = __ffma2_rn(p, f, make_float2(kC2, kC2));
  p = __ffma2_rn(p, f, make_float2(kC1, kC1));
  p = __ffma2_rn(p, f, make_float2(1.0f, 1.0f));
  return make_float2(__uint_as_float(__float_as_uint(p.x) + (__float_as_uint(r.x) << 23)),
                     __uint_as_float(__float_as_uint(p.y) + (__float_as_uint(r.y) << 23)));
}

// Row (of width d) of the first token of block blk of (b, g), or -1 where it is bad.
BSA_DEVFN int64_t block_row(const CacheView& c, int b, int g, int blk, int len, int d) {
  int64_t phys = blk;
  if (c.page_table != nullptr) {
    phys = c.page_table[static_cast<int64_t>(b) * c.pt_stride + blk];
    if (phys < 0 || phys >= c.num_pages) return -1;
  }
  const int64_t off = static_cast<int64_t>(b) * c.seq_stride + phys * c.block_stride +
                      static_cast<int64_t>(g) * c.head_stride;
  if (off < 0 || off + static_cast<int64_t>(min(kBlock, len - blk * kBlock)) * d > c.extent)
    return -1;
  return off / d;
}

// ------------------------------------------------------------------------------- plan
struct Tile {
  int b, row0, ntok, pos0, len, steps;
};

BSA_DEVFN int seq_first(const PackedArgs& a, int b) {
  return a.cu != nullptr ? a.cu[b] : b * (a.N / a.B);
}
BSA_DEVFN int seq_len(const PackedArgs& a, int b) {
  return a.seq_lens != nullptr ? max(0, min(a.seq_lens[b], a.T)) : a.T;
}

// What a step of a unit costs. Calls of 148 heads of 256 rows over 32K keys take 3,350 cycles a
// step of two tiles, starts and ends included (d = 64: 2,900), of 128 rows 1,790 where the keys are
// in L2 and 2,620 from HBM, which is where few rows mostly find theirs (d = 64: 1,520 and 1,550).
// With P in two parts 4,500, 2,440 and 2,450 (3,770, 1,930 and 1,930): few rows have one tile.
BSA_DEVFN int step_cost(int d, bool two) { return two ? 4 : d == 128 ? 3 : 2; }

// Without splits the SMs are evenly loaded where there are several units for each SM and the
// costliest (started first) is no more than an SM's share. Else the cost that a unit may have is
// searched among 32 candidates. The time with one is the costliest unit's where every unit has an
// SM of its own, and otherwise the units in whole rounds of the SMs, and no less than an SM's
// share of all costs and a fifth of the costliest (SMs are not equally fast). A unit costs
// kUnitCost besides its steps, a merge kMergeCost and 1 for each kRowsCost partial rows of an SM,
// which are written and read again (with 20 for 10: 20 chunks of up to 241 rows over 9K keys,
// 32/4 heads, 309 us for 257; with a third for a fifth: 200 rows behind three prefixes 390 for 359).
BSA_DEVFN int candidate(int i, float share) {
  return i == 0 ? 1 << 30 : max(12, static_cast<int>(share * (0.1f + 0.06f * i)) + 1);
}
// Pieces that a tile of cost c is cut into where a piece may cost 1 / per, and what one costs. In
// floats, which are a few instructions each: a block that plans for itself waits for its plan.
BSA_DEVFN int pieces(const PackedArgs& a, int c, float per) {
  return max(1, min(a.smax, __float2int_ru(c * per - 0.001f)));
}
BSA_DEVFN int piece_cost(int c, int k) { return __float2int_ru(__fdividef(c, k) - 0.001f); }
// What a tile of cost c and ntok tokens adds under the candidate: units and the rows (of one kv
// head) that go through the merge; the costliest piece.
BSA_DEVFN void add_tile(const PackedArgs& a, int c, int ntok, float per, int& units, int& piece, int& parts) {
  const int k = pieces(a, c, per);
  units += k;
  piece = max(piece, piece_cost(c, k));
  if (k > 1) parts += k * ntok * a.G;
}
BSA_DEVFN float plan_time(const PackedArgs& a, float share, int units, int piece, int parts) {
  const float unit = piece + kUnitCost, sms = a.num_sms, per_sm = __fdividef(1.f, sms);
  const float merge = (parts > 0 ? kMergeCost : 0.f) + parts * a.Hkv * per_sm * (1.f / kRowsCost);
  // an SM's share of all costs; its share of the units in whole rounds
  const float even = share + units * kUnitCost * per_sm;
  const float rounds = __fdividef(even * sms, max(units, 1)) * ceilf(units * per_sm - 0.001f);
  return merge + (units <= a.num_sms ? unit : max(rounds, even + 0.2f * unit));
}

// One block: lists the units (tile, split of its keys) of one kv head, longest first.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PackedArgs a) {
  __shared__ int warp_sum[32];
  __shared__ int carry, bad, longest, wide;
  __shared__ unsigned long long work, best;   // best: (time, candidate)
  __shared__ int bucket[kBuckets], costs[kPlanTiles];
  // first row, length and first tile of each sequence, for up to kPlanSeqs of them
  __shared__ int s_first[kPlanSeqs + 1], s_len[kPlanSeqs], s_offs[kPlanSeqs];
  grid_launch_dependents();            // the attention kernel sets up meanwhile, and waits for this one
  grid_dependency_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = packed_unit_tokens(a.G), half = per / 2;
  const bool small = a.B <= kPlanSeqs;
  if (tid == 0) {
    carry = 0;
    bad = 0;
    longest = 0;
    wide = 0;
    work = 0;
    best = ~0ull;
  }
  for (int i = tid; i < kBuckets; i += kPlanThreads) bucket[i] = 0;
  __syncthreads();
  // tiles of each sequence, summed up
  for (int base = 0; base < a.B; base += kPlanThreads) {
    const int b = base + tid;
    int tiles = 0;
    if (b < a.B) {
      const int first = seq_first(a, b), last = seq_first(a, b + 1);
      const int len = a.seq_lens != nullptr ? a.seq_lens[b] : a.T;
      if (first < 0 || last < first || last > a.N || (b == 0 && first != 0)) {
        bad = 1;
      } else {
        tiles = (last - first + per - 1) / per;
        if (len < 0 || len > a.T || (a.causal && len < last - first))
          report(a.status, BSA_DEV_BAD_LENGTH);
      }
      if (small) {
        s_first[b] = first;
        if (b == a.B - 1) s_first[a.B] = last;
        s_len[b] = max(0, min(len, a.T));
      }
    }
    int x = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    int before = carry;
    for (int w = 0; w < warp; ++w) before += warp_sum[w];
    if (b < a.B) {
      if (small) s_offs[b] = before + x - tiles; else a.offs[b] = before + x - tiles;
    }
    __syncthreads();
    if (tid == kPlanThreads - 1) carry = before + x;
    __syncthreads();
  }
  const bool refuse = bad != 0;
  const int ntiles = refuse ? 0 : carry;
  if (refuse && tid == 0) report(a.status, BSA_DEV_BAD_LENGTH);
  // tile t of all sequences' tiles, in order
  auto tile_of = [&](int t) {
    int lo = 0, hi = a.B - 1;          // the last b whose first tile is at most t
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((small ? s_offs[mid] : a.offs[mid]) <= t) lo = mid; else hi = mid - 1;
    }
    const int first = small ? s_first[lo] : seq_first(a, lo);
    const int count = (small ? s_first[lo + 1] : seq_first(a, lo + 1)) - first;
    const int i = (t - (small ? s_offs[lo] : a.offs[lo])) * per;
    Tile r;
    r.b = lo;
    r.row0 = first + i;
    r.ntok = min(per, count - i);
    r.len = small ? s_len[lo] : seq_len(a, lo);
    r.pos0 = r.len - count + i;
    const int end = a.causal ? max(0, min(r.len, r.pos0 + r.ntok)) : r.len;
    r.steps = (end + kStep - 1) / kStep;
    return r;
  };
  Tile own;                            // this thread's first tile: one is all there is, mostly
  if (tid < ntiles) own = tile_of(tid);
  auto tile = [&](int t) { return t == tid ? own : tile_of(t); };
  // cost of all tiles and of the costliest
  auto cost_of = [&](const Tile& x) { return step_cost(a.d, x.ntok > half) * x.steps; };
  unsigned long long sum = 0;
  int top = 0;
  for (int t = tid; t < ntiles; t += kPlanThreads) {
    const int c = cost_of(tile(t));
    if (t < kPlanTiles) costs[t] = min(c, 0xfffff) | (tile(t).ntok << 20);
    if (tile(t).ntok > half) wide = 1;
    sum += c;
    top = max(top, c);
  }
  top = __reduce_max_sync(0xffffffffu, top);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0 && sum > 0) {
    atomicAdd(&work, sum);
    atomicMax(&longest, top);
  }
  __syncthreads();
  const float share = static_cast<float>(work) * a.Hkv / a.num_sms;
  int limit = 1 << 30;
  if (a.smax > 1 && ntiles <= kPlanTiles &&
      !(static_cast<float>(longest) <= share && static_cast<long long>(ntiles) * a.Hkv >= 3ll * a.num_sms)) {
    const int cand = candidate(warp, share);    // a warp for each
    const float per_cost = __fdividef(1.f, cand);
    int units = 0, piece = 0, parts = 0;
    for (int t = lane; t < ntiles; t += 32)
      add_tile(a, costs[t] & 0xfffff, costs[t] >> 20, per_cost, units, piece, parts);
    units = __reduce_add_sync(0xffffffffu, units) * a.Hkv;
    parts = __reduce_add_sync(0xffffffffu, parts);
    piece = __reduce_max_sync(0xffffffffu, piece);
    const float time = plan_time(a, share, units, piece, parts);
    if (lane == 0) atomicMin(&best, (static_cast<unsigned long long>(__float_as_uint(time)) << 32) |
                                        static_cast<unsigned>(cand));
    __syncthreads();
    limit = static_cast<int>(best & 0x7fffffffull);
  }
  const float per_limit = __fdividef(1.f, limit);
  const int shift = max(0, 32 - __clz(longest) - 9);
  auto splits_of = [&](const Tile& x) {
    return max(1, min(x.steps, pieces(a, cost_of(x), per_limit)));
  };
  auto bucket_of = [&](const Tile& x, int n) {
    return kBuckets - 1 - min(kBuckets - 1, ((cost_of(x) + n - 1) / n) >> shift);
  };
  bool any = false;
  for (int t = tid; t < ntiles; t += kPlanThreads) {
    const Tile x = tile(t);
    const int n = splits_of(x);
    any |= n > 1;
    atomicAdd(&bucket[bucket_of(x, n)], n);
  }
  any = __syncthreads_or(any);
  // exclusive sums of the buckets (kBuckets <= kPlanThreads)
  int mine = tid < kBuckets ? bucket[tid] : 0, x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < warp; ++w) before += warp_sum[w];
  if (tid < kBuckets) bucket[tid] = before + x - mine;
  if (tid == kPlanThreads - 1) {
    a.head[0] = before + x;
    a.head[1] = 0;
    a.head[2] = any ? 1 : 0;
    a.head[3] = wide ? 0 : 1;
  }
  __syncthreads();
  for (int t = tid; t < ntiles; t += kPlanThreads) {
    const Tile y = tile(t);
    const int n = splits_of(y);
    const int at = atomicAdd(&bucket[bucket_of(y, n)], n);
    for (int s = 0; s < n; ++s) {
      const int s0 = static_cast<int>(static_cast<int64_t>(y.steps) * s / n);
      const int s1 = static_cast<int>(static_cast<int64_t>(y.steps) * (s + 1) / n);
      a.entries[2 * (at + s)] = make_int4(y.b, y.row0, y.ntok, y.pos0);
      a.entries[2 * (at + s) + 1] = make_int4(y.len, s0, s1, s | (n << 16));
    }
    if (any)
      for (int i = 0; i < y.ntok; ++i) a.row_splits[y.row0 + i] = n;
  }
  if (any) {   // rows of no sequence
    const int end = refuse ? 0 : seq_first(a, a.B);
    for (int n = end + tid; n < a.N; n += kPlanThreads) a.row_splits[n] = 0;
  }
}

// the unit that a block which plans for itself takes in round k
BSA_DEVFN int unit_of_round(int k) {
  return k * gridDim.x + (k & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

// The plan of few tiles (at most 32 of as many sequences, and no more for all kv heads than SMs)
// by every block's loader warp for itself, a lane a sequence and then a tile: at most kRounds units
// a block, the first round of them from the costliest down, the second back from the last block to
// the first. The block's entries go to own[], the number of all units is returned. The block of a
// tile's first unit writes its rows' number of splits, block 0 those of rows of no sequence.
// One row over ten keys takes 9.3 us instead of 13.0 with the plan kernel, 32 rows behind 32K keys
// 48 instead of 55, 693 rows over 3K keys (16/8 heads, d = 64) 43 and 47; where units that blocks
// take when they are free would be better it loses (27 rows each of 16 sequences over 12K keys,
// 64/4 heads: 122 and 114, before rows that do not exist cost nothing). More rounds: the same.
BSA_DEVFN int plan_in_warp(const PackedArgs& a, int4* own, int& more) {
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  const int per = packed_unit_tokens(a.G), half = per / 2;
  const bool first_block = blockIdx.x == 0;
  auto sum_up = [&](int x) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kAll, x, o);
      if (lane >= o) x += y;
    }
    return x;
  };
  // how many lanes' sums are at most t, which is less than the last
  auto find = [&](int sums, int t) {
    int lo = 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      if (__shfl_sync(kAll, sums, lo + o - 1) <= t) lo += o;
    return lo;
  };
  int first = 0, last = 0, len = 0;
  bool bad = false, wrong = false;
  if (lane < a.B) {
    first = seq_first(a, lane);
    last = seq_first(a, lane + 1);
    len = a.seq_lens != nullptr ? a.seq_lens[lane] : a.T;
    bad = first < 0 || last < first || last > a.N || (lane == 0 && first != 0);
    wrong = bad || len < 0 || len > a.T || (a.causal && len < last - first);
    len = max(0, min(len, a.T));
  }
  if (wrong && first_block) report(a.status, BSA_DEV_BAD_LENGTH);
  if (__any_sync(kAll, bad)) first = last = 0;
  const int end = __shfl_sync(kAll, last, a.B - 1);
  const int tiles = (last - first + per - 1) / per, sums = sum_up(tiles);
  const int ntiles = __shfl_sync(kAll, sums, 31);
  int n = 0, c = 0;
  Tile x = {};
  {
    const int b = find(sums, lane);    // lanes from ntiles on: any
    const int row = __shfl_sync(kAll, first, b), count = __shfl_sync(kAll, last, b) - row;
    const int i = (lane - __shfl_sync(kAll, sums - tiles, b)) * per;
    const int length = __shfl_sync(kAll, len, b);
    if (lane < ntiles) {
      const int ntok = min(per, count - i), pos0 = length - count + i;
      const int keys = a.causal ? max(0, min(length, pos0 + ntok)) : length;
      x = {b, row + i, ntok, pos0, length, (keys + kStep - 1) / kStep};
      c = step_cost(a.d, ntok > half) * x.steps;
      n = 1;
    }
  }
  if (a.smax > 1) {
    const float share = static_cast<float>(__reduce_add_sync(kAll, static_cast<unsigned>(c))) * a.Hkv / a.num_sms;
    const float cand = __fdividef(1.f, candidate(lane, share));
    int units = 0, piece = 0, parts = 0;
#pragma unroll 1
    for (int t = 0; t < ntiles; ++t)
      add_tile(a, __shfl_sync(kAll, c, t), __shfl_sync(kAll, x.ntok, t), cand, units, piece, parts);
    units *= a.Hkv;
    const float time = units <= kRounds * a.num_sms ? plan_time(a, share, units, piece, parts) : INFINITY;
    const unsigned best = __reduce_min_sync(kAll, __float_as_uint(time));
    const float limit = __shfl_sync(kAll, cand, __ffs(__ballot_sync(kAll, __float_as_uint(time) == best)) - 1);
    if (lane < ntiles) n = max(1, min(x.steps, pieces(a, c, limit)));
  }
  // units of costlier pieces, and of equal ones before this one, come first; without splits all
  // units run at once, and their order is nothing
  int at = lane, entries = ntiles;
  if (a.smax > 1) {
    const int piece = n > 0 ? piece_cost(c, n) : -1;
    at = entries = 0;
#pragma unroll 1
    for (int t = 0; t < ntiles; ++t) {
      const int p = __shfl_sync(kAll, piece, t), m = __shfl_sync(kAll, n, t);
      if (p > piece || (p == piece && t < lane)) at += m;
      entries += m;
    }
  }
  const bool any = __any_sync(kAll, n > 1);
  more = __any_sync(kAll, x.ntok > half) ? 0 : 1;
  if (first_block) {
    if (any)
      for (int r = end + lane; r < a.N; r += 32) a.row_splits[r] = 0;
    if (lane == 0) a.head[2] = any ? 1 : 0;
  }
  const int units = entries * a.Hkv;
#pragma unroll 1
  for (int k = 0; k < kRounds; ++k) {
    const int u = unit_of_round(k);
    if (u >= units) break;
    const int e = u / a.Hkv;
    const bool mine = n > 0 && at <= e && e < at + n;
    if (mine) {
      const int split = e - at;
      own[2 * k] = make_int4(x.b, x.row0, x.ntok, x.pos0);
      own[2 * k + 1] = make_int4(x.len, x.steps * split / n, x.steps * (split + 1) / n, split | (n << 16));
      if (any && split == 0 && u % a.Hkv == 0)
        for (int i = 0; i < x.ntok; ++i) a.row_splits[x.row0 + i] = n;
    }
  }
  __syncwarp();
  return units;
}

// ------------------------------------------------------------------------------- results
// 32 bytes, in one store where `wide` (aligned to 32): lanes that write rows far apart fill whole
// sectors.
BSA_DEVFN void store32(void* p, const uint32_t (&v)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

// Four warps write the units' results while the softmax warps are at the next unit: thread r of
// them has row r of a tile, 16 columns at a time.
template <int D>
BSA_DEVFN void out_role(const PackedArgs& a, Bars* bars, uint32_t tmem) {
  const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3;
  const int row = quarter * 32 + lane, half_tok = 128 >> a.lgG;
  const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
  const bool wide = ((reinterpret_cast<uintptr_t>(a.o) | reinterpret_cast<uintptr_t>(a.o_f32)) & 31) == 0;
  uint32_t un = 0, ml_phase = 0, o_phase = 0;      // o_phase: a bit for each tile
  bool ok = true;
  while (ok) {
    const int slot = un & 1;
    if (!warp_sleep_all(&bars->info_full[slot], (un >> 1) & 1)) break;
    ++un;
    const volatile Unit& U = bars->info[slot];
    if (U.u < 0 || aborted(bars)) return;
    const int steps = U.step1 - U.step0;
    const bool empty = steps <= 0, one = U.ntok <= half_tok;
    // One tile of rows: its steps were taken by both tiles of tensor memory, or by the first.
    const bool two = one && steps > 1;
    for (int t = 0; t < (one ? 1 : 2) && ok; ++t) {
      const int tok = t * half_tok + (row >> a.lgG);
      const bool live = tok < U.ntok, part = U.nsplit > 1;
      const int64_t at = (static_cast<int64_t>(U.row0) + tok) * a.Hq + U.g * a.G + (row & (a.G - 1));
      const bool join = live && !part && a.lse_own != nullptr;
      float w = -INFINITY;                     // o_own is on its way while the unit runs
      if (join) {
        w = a.lse_own[at] * kLog2e;
        for (int c = 0; c < D; c += 32) prefetch_l1(a.o_own + at * D + c);
      }
      float m = -INFINITY, L = 0.f, f0 = 1.0f, f1 = 0.0f;
      if (!empty) {
        ok = warp_sleep_all(&bars->ml_full[t], ml_phase) && warp_sleep_all(&bars->o_full[t], (o_phase >> t) & 1);
        o_phase ^= 1u << t;
        if (ok && one) ok = warp_sleep_all(&bars->ml_full[1], ml_phase);
        if (ok && two) {
          ok = warp_sleep_all(&bars->o_full[1], o_phase >> 1);
          o_phase ^= 2u;
        }
        if (!ok) break;
        tc::fence_after_sync();
        const float2 x = bars->ml[t][row];
        m = x.x;
        L = x.y;
        if (two) {
          const float2 x1 = bars->ml[1][row];
          m = fmaxf(x.x, x1.x);
          const float base = m == -INFINITY ? 0.f : m;
          f0 = ex2(x.x - base);
          f1 = ex2(x1.x - base);
          L = x.y * f0 + x1.y * f1;
        }
      }
      float own = 0.f;                         // weight of o_own, which is normalised
      if (w != -INFINITY) {
        const float top = fmaxf(m, w), base = top == -INFINITY ? 0.f : top;
        const float f = ex2(m - base);
        own = ex2(w - base);
        L = L * f + own;
        f0 *= f;
        f1 *= f;
        m = top;
      }
      if (!part) {
        const float inv = L == 0.f ? 0.f : 1.0f / L;
        f0 *= inv;
        f1 *= inv;
        own *= inv;
      }
      const int64_t pat = static_cast<int64_t>(U.split) * a.N * a.Hq + at;
      float* of = part ? a.part_o + pat * D : a.o_f32 != nullptr ? a.o_f32 + at * D : nullptr;
      if (live) {
        if (part)
          *reinterpret_cast<float2*>(a.part_ml + 2 * pat) = make_float2(m, L);
        else
          a.lse[at] = L == 0.f ? -INFINITY : (m + log2f(L)) * kLn2;
      }
      const uint32_t o_tm = tmem + lane_addr + D * t;
#pragma unroll 1
      for (int c = 0; c < D; c += 16) {
        __syncwarp();
        float v[16];
        if (empty) {
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = 0.f;
        } else {
          uint32_t x[16];
          ld16(o_tm + c, x);
          tc::wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(x[i]) * f0;
          if (two) {
            ld16(o_tm + D + c, x);
            tc::wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = fmaf(__uint_as_float(x[i]), f1, v[i]);
          }
        }
        if (c + 16 == D && !empty) {           // the last of O is read
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&bars->o_empty[t]);
            if (one) mbar_arrive(&bars->o_empty[1]);
          }
        }
        if (w != -INFINITY) {                  // (then live; the weight itself may be NaN)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 y = *reinterpret_cast<const float4*>(a.o_own + at * D + c + 4 * i);
            v[4 * i] = fmaf(y.x, own, v[4 * i]);
            v[4 * i + 1] = fmaf(y.y, own, v[4 * i + 1]);
            v[4 * i + 2] = fmaf(y.z, own, v[4 * i + 2]);
            v[4 * i + 3] = fmaf(y.w, own, v[4 * i + 3]);
          }
        }
        if (live && of != nullptr) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[8 * h + i]);
            store32(of + c + 8 * h, w, wide || part);
          }
        }
        if (live && !part) {
          uint32_t w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
          store32(static_cast<__nv_bfloat16*>(a.o) + at * D + c, w, wide);
        }
      }
    }
    if (!ok) break;
    if (!empty) ml_phase ^= 1;
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->info_empty[slot]);
  }
  if (lane == 0) set_abort(bars, a.status);
}

// ------------------------------------------------------------------------------- main
template <int D, int kParts>
__global__ void __launch_bounds__(kThreads, 1)
    packed_attn_kernel(const PackedArgs a, const __grid_constant__ CUtensorMap tmq,
                       const __grid_constant__ CUtensorMap tmk,
                       const __grid_constant__ CUtensorMap tmv) {
  using C = Cfg<D>;
  constexpr int NS = C::kStages;
  extern __shared__ __align__(1024) unsigned char smem[];   // the swizzle needs 1024-byte tiles
  Bars* bars = reinterpret_cast<Bars*>(smem + C::kOffBar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int half_tok = 128 >> a.lgG;      // tokens of one tile
  if ((smem_u32(smem) & 1023u) != 0) {   // dynamic shared memory starts on a 1 KB boundary
    if (threadIdx.x == 0) report(a.status, BSA_DEV_TIMEOUT);
    return;
  }

  if (threadIdx.x == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bars->info_full[x], 1);
      mbar_init(&bars->info_empty[x], 7 + kSoftmaxWarps);   // with the issuer, patch, Q, out warps
      mbar_init(&bars->q_full[x], 1);
      mbar_init(&bars->q_empty[x], 1);
      for (int b = 0; b < 3; ++b) {
        mbar_init(&bars->s_full[x][b], 1);
        mbar_init(&bars->p_ready[b][x], 4);  // the tile's softmax warps
        mbar_init(&bars->p_ready[b][x + 2], 4);
      }
      mbar_init(&bars->pv_done[x], 1);
      mbar_init(&bars->ml_full[x], 4);
      mbar_init(&bars->o_empty[x], 4);       // the out warps
      mbar_init(&bars->o_full[x], 1);
    }
    mbar_init(&bars->mma_done, 1);
    for (int s = 0; s < NS + 1; ++s) {
      mbar_init(&bars->kv_full[s], 1);
      mbar_init(&bars->kv_empty[s], 1);
      mbar_init(&bars->kv_raw[s], 1);
    }
    bars->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) {
    tc::tmem_alloc(&bars->tmem_base, kTmemCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = bars->tmem_base;
  if (warp == kWarpLoad && lane == 0) {
    prefetch_tensormap(&tmq);
    prefetch_tensormap(&tmk);
    prefetch_tensormap(&tmv);
  }
  grid_launch_dependents();            // the merge kernel may be set up, and waits for this one
  grid_dependency_wait();
  int own_units = 0, more = 0;         // (before the registers are shared out: it takes more)
  if (a.in_block && warp == kWarpLoad) own_units = plan_in_warp(a, bars->own, more);

  if (warp >= kWarpOut) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kRegsOut));
    out_role<D>(a, bars, tmem);
  } else if (warp >= kSoftmaxWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kRegsOther));
    if (warp == kWarpLoad) {
      // ------------------------------------------------------------------ units, K, V
      uint32_t un = 0, st = 0, phase = 1;      // the next stage of the ring
      bool ok = true;
      int next = 0, units = 0;
      while (ok) {
        const int slot = un & 1;
        Unit U = {-1, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
        // the first unit; the others come from the counter
        int u = blockIdx.x;
        if (un > 0) u = a.in_block ? unit_of_round(un)
                                   : gridDim.x + __shfl_sync(0xffffffffu, next, 0);
        // The heads of an entry are neighbours: the longest units of all heads start first
        // (prompts of 2K and 4K: 51 and 132 us, 67 and 155 with one head after the other; prefixes
        // that many rows share: the same within 4%).
        const int e = min(u / a.Hkv, a.max_entries - 1), g = u % a.Hkv;
        const int4* from = a.in_block ? bars->own + 2 * (un % kRounds) : a.entries + 2 * e;
        const int4 e0 = from[0], e1 = from[1];
        if (un == 0) {
          units = a.in_block ? own_units : a.head[0] * a.Hkv;
          if (!a.in_block) more = a.head[3];
        }
        if (un == kRounds && a.in_block) units = 0;
        int rk = -1, rv = -1, nblk = 0;
        // the cache rows of the unit's blocks from `first`, one a lane: -1 behind the end, and
        // for a bad block
        auto look_up = [&](int first) {
          const int blk = first + lane;
          rk = rv = -1;
          bool bad = false;
          if (blk < nblk && blk < 2 * U.step1) {
            rk = static_cast<int>(block_row(a.k, U.b, U.g, blk, U.len, D));
            rv = static_cast<int>(block_row(a.v, U.b, U.g, blk, U.len, D));
            bad = rk < 0 || rv < 0;
            if (bad) rk = rv = -1;
          }
          return __any_sync(0xffffffffu, bad);
        };
        // whether a block blk, blk + 32, .. of the unit is bad. Where every page of the cache lies
        // inside its extent (safe), that is the page's number alone, and the loads of a lane do
        // not wait for each other.
        auto scan = [&](const CacheView& c, int safe, const Unit& U, int blk, int end) {
          bool bad = false;
          if (!safe) {
            for (; blk < end; blk += 32) bad |= block_row(c, U.b, U.g, blk, U.len, D) < 0;
          } else if (c.page_table != nullptr) {
            const int32_t* pt = c.page_table + static_cast<int64_t>(U.b) * c.pt_stride;
            const unsigned pages = c.num_pages;
#pragma unroll 8
            for (; blk < end; blk += 32) bad |= static_cast<unsigned>(pt[blk]) >= pages;
          }
          return bad;
        };
        if (u < units) {
          U = {u, e0.x, g, e0.y, e0.z, e0.w, e1.x, e1.y, e1.z, e1.w & 0xffff, e1.w >> 16, 0, more};
          nblk = (U.len + kBlock - 1) / kBlock;
          // blocks with a bad page or beyond the cache are found before the unit starts
          bool bad = look_up(2 * U.step0);
          const int end = min(2 * U.step1, nblk), from = 2 * U.step0 + 32;
          if (from < end) {
            bool later = scan(a.k, a.k_safe, U, from + lane, end);
            if (a.v.page_table != a.k.page_table || a.v.pt_stride != a.k.pt_stride || !a.k_safe || !a.v_safe ||
                a.v.num_pages < a.k.num_pages)
              later |= scan(a.v, a.v_safe, U, from + lane, end);
            bad |= __any_sync(0xffffffffu, later) != 0;
          }
          U.bad = bad ? 1 : 0;
          if (bad && lane == 0) report(a.status, BSA_DEV_BAD_PAGE);
        }
        if (lane == 0) {
          if (!mbar_wait_sleep(&bars->info_empty[slot], ((un >> 1) & 1) ^ 1)) {
            ok = false;
          } else {
            bars->info[slot] = U;
            mbar_arrive(&bars->info_full[slot]);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        if (!ok || U.u < 0 || aborted(bars)) break;
        ++un;
        if (U.step1 <= U.step0 && lane == 0 && !a.in_block) next = atomicAdd(&a.head[1], 1);
        for (int s0 = U.step0; s0 < U.step1 && ok; s0 += 16) {
          if (s0 > U.step0) look_up(2 * s0);
          const int n_here = min(16, U.step1 - s0);
          for (int q = 0; q < n_here; ++q) {
            const int k0 = __shfl_sync(0xffffffffu, rk, 2 * q), k1 = __shfl_sync(0xffffffffu, rk, 2 * q + 1);
            const int v0 = __shfl_sync(0xffffffffu, rv, 2 * q), v1 = __shfl_sync(0xffffffffu, rv, 2 * q + 1);
            if (lane == 0) {
              // the next unit, shortly before this one's copies end: not earlier, since a unit
              // waits while its block is busy
              if (s0 + q == max(U.step1 - 3, U.step0) && !a.in_block) next = atomicAdd(&a.head[1], 1);
              // a step that has the sequence's end or a bad block goes through the patch warp
              const bool patch = (s0 + q + 1) * kStep > U.len || k0 < 0 || k1 < 0;
              for (int kv = 0; kv < 2 && ok; ++kv) {
                if (!mbar_wait_sleep(&bars->kv_empty[st], phase)) { ok = false; break; }
                uint64_t* bar = kv == 1 && patch ? &bars->kv_raw[st] : &bars->kv_full[st];
                const int r0 = kv ? v0 : k0, r1 = kv ? v1 : k1;
                const uint32_t bytes = ((r0 >= 0) + (r1 >= 0)) * (C::kTile / 2);
                if (bytes > 0) mbar_arrive_expect_tx(bar, bytes); else mbar_arrive(bar);
                unsigned char* to = smem + C::kOffKV + (static_cast<int>(st) - more) * C::kTile;
                const CUtensorMap* map = kv ? &tmv : &tmk;
                for (int x = 0; x < C::kHalves; ++x) {
                  if (r0 >= 0) tma_load_2d(to + x * C::kSlab, map, x * 64, r0, bar);
                  if (r1 >= 0) tma_load_2d(to + x * C::kSlab + 8192, map, x * 64, r1, bar);
                }
                if (++st == NS + more) {
                  st = 0;
                  phase ^= 1;
                }
              }
            }
          }
          ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        }
      }
      if (lane == 0 && !ok) {
        set_abort(bars, a.status);
        // copies in flight must land before the block exits (bounded): the last of each stage
        for (uint32_t k = 0; k < static_cast<uint32_t>(NS + more); ++k)
          mbar_wait_sleep(&bars->kv_full[k], k < st ? phase ^ 1 : phase, 100000000ull);
      }
    } else if (warp == kWarpQ && lane == 0) {
      // ------------------------------------------------------------------------------ Q
      // A warp of its own: Q of the next unit waits for the last scores of this one, and the
      // copies of its keys must not wait with it (bubbles of 14,000 cycles between units).
      uint32_t un = 0, phase = 0;      // phase: a bit for each tile
      bool ok = true;
      while (true) {
        const int slot = un & 1;
        ok = mbar_wait_sleep(&bars->info_full[slot], (un >> 1) & 1);
        if (!ok) break;
        const Unit U = bars->info[slot];
        mbar_arrive(&bars->info_empty[slot]);
        ++un;
        if (U.u < 0 || aborted(bars)) break;
        const int ntiles = U.step1 <= U.step0 ? 0 : U.ntok > half_tok ? 2 : 1;
        for (int t = 0; t < ntiles && ok; ++t) {
          ok = mbar_wait_sleep(&bars->q_empty[t], ((phase >> t) & 1) ^ 1);
          if (!ok) break;
          phase ^= 1u << t;
          mbar_arrive_expect_tx(&bars->q_full[t], C::kTile);
          for (int x = 0; x < C::kHalves; ++x)
            tma_load_3d(smem + t * C::kTile + x * C::kSlab, &tmq, x * 64, U.g * a.G,
                        U.row0 + t * half_tok, &bars->q_full[t]);
        }
        if (!ok) break;
      }
      if (!ok) {
        set_abort(bars, a.status);
        // copies in flight must land before the block exits (bounded): a tile's last copy has
        // landed when q_full has left the phase before this one's
        for (int t = 0; t < 2; ++t)
          mbar_wait_sleep(&bars->q_full[t], ((phase >> t) & 1) ^ 1, 100000000ull);
      }
    } else if (warp == kWarpPatch) {
      // -------------------------- V rows behind the end (or of a bad block) become zero
      uint32_t un = 0, kc = 0, raw_phase = 0;
      while (true) {
        const int slot = un & 1;
        if (!warp_wait_sleep(&bars->info_full[slot], (un >> 1) & 1)) {
          if (lane == 0) set_abort(bars, a.status);
          break;
        }
        const Unit U = bars->info[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->info_empty[slot]);
        ++un;
        if (U.u < 0 || aborted(bars)) break;
        const int n = U.step1 - U.step0;
        // without bad blocks only the last step can have the end
        bool ok = true;
        for (int j = U.bad ? 0 : max(0, n - 1); j < n && ok; ++j) {
          const int step = U.step0 + j, nblk = (U.len + kBlock - 1) / kBlock;
          int keep[2];                 // rows of each block that stay
          bool patch = (step + 1) * kStep > U.len;
          for (int i = 0; i < 2; ++i) {
            const int blk = 2 * step + i;
            keep[i] = max(0, min(kBlock, U.len - blk * kBlock));
            if (U.bad && blk < nblk && (block_row(a.k, U.b, U.g, blk, U.len, D) < 0 ||
                                        block_row(a.v, U.b, U.g, blk, U.len, D) < 0)) {
              keep[i] = 0;
              patch = true;
            }
          }
          if (!patch) continue;
          const int s = (kc + 2 * j + 1) % (NS + U.more);
          if (!warp_wait_sleep(&bars->kv_raw[s], (raw_phase >> s) & 1)) { ok = false; break; }
          raw_phase ^= 1u << s;
          unsigned char* st = smem + C::kOffKV + (s - U.more) * C::kTile;
          for (int x = 0; x < C::kHalves; ++x)
            for (int i = 0; i < 2; ++i)
              for (int c = keep[i] * 8 + lane; c < kBlock * 8; c += 32)
                *reinterpret_cast<uint4*>(st + x * C::kSlab + i * 8192 + c * 16) =
                    make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->kv_full[s]);
        }
        if (!ok) {
          if (lane == 0) set_abort(bars, a.status);
          break;
        }
        kc += 2 * max(0, n);
      }
    } else if (warp == kWarpMma && elect_one()) {
      // ------------------------------------------------- MMA issuer of both tiles
      // One thread, the tiles in turn: P V (j) and S (j + 1) of tile 0, then of tile 1. The
      // tensor cores work in that order, so the tiles' softmax phases are half a period
      // apart (with an issuer for each tile both were in their softmax, then both on the
      // tensor cores: 5900 cycles a step at d = 128).
      const uint32_t idS = tc::idesc_f16(128, kStep, 1, false);
      const uint32_t idPV = tc::idesc_f16(128, D, 1, true);
      const uint32_t sbase = smem_u32(smem);
      const uint64_t dq0 = tc::smem_desc_sw128(sbase, 16, 1024);
      const uint64_t dk0 = tc::smem_desc_sw128(sbase + C::kOffKV, 16, 1024);
      const uint64_t dv0 = tc::smem_desc_sw128(sbase + C::kOffKV, C::kSlab, 1024);
      uint32_t un = 0, q_phase = 0, p_phase = 0;   // phases: a bit for each tile or buffer
      uint32_t o_phase = 1;                        // of o_empty, at the unit before
      struct Pos {                                 // a stage of the ring and its phase
        int st;
        uint32_t phase;
      };
      int more = 0;
      auto step = [&](Pos& p) {                    // to the same operand of the next step
        p.st += 2;
        if (p.st >= NS + more) {
          p.st -= NS + more;
          p.phase ^= 1;
        }
      };
      Pos kp = {0, 0}, vp = {1, 0};                // K and V take the stages in turn
      int total = 0;                               // (step, tile) pairs of the unit
      bool one = false;                            // one tile of rows
      // the next unit that has keys; total = 0 at the end. False: a wait gave up.
      auto fetch = [&]() {
        while (true) {
          const int slot = un & 1;
          if (!mbar_wait_sleep(&bars->info_full[slot], (un >> 1) & 1)) return false;
          const Unit U = bars->info[slot];
          mbar_arrive(&bars->info_empty[slot]);
          ++un;
          const bool stop = U.u < 0 || aborted(bars);
          one = U.ntok <= half_tok;
          more = U.more;
          total = stop ? 0 : (U.step1 - U.step0) * (one ? 1 : 2);
          if (stop || total > 0) return true;
        }
      };
      // sums with a descriptor are made where they are used: made ahead, they spill
      auto keep = [](uint64_t& desc) { asm volatile("" : "+l"(desc)); };
      auto full = [&](const Pos& p) { return mbar_wait(&bars->kv_full[p.st], p.phase); };
      auto release = [&](const Pos& p) { tc::commit(&bars->kv_empty[p.st]); };
      // S of tile t from Q tile q, in buffer b
      auto scores = [&](int t, int b, int q, const Pos& p) {
        uint64_t dq = dq0 + ((q * C::kTile) >> 4), dk = dk0 + (((p.st - more) * C::kTile) >> 4);
        keep(dq);
        keep(dk);
        tc::fence_after_sync();
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t off = ((ks >> 2) * C::kSlab + (ks & 3) * 32) >> 4;
          tc::mma_ss(tmem + C::kScores + 128 * b, dq + off, dk + off, idS, ks > 0);
        }
        tc::commit(&bars->s_full[t][C::kRing == 2 ? 0 : b]);
      };
      // O of tile t += P V, P (buffer b) by quarters of the keys as the softmax hands them over
      auto values = [&](int t, int b, const Pos& p, bool first) {
        const uint32_t s_tm = tmem + C::kScores + 128 * b, o_tm = tmem + D * t;
        const uint32_t phase = (p_phase >> b) & 1;
        p_phase ^= 1u << b;
        uint64_t dv = dv0 + (((p.st - more) * C::kTile) >> 4);
        keep(dv);
        if (first && !mbar_wait(&bars->o_empty[t], o_phase)) return false;
        if (!full(p)) return false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (!mbar_wait(&bars->p_ready[b][i], phase)) return false;
          tc::fence_after_sync();
#pragma unroll
          for (int kk = 2 * i; kk < 2 * i + 2; ++kk) {
            tc::mma_ts(o_tm, s_tm + kk * 8, dv + ((kk * 2048) >> 4), idPV, !first || kk > 0);
            if constexpr (kParts == 2)
              tc::mma_ts(o_tm, s_tm + kStep / 2 + kk * 8, dv + ((kk * 2048) >> 4), idPV, true);
          }
        }
        return true;
      };
      auto query = [&](int t) {
        const uint32_t phase = (q_phase >> t) & 1;
        q_phase ^= 1u << t;
        return mbar_wait(&bars->q_full[t], phase);
      };
      // Pair i is step i / 2 of tile i % 2 (the K and V of a step are used twice) or, with one
      // tile of rows, step i in tile i % 2 of tensor memory. With a buffer of scores for each
      // tile, pair i + 2 is scored behind the P V of pair i: a tile's softmax waits for it,
      // at d = 64 for a part of 2,820 cycles a step. There tensor memory has room for a third, which
      // the tiles take in turn, and pair i + 3 is scored then (2,730 cycles; 1,008 rows over 9K
      // keys, 64/4 heads, 949 us instead of 1,012). What is left is latency: a prompt of 8K has its
      // issue slots 56% busy, its exponentials' units 55%, the tensor pipe 36%.
      int ring = 0;                                // with three: the buffer of the unit's pair 0
      bool ok = fetch();
      while (ok && total > 0) {
        if constexpr (C::kRing == 2) {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int q = one ? 0 : t;
            if (t >= total || !ok) break;
            if (t == 0 || !one) ok = query(q);
            ok = ok && full(kp);
            if (!ok) break;
            scores(t, t, q, kp);
            // Q is free after the unit's last scores
            if (one ? t + 1 == total : t + 2 >= total) tc::commit(&bars->q_empty[q]);
            if (one || t == 1) {
              release(kp);
              step(kp);
            }
          }
          for (int i0 = 0; i0 < total && ok; i0 += 2) {
#pragma unroll 1
            for (int t = 0; t < 2; ++t) {
              const int i = i0 + t, q = one ? 0 : t;
              if (i >= total) break;
              ok = values(t, t, vp, i0 == 0);
              if (!ok) break;
              const bool more = i + 2 < total;
              if (more) {
                if (one || t == 0) ok = full(kp);
                if (!ok) break;
                scores(t, t, q, kp);
                if (one ? i + 3 == total : i + 4 >= total) tc::commit(&bars->q_empty[q]);
              } else {
                tc::commit(&bars->o_full[t]);
              }
              // the stages behind the scores: a commit takes its time, and the softmax waits for S
              if (one || t == 1) {
                release(vp);
                step(vp);
                if (more) {
                  release(kp);
                  step(kp);
                }
              }
            }
          }
        } else {
          int sb = ring, vb = ring;                // the next buffers of scores and of values
          // pair i is scored; `after` of the unit come after it
          auto score = [&](int i, int after) {
            const int t = i & 1, q = one ? 0 : t;
            if (i < 2 && (i == 0 || !one)) ok = query(q);
            ok = ok && full(kp);
            if (!ok) return;
            scores(t, sb, q, kp);
            if (++sb == C::kRing) sb = 0;
            if (one ? after == 0 : after < 2) tc::commit(&bars->q_empty[q]);
            if (one || t == 1) {
              release(kp);
              step(kp);
            }
          };
#pragma unroll 1
          for (int i = 0; i < C::kRing && i < total && ok; ++i) score(i, total - 1 - i);
#pragma unroll 1
          for (int i = 0; i < total && ok; ++i) {
            const int t = i & 1;
            ok = values(t, vb, vp, i < 2);
            if (!ok) break;
            tc::commit(&bars->pv_done[t]);
            if (++vb == C::kRing) vb = 0;
            if (i + C::kRing < total) score(i + C::kRing, total - 1 - i - C::kRing);
            if (i + 2 >= total) tc::commit(&bars->o_full[t]);
            if (one || t == 1) {
              release(vp);
              step(vp);
            }
          }
          ring = vb;
        }
        o_phase ^= 1;
        if (ok) ok = fetch();
      }
      if (!ok) set_abort(bars, a.status);
      // every MMA this thread issued must finish before tensor memory is freed (bounded)
      tc::commit(&bars->mma_done);
      mbar_wait_sleep(&bars->mma_done, 0, 200000000ull);
    }
  } else {
    // ------------------------------------------------------------------ softmax of tile t
    // Warp w has rows 32 (w % 4) .. + 31 of the tile (the quarter of tensor memory that it
    // reaches), one a thread: row maxima and sums need no exchange.
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kRegsSoftmax));
    const int t = warp >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t o_col = tmem + lane_addr + D * t;
    uint32_t s_col = tmem + lane_addr + C::kScores + 128 * t;
    uint32_t ring = 0, buf = t;                // with three buffers: of the unit's pair 0, of this step
    const float sc = a.scale_log2;
    // barrier phases, a bit each: 0 o_empty, at the unit before, 3 s_full (with three buffers:
    // pv_done), 4-5 units mod 4, 6-8 s_full of three buffers
    uint32_t bits = 1;
    while (true) {
      const int slot = (bits >> 4) & 1;
      if (!warp_sleep_all(&bars->info_full[slot], (bits >> 5) & 1)) {
        if (lane == 0) set_abort(bars, a.status);
        break;
      }
      // Read again where it is needed and given back at the end: what lives across the step
      // loop takes registers from the scores.
      const volatile Unit& U = bars->info[slot];
      bits = (bits & ~48u) | ((bits + 16) & 48);
      if (U.u < 0 || aborted(bars)) break;
      float m = -INFINITY;
      float l = 0.f, comp = 0.f;                // see the end of a step
      bool ok = true;
      // One tile of rows (twin): both tiles have the same rows and take the steps in turn.
      int lim;                                  // columns 0 .. lim of the step are visible
      bool idle;                                // no row of this warp exists
      const int stride = U.ntok <= half_tok ? 2 : 1;
      int left = U.step1 - U.step0 - (stride - 1) * t;
      {
        const int tok0 = stride == 2 ? 0 : t * half_tok, tok = tok0 + (row >> a.lgG);
        // The last key this row sees. Rows that do not exist are masked like the others: if they
        // saw nothing, their warp would mask every step (3,900 cycles instead of 3,050 where they
        // are the rest of a tile). Nobody reads them, whatever they hold.
        const int last = a.causal ? min(U.pos0 + tok, U.len - 1) : U.len - 1;
        lim = last - (U.step0 + (stride - 1) * t) * kStep;
        idle = tok0 + ((quarter * 32) >> a.lgG) >= U.ntok;
      }
      for (; left > 0; left -= stride, lim -= stride * kStep, bits ^= 8) {
        if constexpr (C::kRing == 2) {
          if (!warp_wait_all(&bars->s_full[t][0], (bits >> 3) & 1)) { ok = false; break; }
        } else {
          if (!warp_wait_all(&bars->s_full[t][buf], (bits >> (6 + buf)) & 1)) { ok = false; break; }
          bits ^= 64u << buf;
          s_col = tmem + lane_addr + C::kScores + 128 * buf;
        }
        uint64_t* ready = bars->p_ready[buf];
        if constexpr (C::kRing == 3) buf = buf == 0 ? 2 : buf - 1;     // two pairs on
        if (idle) {   // rows of P that nobody reads
          if (lane == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) mbar_arrive(&ready[i]);
          }
          continue;
        }
        tc::fence_after_sync();
        uint32_t s[4][32];
#pragma unroll
        for (int i = 0; i < 4; ++i) tc::ld32(s_col + 32 * i, s[i]);
        tc::wait_ld();
        if (lim < kStep - 1) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (32 * i + c > lim) s[i][c] = 0xff800000u;
        }
        if (U.bad) {
          for (int x = 0; x < 2; ++x) {
            const int blk = 2 * (U.step1 - left) + x;
            if (blk * kBlock < U.len && (block_row(a.k, U.b, U.g, blk, U.len, D) < 0 ||
                                         block_row(a.v, U.b, U.g, blk, U.len, D) < 0)) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < 32; ++c)
                  if ((i >> 1) == x) s[i][c] = 0xff800000u;
            }
          }
        }
        float mx[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          mx[i] = max3(__uint_as_float(s[i][0]), __uint_as_float(s[i][1]), __uint_as_float(s[i][2]));
#pragma unroll
          for (int c = 3; c < 31; c += 2)
            mx[i] = max3(mx[i], __uint_as_float(s[i][c]), __uint_as_float(s[i][c + 1]));
          mx[i] = fmaxf(mx[i], __uint_as_float(s[i][31]));
        }
        const float x = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;
        const bool up = x > m + 8.0f;
        const float f = up ? ex2(m - x) : 1.0f;
        if (__any_sync(0xffffffffu, up)) {
          if (up) {
            l *= f;
            comp *= f;
            m = x;
          }
          if (left < U.step1 - U.step0 - (stride - 1) * t) {
            // the tile's P V of the last step is done: with two buffers its S was issued behind it
            if constexpr (C::kRing == 3) {
              if (!warp_wait_all(&bars->pv_done[t], ((bits >> 3) & 1) ^ 1)) { ok = false; break; }
              tc::fence_after_sync();
            }
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t ov[32];
              tc::ld32(o_col + c, ov);
              tc::wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * f);
              tc::st32(o_col + c, ov);
            }
          }
        }
        const float neg = m == -INFINITY ? 0.f : -m;
        const float2 neg2 = make_float2(neg, neg), sc2 = make_float2(sc, sc);
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {   // the P V of 32 keys starts when they are written
          uint32_t hi[16], lo[16];
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const float2 v = __ffma2_rn(
                make_float2(__uint_as_float(s[i][c]), __uint_as_float(s[i][c + 1])), sc2, neg2);
            const float2 p = (c / 2) % kPolyOf >= kPolyOf - C::kPoly
                                 ? exp2_poly(v) : make_float2(ex2(v.x), ex2(v.y));
            sum = __fadd2_rn(sum, p);
            if constexpr (kParts == 2) {   // the leading 8 bits, and the rest rounded to 8 more
              const uint32_t x = __float_as_uint(p.x), y = __float_as_uint(p.y);
              const float2 rest = __fadd2_rn(p, make_float2(-__uint_as_float(x & 0xffff0000u),
                                                            -__uint_as_float(y & 0xffff0000u)));
              hi[c / 2] = __byte_perm(x, y, 0x7632);
              lo[c / 2] = pack_bf16(rest.x, rest.y);
            } else {
              hi[c / 2] = pack_bf16(p.x, p.y);
            }
          }
          st16(s_col + 16 * i, hi);
          if constexpr (kParts == 2) st16(s_col + kStep / 2 + 16 * i, lo);
          tc::wait_st();
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ready[i]);
        }
        // A step's sum joins l with what the last one lost in the rounding (Kahan's summation): l is
        // within 64 2^-24 of the sum of its terms at any length. Added one by one to two running sums,
        // equal scores behind a larger one round the same way each time: off by 7.8e-3 of l at 2^20 keys.
        const float y = (sum.x + sum.y) - comp, z = l + y;
        comp = (z - l) - y;
        l = z;
      }
      if (!ok || aborted(bars)) {
        if (lane == 0) set_abort(bars, a.status);
        break;
      }
      // (m, l) goes to the out warps, which have read the last unit's
      if (U.step1 > U.step0) {
        if (!warp_wait_all(&bars->o_empty[t], bits & 1)) {
          if (lane == 0) set_abort(bars, a.status);
          break;
        }
        bits ^= 1;
        if constexpr (C::kRing == 3) {
          const int n = U.step1 - U.step0;
          ring = (ring + (U.ntok <= half_tok ? n : 2 * n)) % 3;
          buf = ring + t < 3 ? ring + t : 0;
        }
        // A score beyond fp32 makes its row NaN, as inf - inf does in ex2 (exp2_poly has 0 there).
        bars->ml[t][row] = make_float2(m, m == INFINITY ? NAN : l);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->ml_full[t]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->info_empty[slot]);
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  if (warp == kWarpMma) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

// ------------------------------------------------------------------------------- merge
// A warp joins the splits' (o, m, l) of a (row, head) and, with o_own, what the row's own tokens
// gave. All loads of up to 8 (d = 64: 16) splits are under way before the first is used; a lane
// holds (m, l) of splits lane and lane + 32 (there are no more than 64), and 16 bytes of the
// partial rows, which 32 or, at d = 64, two times 16 lanes read and add in a fixed order.
template <int D>
__global__ void __launch_bounds__(kMergeThreads) packed_merge_kernel(const PackedArgs a) {
  grid_dependency_wait();
  if (a.head[2] == 0) return;
  constexpr int kLanes = D / 4, kRows = 32 / kLanes;   // lanes a partial row, rows at a time
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = threadIdx.x & 31, sub = lane % kLanes, slot = lane / kLanes;
  const int64_t rows = static_cast<int64_t>(a.N) * a.Hq;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kMergeThreads / 32);
  for (int64_t at = blockIdx.x * (kMergeThreads / 32) + (threadIdx.x >> 5); at < rows; at += warps) {
    const int n = a.row_splits[at / a.Hq];
    if (n <= 1) continue;
    const float* from = a.part_o + at * D + sub * 4;
    float4 v[8];
    auto load = [&](int j0) {
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int j = j0 + u * kRows + slot;
        v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (j < n) v[u] = *reinterpret_cast<const float4*>(from + j * rows * D);
      }
    };
    load(0);
    float2 x[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      x[i] = make_float2(-INFINITY, 0.f);
      if (lane + 32 * i < n)
        x[i] = *reinterpret_cast<const float2*>(a.part_ml + 2 * ((lane + 32 * i) * rows + at));
    }
    float own = -INFINITY;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    if (a.lse_own != nullptr) {
      own = a.lse_own[at] * kLog2e;
      y = *reinterpret_cast<const float4*>(a.o_own + at * D + sub * 4);
    }
    float M = fmaxf(own, fmaxf(x[0].x, x[1].x));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kAll, M, o));
    const float base = M == -INFINITY ? 0.f : M;
    const float f0 = ex2(x[0].x - base), f1 = ex2(x[1].x - base);
    float L = x[0].y * f0 + x[1].y * f1;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(kAll, L, o);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j0 = 0; j0 < n; j0 += 8 * kRows) {
      if (j0 > 0) load(j0);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int j = j0 + u * kRows + slot;      // a batch is in one half of the 64
        const float f = __shfl_sync(kAll, j0 < 32 ? f0 : f1, j & 31);
        o.x = fmaf(v[u].x, f, o.x);
        o.y = fmaf(v[u].y, f, o.y);
        o.z = fmaf(v[u].z, f, o.z);
        o.w = fmaf(v[u].w, f, o.w);
      }
    }
    if constexpr (kRows == 2) {
      o.x += __shfl_xor_sync(kAll, o.x, 16);
      o.y += __shfl_xor_sync(kAll, o.y, 16);
      o.z += __shfl_xor_sync(kAll, o.z, 16);
      o.w += __shfl_xor_sync(kAll, o.w, 16);
    }
    if (own != -INFINITY) {     // o_own is normalised: a part with l = 1 at its log-sum
      const float f = ex2(own - base);
      L += f;
      o.x = fmaf(y.x, f, o.x);
      o.y = fmaf(y.y, f, o.y);
      o.z = fmaf(y.z, f, o.z);
      o.w = fmaf(y.w, f, o.w);
    }
    const float inv = L == 0.f ? 0.f : 1.0f / L;
    o = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    __syncwarp();               // o_f32 may be o_own, lse lse_own: every lane has read them
    if (slot == 0) {
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + at * D + sub * 4) =
          make_uint2(pack_bf16(o.x, o.y), pack_bf16(o.z, o.w));
      if (a.o_f32 != nullptr) *reinterpret_cast<float4*>(a.o_f32 + at * D + sub * 4) = o;
    }
    if (lane == 0) a.lse[at] = L == 0.f ? -INFINITY : (base + log2f(L)) * kLn2;
  }
}

template <int D, int kParts>
cudaError_t launch_d(const PackedArgs& a, const CUtensorMap& tq, const CUtensorMap& tk,
                     const CUtensorMap& tv, int num_sms, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (!a.in_block) e = launch_pdl(plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, a);
  if (e != cudaSuccess) return e;
  constexpr int smem = smem_bytes<D>();
  auto kern = packed_attn_kernel<D, kParts>;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int64_t units = static_cast<int64_t>(a.max_entries) * a.Hkv;
  const int grid = static_cast<int>(units < num_sms ? units : num_sms);
  e = launch_pdl(kern, dim3(grid), dim3(kThreads), smem, s, a, tq, tk, tv);
  if (e != cudaSuccess || a.smax == 1) return e;
  constexpr int kWarps = kMergeThreads / 32;
  const int64_t blocks = (static_cast<int64_t>(a.N) * a.Hq + kWarps - 1) / kWarps;
  const int64_t most = static_cast<int64_t>(kMergeBlocks) * num_sms;
  return launch_pdl(packed_merge_kernel<D>, dim3(static_cast<unsigned>(std::min(blocks, most))),
                    dim3(kMergeThreads), 0, s, a);
}

}  // namespace

cudaError_t launch_packed(const PackedArgs& a, const CUtensorMap& tq, const CUtensorMap& tk,
                          const CUtensorMap& tv, int num_sms, cudaStream_t s) {
  if (a.p_parts == 2)
    return a.d == 128 ? launch_d<128, 2>(a, tq, tk, tv, num_sms, s) : launch_d<64, 2>(a, tq, tk, tv, num_sms, s);
  return a.d == 128 ? launch_d<128, 1>(a, tq, tk, tv, num_sms, s) : launch_d<64, 1>(a, tq, tk, tv, num_sms, s);
}

}  // namespace bsa
