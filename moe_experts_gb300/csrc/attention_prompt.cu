// Causal attention of a prompt's appended rows over a paged Q8_0 cache
// (epq_attention_prompt).
//
//   s_ij = scale q_i . k_j,  o_i = sum_j exp(s_ij - m_i) v_j / sum_j exp(s_ij - m_i)
//
// over the positions j <= length + i.  The rows of one (sequence, key/value
// head) are its tokens times its `group` query heads (row r: token r / group,
// head r % group); an item is 128 of them and 128 columns of the output.
//
// One pass over the positions in tiles of 128 (64 for heads of 256), both
// products on the tensor core (tcgen05, fp16 operands, float32 sums) without
// giving up float32 accuracy: each operand is two fp16 parts, a = a1 + a2 with
// a1 the 11 leading bits, and a product is a1 b1 + a1 b2 + a2 b1 (what is left
// out is 2^-22 of it).  Powers of two keep the parts in fp16's range:
//   queries  a row's largest element in [2^14, 2^15);
//   keys     a tile's largest factor in [2^7, 2^8): code * factor < 2^15, its
//            two parts exact;
//   values   the same for each block of 32 columns of a tile;
//   weights  2^15 at the row's maximum.
// Halves are multiples of 2^-24, which is the floor: a weight is off by up to
// 2^-39 of the one at the maximum, whatever it is, and a factor below 2^-21 of
// its tile's largest by 2^-32 of that.
// The sum of a tile is read from tensor memory and added to the output's
// registers, scaled by the change of the row's maximum, so no sum in tensor
// memory outlives a tile.
//
// Roles of a CTA's warps, each a step ahead of the next:
//   copies   (1 warp) a tile's rows, page by page, into shared memory as the
//            cache holds them
//   scan     (2) their factors' maxima and scaled factors, what is missing
//   operands (8) keys of tile t + 1, then values of tile t: codes times
//            factors, two fp16 parts in swizzled shared memory
//   products (1) issues them: scores of tile t + 1, then values of tile t, so
//            that the tensor core works on one while the weights of the other
//            are made
//   weights  (4) one row a thread: maximum, exponentials, two parts, written
//            over the scores in tensor memory
//   output   (4) one row a thread: 128 columns in registers
// Work: the tiles of all items in a row, cut into equal shares, one per CTA.
// An item counts kExtra tiles more than it has: beginning it (its queries, then
// one tile through all roles) takes about that long.  A CTA's part of an item
// that it does not hold whole goes to the workspace (maximum, sum, unnormalised
// output), and a second launch joins the parts.
//
// Measured with 32 query and 8 key/value heads of 128 (both launches, from a
// graph): 65 tokens over themselves 17.9 us, 4096 over themselves 350 us, 2048
// behind 32768 positions 2.28 ms: 500 TFLOP/s of the formula's products, three
// fp16 products for each, 0.77 of the measured bf16 rate.  Heads of 256 compute
// their scores once for each half of the columns (registers and tensor memory
// hold 128 columns of sums): 250 TFLOP/s.
// A tile takes 4300 cycles, of which the tensor core's own 48 products are 70 %;
// the thread that issues them waits 17 % of the time for operands or weights.
// Beside them the shared memory is as busy (operands written 128 KB, read by the
// tensor core 192 KB a tile), and the operands' and the weights' warps are at work
// for 85 % of it: none of the three can be made faster alone.  A call with few
// tiles is one chain: the work found (3 us), an item begun (4), a tile through
// the roles (4), outputs written (3), the join.
// What did not pay: keys and values handed over in halves, so that an operand's
// place is free earlier (twice the barriers: 3.3 ms); queries prefetched to L2
// when the item before begins (355 -> 366 us for 4096 tokens).
#include <algorithm>
#include <cmath>

#include "pages.cuh"
#include "tcgen05.cuh"

namespace epq {
namespace {

constexpr int kRows = 128;     // rows of an item
constexpr int kCols = 128;     // output columns of an item
constexpr int kMaxCtas = 152;  // one per SM of a GB300
constexpr int kMaxGroupPrompt = 16;
constexpr int kExtra = 4;      // (4096 tokens: 3 365 us, 4 347, 5 350; unequal prompts: 3 31.2, 4 30.9, 5 33.2)
constexpr int kAhead = 4;  // tiles that the scan may be ahead of the output
constexpr int kRaw = 2;    // tiles of keys, and of values, as the cache holds them
constexpr int kJoinWarps = 8;
constexpr int kPartLd = kCols + 4;

// Warps: 0-3 weights, 4-7 output, 8-15 operands, 16 products, 17 copies, 18-19
// scan.  Registers of each group of four warps: the launch has 5 * 128 threads *
// 96, and 5 * 96 = 104 + 168 + 72 + 72 + 64.
constexpr int kThreads = 640;
constexpr int kRegsWeights = 104, kRegsOutput = 168, kRegsOperand = 72, kRegsRest = 64;
constexpr int kRegsLaunch = 96;
static_assert(kRegsWeights + kRegsOutput + 2 * kRegsOperand + kRegsRest <= 5 * kRegsLaunch,
              "a split above the launch's total waits forever");

struct Part {  // what a CTA left in the workspace: tiles a..b-1 of an item of `tiles` (0: nothing)
  int s, rt, y, a, b, tiles, pad[2];
};

struct PromptParams {
  PagesView v;
  const float *q;
  const int32_t *n_tok;
  int64_t q_ld, q_seq_ld;
  int layer, n_heads, group, ntok, window;
  float scale;
  float *out;
  Part *notes;   // workspace: [2 per CTA]
  float *parts;  // workspace: [2 per CTA][kRows][kPartLd]
  unsigned *err;
};

// Sizes that follow from the head.
template <int kD>
struct Shape {
  static constexpr int kPos = kD == 128 ? 128 : 64;  // positions of a tile
  static constexpr int kSplit = kD / kCols;          // items that share a row tile's scores' rows
  static constexpr uint32_t kKPart = kPos * kD * 2;  // bytes of one part of a tile's keys
  static constexpr uint32_t kVPart = kPos * kCols * 2;  // and of its values
  static constexpr uint32_t kRow = kD + kD / 16;        // bytes of a row
  static constexpr uint32_t kPlane = kPos * kRow;       // of a tile's rows
  // shared memory: keys, values, rows
  static constexpr uint32_t kV = 2 * kKPart, kRows = kV + 2 * kVPart, kBytes = kRows + kRaw * 2 * kPlane;
  // columns of tensor memory
  static constexpr uint32_t kQ = 0, kS = kD, kT = kD + 2 * kPos;
  static_assert(kT + kCols <= 512, "");
};

// What the scan says of a tile.
struct alignas(16) Entry {
  __half kf[512], vf[512];  // scaled factors [position][block], 0 where there is nothing to read
  float lost[128];          // 0; NaN: a factor is not finite; -inf: no page
  float kmul, vmul[4];      // what undoes the factors' scales
  int any;                  // whether some `lost` matters
};

// An item of the CTA's share, in the order of the work.
struct Item {
  int s, h, col, rt;   // sequence, head, first output column, row tile
  int len, rows;       // the sequence's committed length and rows
  int t0, t1;          // tokens of the row tile
  int end;             // positions that any of its rows sees
  int from, tiles;     // first position that any of them sees, and tiles, of the CTA's part of it; no tiles: there is no further item
  int before;          // tiles of the items before
  int slot;            // where a part of an item goes, -1: the item is whole
};
constexpr int kItems = 8;

struct Control {
  uint64_t item_full[kItems], item_free[kItems];
  Item item[kItems];
  uint64_t raw_full[2][kRaw], raw_free[2][kRaw], k_full, v_full, s_full[2], p_full[2], t_full, t_free, q_full, c_full[kAhead],
      fin_full, fin_empty, scan_full[kAhead], entry_free[kAhead], drain;
  uint32_t tmem;
  long long begin, end;  // the CTA's share
  int s, rt, y, tile;    // where it begins
  long long sums[kThreads / 32];
  int pair0[kMaxSeq + 1];  // row tiles of the sequences before each
  int2 seq[kMaxSeq];       // length, tokens
  Entry entry[kAhead];
  uint32_t scan[2][2][6];  // what the two scanning warps tell each other
  float corr[kAhead][kRows];
  float off[kRows], den[kRows], row_mul[kRows];
};

// The code of all roles together has to fit the SM's instruction cache (unrolled
// further the warps waited for instructions half of the time, 5.0 ms where 2.3
// are now): loops are unrolled only as far as registers or latencies ask for,
// and what a wait does when it gives up is out of line.  (No other call: a role's
// registers are fewer than the launch's.)
__device__ __noinline__ void gave_up(unsigned *err, unsigned code, unsigned where) { record_error(err, code, where); }

__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, unsigned *err, unsigned code, unsigned where = 0) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
  while (!mbar_try_wait(bar, parity))
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      gave_up(err, code, where);
      return false;
    }
  return true;
}

// All lanes of the warp wait; the same answer for all, so that they leave
// together and meet in the warp-wide instructions that follow.
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, unsigned *err, unsigned code, unsigned where) {
  return __all_sync(0xffffffffu, wait(bar, parity, err, code, where));
}

__device__ __forceinline__ int row_tiles(const PromptParams &p, int n) { return (n * p.group + kRows - 1) / kRows; }

// Row tile rt of a sequence: its tokens, and the positions that any of them sees.
struct Span {
  int t0, t1, begin, end, first, tiles;  // first: the first tile's index; tiles: how many
};

template <int kD>
__device__ __forceinline__ Span span_of(const PromptParams &p, int len, int n, int rt) {
  constexpr int kPos = Shape<kD>::kPos;
  Span x;
  x.t0 = rt * kRows / p.group;
  x.t1 = (min((rt + 1) * kRows, n * p.group) - 1) / p.group;
  x.end = len + x.t1 + 1;
  x.begin = p.window ? max(0, len + x.t0 - p.window + 1) : 0;
  x.first = x.begin / kPos;
  x.tiles = (x.end + kPos - 1) / kPos - x.first;
  return x;
}

// Inclusive sum over the CTA.
__device__ __forceinline__ long long scan_sum(long long x, long long *sums, long long *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  long long all = 0, base = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w == warp) base = all;
    all += sums[w];
  }
  *total = all;
  return base + x;
}

// The CTA's share of the tiles and where it begins; ends with a CTA barrier.
template <int kD>
__device__ __forceinline__ void find_work(const PromptParams &p, Control &c) {
  const int tid = threadIdx.x, lane = tid & 31;
  for (int s = tid; s < p.v.n_seq; s += kThreads)
    c.seq[s] = make_int2(seq_length(p.v, s), p.n_tok ? min(max(p.n_tok[s], 0), p.ntok) : p.ntok);
  __syncthreads();
  if (tid < 32) {
    int run = 0;
    for (int s0 = 0; s0 < p.v.n_seq; s0 += 32) {
      int x = s0 + lane < p.v.n_seq ? row_tiles(p, c.seq[s0 + lane].y) : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (s0 + lane < p.v.n_seq) c.pair0[s0 + lane + 1] = run + x;
      run += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) c.pair0[0] = 0, c.begin = c.end = 0;
  }
  __syncthreads();
  const int pairs = c.pair0[p.v.n_seq], heads = p.v.n_kv * Shape<kD>::kSplit;
  const auto find = [&](int pair) {  // the last sequence with pair0 <= pair (empty ones are passed over)
    int lo = 0, hi = p.v.n_seq - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (c.pair0[mid] <= pair) lo = mid;
      else hi = mid - 1;
    }
    return lo;
  };
  const auto units = [&](int pair, int s) {
    return span_of<kD>(p, c.seq[s].x, c.seq[s].y, pair - c.pair0[s]).tiles + kExtra;
  };
  // the tiles of all row tiles, and those before the thread's own (of the first kThreads)
  long long mine = 0, first = 0, total;
  for (int k = tid; k < pairs; k += kThreads) {
    const int each = units(k, find(k));
    if (k == tid) first = each;
    mine += each;
  }
  long long upto = scan_sum(mine, c.sums, &total);
  const bool once = pairs <= kThreads;  // then that is the sum which the second look needs
  total *= heads;
  const long long ctas = total < gridDim.x ? total : gridDim.x;
  if (blockIdx.x < ctas) {
    // 32 bits, where they are enough, divide in a fraction of the time
    const long long share = total >> 32 ? total / ctas : static_cast<unsigned>(total) / static_cast<unsigned>(ctas);
    const long long rest = total - share * ctas, b = blockIdx.x;
    const long long begin = b * share + (b < rest ? b : rest), end = begin + share + (b < rest);
    long long run = 0;
    for (int k0 = 0; run <= begin; k0 += kThreads) {
      const int k = k0 + tid, s = k < pairs ? find(k) : 0;
      long long each = first, all = 0;
      if (!once) {
        each = k < pairs ? units(k, s) : 0;
        upto = scan_sum(each, c.sums, &all);
      }
      const long long to = run + heads * upto, from = to - heads * each;
      run = once ? total : run + heads * all;
      if (from <= begin && begin < to) {
        const long long at = begin - from;
        c.s = s, c.rt = k - c.pair0[s];
        c.y = static_cast<int>(at >> 32 ? at / each : static_cast<unsigned>(at) / static_cast<unsigned>(each));
        c.tile = static_cast<int>(at - c.y * each);
        c.begin = begin, c.end = end;
      }
    }
  }
  __syncthreads();
}

// The items of a CTA's share, one after the other.  The copies' warp walks and
// tells the other roles.
template <int kD>
struct Walk {
  long long left;
  int s, rt, y, tile, before;  // where the next item begins; tiles before it
  bool begins;                 // whether the share begins with it (or in it)
  __device__ explicit Walk(const Control &c)
      : left(c.end - c.begin), s(c.s), rt(c.rt), y(c.y), tile(c.tile), before(0), begins(true) {}
  // The next item; its part's note for the join is written, where it is one.
  __device__ Item next(const PromptParams &p, const Control &c) {
    Item x = {};
    while (left > 0) {
      const int len = c.seq[s].x, n = c.seq[s].y;
      if (rt >= row_tiles(p, n)) {
        ++s, rt = 0;
        continue;
      }
      const Span span = span_of<kD>(p, len, n, rt);
      const long long take = min(left, static_cast<long long>(span.tiles + kExtra - tile));
      const int a = tile, b = min(tile + static_cast<int>(take), span.tiles);
      if (a < b) {
        x = {s, y / Shape<kD>::kSplit, y % Shape<kD>::kSplit * kCols, rt, len, n * p.group, span.t0, span.t1, span.end,
             max(span.begin, (span.first + a) * Shape<kD>::kPos), b - a, before, -1};
        if (a > 0 || b < span.tiles) {
          x.slot = begins ? 0 : 1;
          if ((threadIdx.x & 31) == 0) p.notes[2 * blockIdx.x + x.slot] = Part{s, rt, y, a, b, span.tiles, {0, 0}};
        }
        before += b - a;
      }
      left -= take;
      tile = 0;
      begins = false;
      if (++y == p.v.n_kv * Shape<kD>::kSplit) y = 0, ++rt;
      if (a < b) break;
    }
    return x;
  }
};

// Item n of the walk, once it is known.  A role that has what it needs of it
// gives the place back (one arrival a warp).
template <bool kWarp = true>
__device__ __forceinline__ bool item_at(const PromptParams &p, Control &c, int n, Item &x) {
  uint64_t *bar = &c.item_full[n % kItems];
  const int phase = (n / kItems) & 1;
  if (!(kWarp ? wait_warp(bar, phase, p.err, DEVERR_FULL_WAIT, n) : wait(bar, phase, p.err, DEVERR_FULL_WAIT, n))) return false;
  x = c.item[n % kItems];
  return x.tiles > 0;
}

__device__ __forceinline__ void item_done(Control &c, int n) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&c.item_free[n % kItems]);
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<const __half2 *>(&x); }
__device__ __forceinline__ uint32_t as_bits(__half2 x) { return *reinterpret_cast<const uint32_t *>(&x); }

// x, y as two fp16 parts each: the 11 leading bits, and the rest rounded.
__device__ __forceinline__ void split2(float x, float y, uint32_t &first, uint32_t &rest) {
  const float a = __uint_as_float(__float_as_uint(x) & 0xffffe000u);
  const float b = __uint_as_float(__float_as_uint(y) & 0xffffe000u);
  first = pack_half2(a, b);
  rest = pack_half2(x - a, y - b);
}

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Exponent of a finite half's bits (of 0: 0).
__device__ __forceinline__ int half_exponent(int bits) {
  return bits ? static_cast<int>(__float_as_uint(half_bits_to_float(bits)) >> 23) - 127 : 0;
}

// ------------------------------------------------------------------ copies
// One warp.  A tile's rows lie in runs, each within a page; lane r brings run r
// of the keys and of the values, where any of its positions is seen (a page that
// lies below the window of all rows need not be there).
template <int kD>
__device__ void copies_role(const PromptParams &p, Control &c, uint8_t *smem) {
  using S = Shape<kD>;
  const int lane = threadIdx.x & 31, run = min(p.v.P, S::kPos);
  const uint32_t bytes = run * S::kRow;
  Walk<kD> w(c);
  int issued[2] = {};
  bool ok = true;
  int told = 0;  // items that the other roles know of: one more than the copies are at
  const auto tell = [&]() {
    if (told >= kItems) ok = wait_warp(&c.item_free[told % kItems], (told / kItems - 1) & 1, p.err, DEVERR_EMPTY_WAIT, told);
    if (!ok) return;
    const Item x = w.next(p, c);
    if (lane == 0) {
      c.item[told % kItems] = x;
      mbar_arrive(&c.item_full[told % kItems]);
    }
    __syncwarp();
    ++told;
  };
  tell();
  for (int n = 0; ok; ++n) {
    const Item x = c.item[n % kItems];
    if (x.tiles == 0) break;
    tell();
    for (int k = 0; ok && k < x.tiles; ++k) {
      const int g = x.before + k, stage = g % kRaw;
      const int pos = (x.from & -S::kPos) + k * S::kPos + lane * run;
      const bool used = lane * run < S::kPos && pos < x.end && pos + run > x.from;
      const int page = used ? seq_page(p.v, x.s, pos / p.v.P) : -1;
      if (used && page < 0) record_error(p.err, DEVERR_NO_PAGE, static_cast<unsigned>(x.s));
      const uint32_t all = __popc(__ballot_sync(0xffffffffu, page >= 0)) * bytes;
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        if (ok && g >= kRaw) ok = wait_warp(&c.raw_free[v][stage], (g / kRaw - 1) & 1, p.err, DEVERR_EMPTY_WAIT, g);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&c.raw_full[v][stage], all);
        __syncwarp();
        if (page >= 0)
          bulk_g2s(smem + S::kRows + (2 * stage + v) * S::kPlane + lane * bytes,
                   page_row(p.v, p.layer, page, x.h, v, pos % p.v.P), bytes, &c.raw_full[v][stage]);
        issued[v] = g + 1;
      }
    }
    item_done(c, n);
  }
  for (int x = 0; x < 2; ++x)  // no copy is in flight when the CTA ends
    for (int g = max(0, issued[x] - kRaw); g < issued[x]; ++g)
      wait_warp(&c.raw_full[x][g % kRaw], (g / kRaw) & 1, p.err, DEVERR_DRAIN_WAIT, g);
}

// ------------------------------------------------------------------ scan
// Four halves times a power of two (one that is not finite: 0).
__device__ __forceinline__ uint2 scale4(uint2 f, const float (&mul)[4]) {
  float y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t h = ((i & 2 ? f.y : f.x) >> (16 * (i & 1))) & 0xffffu;
    y[i] = (h & 0x7fffu) < 0x7c00u ? half_bits_to_float(h) * mul[i] : 0.0f;
  }
  return make_uint2(pack_half2(y[0], y[1]), pack_half2(y[2], y[3]));
}

// Largest of two pairs of halves, as bits without the sign (an element that is
// not finite counts as 0).
__device__ __forceinline__ uint32_t larger2(uint32_t a, uint32_t b) {
  b &= 0x7fff7fffu;
  if ((b & 0x7fffu) >= 0x7c00u) b &= 0xffff0000u;
  if (b >= 0x7c000000u) b &= 0xffffu;
  return __vmaxu2(a, b);
}

// Two warps, kPos / 64 positions a lane.  They meet for each tile.  One that gives
// up says so where its note of the next tile would be, and arrives without
// waiting: the other one, which meets it there, leaves too, so that neither waits
// for a warp that has left.
constexpr uint32_t kGone = 2;
template <int kD>
__device__ void scan_role(const PromptParams &p, Control &c) {
  using S = Shape<kD>;
  constexpr int kPos = S::kPos, kWords = kD / 128, kMine = kPos / 64;
  const int t = threadIdx.x - 18 * 32, lane = t & 31;
  int g = 0;  // the next tile
  Item it;
  it.tiles = 1;
  for (int n = 0; item_at(p, c, n, it); ++n) {
    item_done(c, n);
    const int split = it.col / kCols;
#pragma unroll 1
    for (int k = 0; k < it.tiles; ++k, ++g) {
      const int p0 = (it.from & -kPos) + k * kPos;
      Entry &e = c.entry[g % kAhead];
      uint2 kf[kMine][kWords], vf[kMine][kWords];
      bool read[kMine];
#pragma unroll
      for (int m = 0; m < kMine; ++m) {
        const int pos = p0 + t + 64 * m;
        const int page = pos >= it.from && pos < it.end ? seq_page(p.v, it.s, pos / p.v.P) : -1;
        read[m] = page >= 0;
        const uint8_t *row = page_row(p.v, p.layer, max(page, 0), it.h, 0, pos % p.v.P);
#pragma unroll
        for (int x = 0; x < kWords; ++x) {
          kf[m][x] = read[m] ? *reinterpret_cast<const uint2 *>(row + 8 * x) : make_uint2(0, 0);
          vf[m][x] = read[m] ? *reinterpret_cast<const uint2 *>(row + p.v.P * S::kRow + 8 * x) : make_uint2(0, 0);
        }
      }
      uint32_t kmax = 0, vmax[2] = {};
      bool bad[kMine], any = false;
#pragma unroll
      for (int m = 0; m < kMine; ++m) {
        bad[m] = false;
#pragma unroll
        for (int x = 0; x < kWords; ++x) {
          const uint32_t four[4] = {kf[m][x].x, kf[m][x].y, vf[m][x].x, vf[m][x].y};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            bad[m] |= (four[i] & 0x7c00u) == 0x7c00u || (four[i] & 0x7c000000u) == 0x7c000000u;
          kmax = larger2(larger2(kmax, kf[m][x].x), kf[m][x].y);
          if (kWords == 1 || x == split) vmax[0] = larger2(vmax[0], vf[m][x].x), vmax[1] = larger2(vmax[1], vf[m][x].y);
        }
        const int pos = p0 + t + 64 * m;
        any |= bad[m] || (!read[m] && pos >= it.from && pos < it.end);
      }
      if (g >= kAhead && !wait_warp(&c.entry_free[g % kAhead], (g / kAhead - 1) & 1, p.err, DEVERR_EMPTY_WAIT, g)) goto gone;
      // the largest of both warps: of the keys, and of the values by block
      uint32_t most[5];
      most[4] = max(kmax & 0xffffu, kmax >> 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) most[i] = (vmax[i / 2] >> (16 * (i & 1))) & 0xffffu;
#pragma unroll
      for (int i = 0; i < 5; ++i) most[i] = __reduce_max_sync(0xffffffffu, most[i]);
      any = __any_sync(0xffffffffu, any);
      uint32_t *mine = c.scan[g & 1][t >> 5];
      if (lane == 0) {
#pragma unroll
        for (int i = 0; i < 5; ++i) mine[i] = most[i];
        mine[5] = any;
      }
      named_sync(1, 64);
      const uint32_t *other = c.scan[g & 1][1 - (t >> 5)];
      if (other[5] == kGone) return;
      float mul[5];
#pragma unroll
      for (int i = 0; i < 5; ++i) mul[i] = exp2i(7 - half_exponent(max(most[i], other[i])));
#pragma unroll
      for (int m = 0; m < kMine; ++m) {
        const int row = t + 64 * m;
        e.lost[row] = !read[m] ? -INFINITY : bad[m] ? __int_as_float(0x7fffffff) : 0.0f;
        const float kmul[4] = {mul[4], mul[4], mul[4], mul[4]}, vmul[4] = {mul[0], mul[1], mul[2], mul[3]};
#pragma unroll
        for (int x = 0; x < kWords; ++x)
          *reinterpret_cast<uint2 *>(e.kf + row * (kD / 32) + 4 * x) = scale4(kf[m][x], kmul);
        *reinterpret_cast<uint2 *>(e.vf + row * 4) = scale4(kWords == 1 || split == 0 ? vf[m][0] : vf[m][kWords - 1], vmul);
      }
      if (t == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) e.vmul[i] = __frcp_rn(mul[i]);  // exact: powers of two
        e.kmul = __frcp_rn(mul[4]);
        e.any = any | other[5];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.scan_full[g % kAhead]);
    }
  }
  if (it.tiles == 0) return;  // no further item, for both; else the item's wait gave up
gone:
  if (lane == 0) c.scan[g & 1][t >> 5][5] = kGone;
  __threadfence_block();
  __syncwarp();
  asm volatile("bar.arrive 1, 64;" ::: "memory");
}

// ------------------------------------------------------------------ operands
// Eight codes times a factor as fp16: the rounded products, and what the
// rounding lost (exact: a product has 18 bits).  A byte u = code + 128 under
// the byte 0x64 is the half 1024 + u.
__device__ __forceinline__ void convert8(uint2 x, __half factor, uint4 &first, uint4 &rest) {
  const __half2 f = __half2half2(factor), bias = __half2half2(__ushort_as_half(0x6480));
  uint32_t *a = &first.x, *b = &rest.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t u = (i < 2 ? x.x : x.y) ^ 0x80808080u;
    const __half2 code = __hsub2(as_half2(__byte_perm(u, 0x64646464u, i & 1 ? 0x4342 : 0x4140)), bias);
    const __half2 y = __hmul2(code, f);
    a[i] = as_bits(y);
    b[i] = as_bits(__hfma2(code, f, __hneg2(y)));
  }
}

// What a thread does of a tile's keys or values: every `step` positions from
// its first one on, eight codes of a row.  Position r's row of 64 columns is 128
// bytes, its 16-byte pieces permuted by r % 8; a step is a multiple of 8
// positions, so that the permutation is the thread's own.
struct Piece {
  uint32_t codes, factor, to;  // bytes from the tile's rows, factors and operand
  uint32_t step, blocks;
  template <int kPos, int kWidth, int kRowBytes>
  __device__ void set() {
    constexpr int kChunks = kWidth / 8;
    const int t = threadIdx.x & 255, chunk = t % kChunks, r0 = t / kChunks;
    step = 256 / kChunks, blocks = kWidth / 32;
    codes = r0 * kRowBytes + 8 * chunk;
    factor = 2 * (r0 * blocks + chunk / 4);
    to = (chunk / 8) * (kPos * 128) + r0 * 128 + (((chunk % 8) ^ (r0 % 8)) * 16);
  }
};

template <int kD>
__device__ void operands_role(const PromptParams &p, Control &c, uint8_t *smem) {
  using S = Shape<kD>;
  const bool one = (threadIdx.x & 31) == 0;
  Piece piece[2];
  piece[0].set<S::kPos, kD, S::kRow>();
  piece[1].set<S::kPos, kCols, S::kRow>();
  int last = -1, col = 0;  // the tile whose values come next, and their first column
  bool more = true;
  for (int n = 0; more; ++n) {
    Item it;
    more = item_at(p, c, n, it);
    item_done(c, n);
    const int begin = more ? it.before : last + 1, end = more ? begin + it.tiles : begin + 1;  // (once more for the last values)
#pragma unroll 1
    for (int g = begin; g < end; ++g) {
#pragma unroll 1
      for (int x = 0; x < 2; ++x) {  // keys of tile g, then values of the tile before
        const int t = x ? last : g;
        if (x ? last < 0 : !more) continue;
        if (!x && !wait_warp(&c.scan_full[t % kAhead], (t / kAhead) & 1, p.err, DEVERR_FULL_WAIT, t)) return;
        if (!wait_warp(&c.raw_full[x][t % kRaw], (t / kRaw) & 1, p.err, DEVERR_FULL_WAIT, t)) return;
        // the tile before t has its scores (its products with the values are done): its place is free
        if (t > 0 && !wait_warp(x ? &c.t_full : &c.s_full[(t - 1) & 1], (x ? t - 1 : (t - 1) >> 1) & 1, p.err, DEVERR_EMPTY_WAIT, t))
          return;
        const Piece &m = piece[x];
        const Entry &e = c.entry[t % kAhead];
        const uint8_t *codes = smem + S::kRows + (2 * (t % kRaw) + x) * S::kPlane + kD / 16 + (x ? col : 0) + m.codes;
        const uint8_t *factors = reinterpret_cast<const uint8_t *>(x ? e.vf : e.kf) + m.factor;
        uint8_t *to = smem + (x ? S::kV : 0) + m.to, *rest = to + (x ? S::kVPart : S::kKPart);
        const uint32_t step = m.step, blocks = m.blocks;
#pragma unroll 1
        for (uint32_t i = 0; i < S::kPos; i += 4 * step)
#pragma unroll
          for (uint32_t k = 0; k < 4; ++k) {
            const uint32_t r = i + k * step;
            uint4 a, b;
            convert8(*reinterpret_cast<const uint2 *>(codes + r * S::kRow),
                     *reinterpret_cast<const __half *>(factors + 2 * r * blocks), a, b);
            *reinterpret_cast<uint4 *>(to + r * 128) = a;
            *reinterpret_cast<uint4 *>(rest + r * 128) = b;
          }
        fence_shared_async();
        __syncwarp();
        if (one) {
          mbar_arrive(x ? &c.v_full : &c.k_full);
          mbar_arrive(&c.raw_free[x][t % kRaw]);
        }
      }
      last = g, col = it.col;
    }
  }
}

// ------------------------------------------------------------------ products
// One thread.  8 columns of tensor memory are 16 elements of a query's first
// parts, D/2 columns on are the second ones; of the weights the first and
// second parts of 16 positions follow one another.
template <int kD>
__device__ bool products(const PromptParams &p, Control &c, uint32_t smem) {
  using S = Shape<kD>;
  constexpr int kPos = S::kPos;
  constexpr uint32_t kScores = mma_f16_shape<kPos, false>(), kValues = mma_f16_shape<kCols, true>();
  const uint32_t tm = c.tmem;
  Item it;
  for (int m = 0; item_at<false>(p, c, m, it); ++m) {
    mbar_arrive(&c.item_free[m % kItems]);
    const int n = it.tiles;
    if (!wait(&c.q_full, m & 1, p.err, DEVERR_FULL_WAIT, m)) return false;
#pragma unroll 1
    for (int i = 0; i <= n; ++i) {
      if (i < n) {
        const int g = it.before + i;
        if (!wait(&c.k_full, g & 1, p.err, DEVERR_FULL_WAIT, g)) return false;
        tmem_fence_after();
        const uint32_t d = tm + S::kS + (g & 1) * kPos;
        // the small products first
#pragma unroll 1
        for (int x = 0; x < 3; ++x) {
          const uint32_t a = tm + S::kQ + (x == 0 ? kD / 2 : 0);
          const uint64_t b = mma_b_descriptor(smem + (x == 1 ? S::kKPart : 0), 16);
#pragma unroll
          for (int k = 0; k < kD / 16; ++k)
            mma_f16(d, a + 8 * k, b + ((k / 4) * (kPos * 128) + (k % 4) * 32) / 16, kScores, x + k > 0);
        }
        mma_commit(&c.s_full[g & 1]);
      }
      if (i > 0) {
        const int g = it.before + i - 1;
        if (!wait(&c.v_full, g & 1, p.err, DEVERR_FULL_WAIT, g)) return false;
        if (!wait(&c.p_full[g & 1], (g >> 1) & 1, p.err, DEVERR_FULL_WAIT, g)) return false;
        if (g > 0 && !wait(&c.t_free, (g - 1) & 1, p.err, DEVERR_EMPTY_WAIT, g)) return false;
        tmem_fence_after();
#pragma unroll 1
        for (int x = 0; x < 3; ++x) {
          const uint32_t a = tm + S::kS + (g & 1) * kPos + (x == 0 ? 8 : 0);
          const uint64_t b = mma_b_descriptor(smem + S::kV + (x == 1 ? S::kVPart : 0), kPos * 128);
#pragma unroll
          for (int k = 0; k < kPos / 16; ++k) mma_f16(tm + S::kT, a + 16 * k, b + k * 2048 / 16, kValues, x + k > 0);
        }
        mma_commit(&c.t_full);
      }
    }
  }
  return true;
}

template <int kD>
__device__ void products_role(const PromptParams &p, Control &c, uint32_t smem) {
  products<kD>(p, c, smem);
  // no product is in flight when the tensor memory is given back
  mma_commit(&c.drain);
  wait(&c.drain, 0, p.err, DEVERR_DRAIN_WAIT);
}

// ------------------------------------------------------------------ weights
// Two float32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t x, y, z;
  float2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(z) : "f"(c.x), "f"(c.y));
  asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(x) : "l"(y), "l"(z));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}

// A pair of weights as two fp16 parts each: the 11 leading bits, and the rest rounded.
__device__ __forceinline__ void split_weights(float2 w, uint32_t &first, uint32_t &rest) {
  const float2 a = make_float2(__uint_as_float(__float_as_uint(w.x) & 0xffffe000u),
                               __uint_as_float(__float_as_uint(w.y) & 0xffffe000u));
  const float2 b = fma2(a, make_float2(-1.0f, -1.0f), w);
  first = pack_half2(a.x, a.y);
  rest = pack_half2(b.x, b.y);
}

// The queries of an item's rows in two parts; what undoes a row's scale goes to
// c.row_mul.  Four threads share a row: a thread for each row would touch 32
// lines with every read.
template <int kD>
__device__ __forceinline__ void queries(const PromptParams &p, Control &c, const Item &it) {
  using S = Shape<kD>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, mine = 4 * (lane & 3);
#pragma unroll 1
  for (int half = 0; half < 2; ++half) {
    const int row0 = 32 * warp + 16 * half + (lane >> 2);  // and 8 rows on
    const float *q[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = it.rt * kRows + row0 + 8 * i;
      q[i] = r < it.rows ? p.q + it.s * p.q_seq_ld + r / p.group * p.q_ld + (it.h * p.group + r % p.group) * kD + mine : nullptr;
    }
    float4 x[2][8];
    const auto load = [&](int col) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k)
          x[i][k] = q[i] ? *reinterpret_cast<const float4 *>(q[i] + col + 16 * k) : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    float big[2] = {};
#pragma unroll 1
    for (int col = 0; col < kD; col += 128) {
      load(col);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k)
          big[i] = fmaxf(fmaxf(big[i], fmaxf(fabsf(x[i][k].x), fabsf(x[i][k].y))), fmaxf(fabsf(x[i][k].z), fabsf(x[i][k].w)));
    }
    int up[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      big[i] = fmaxf(big[i], __shfl_xor_sync(0xffffffffu, big[i], 1));
      big[i] = fmaxf(big[i], __shfl_xor_sync(0xffffffffu, big[i], 2));
      up[i] = big[i] > 0.0f ? 14 - max(static_cast<int>(__float_as_uint(big[i]) >> 23) - 127, -126) : 0;
      if (mine == 0) c.row_mul[row0 + 8 * i] = scale_pow2(p.scale, -up[i]) * 1.44269504088896f;
    }
    const uint32_t to = c.tmem + S::kQ + (static_cast<uint32_t>(32 * warp + 16 * half) << 16);
#pragma unroll 1
    for (int col = 0; col < kD; col += 128) {
      if (kD > 128) load(col);
#pragma unroll
      for (int k0 = 0; k0 < 8; k0 += 4) {
        uint32_t first[16], rest[16];
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float4 a = x[i][k0 + k];
            const int u = 4 * k + 2 * i;
            split2(scale_pow2(a.x, up[i]), scale_pow2(a.y, up[i]), first[u], rest[u]);
            split2(scale_pow2(a.z, up[i]), scale_pow2(a.w, up[i]), first[u + 1], rest[u + 1]);
          }
        tmem_store_quads(to + col / 2 + 8 * k0, first);
        tmem_store_quads(to + kD / 2 + col / 2 + 8 * k0, rest);
      }
    }
  }
}

template <int kD>
__device__ void weights_role(const PromptParams &p, Control &c) {
  using S = Shape<kD>;
  constexpr int kPos = S::kPos;
  const int row = threadIdx.x;
  const uint32_t tm = c.tmem + (static_cast<uint32_t>(row & ~31) << 16);
  Item it;
  for (int n = 0; item_at(p, c, n, it); ++n) {
    item_done(c, n);
    // All scores of the item before have been seen: nothing reads its queries any more.
    queries<kD>(p, c, it);
    tmem_wait_stores();
    tmem_fence_before();
    mbar_arrive(&c.q_full);
    __syncwarp();
    const float row_mul = c.row_mul[row];
    const int at = it.len + min((it.rt * kRows + row) / p.group, it.t1), low = p.window ? at - p.window + 1 : 0;
    float top = -INFINITY, off = 0.0f, den = 0.0f;  // weights are exp2(x - off): 2^15 at the maximum
#pragma unroll 1
    for (int k = 0; k < it.tiles; ++k) {
      const int g = it.before + k, p0 = (it.from & -kPos) + k * kPos;
      const uint32_t s = tm + S::kS + (g & 1) * kPos;
      if (!wait_warp(&c.scan_full[g % kAhead], (g / kAhead) & 1, p.err, DEVERR_FULL_WAIT, g)) return;
      const Entry &e = c.entry[g % kAhead];
      float mul = row_mul * e.kmul;
      // some position of the tile is not for all rows
      const bool masked =
          p0 + kPos - 1 > it.len + it.t0 || (p.window && p0 <= it.len + it.t1 - p.window) || e.any;
      if (!wait_warp(&c.s_full[g & 1], (g >> 1) & 1, p.err, DEVERR_FULL_WAIT, g)) return;
      tmem_fence_after();
      float up_to = -INFINITY;
      if (masked) {
        // the scores as they count, over the products
#pragma unroll 1
        for (int j0 = 0; j0 < kPos; j0 += 16) {
          uint32_t x[16];
          tmem_load16(s + j0, x);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int pos = p0 + j0 + j;
            const float y = pos >= low && pos <= at ? fmaf(__uint_as_float(x[j]), mul, e.lost[j0 + j]) : -INFINITY;
            up_to = fmaxf(up_to, y);
            x[j] = __float_as_uint(y);
          }
          tmem_store16(s + j0, x);
        }
        tmem_wait_stores();
        mul = 1.0f;
      } else {
        float m2[2] = {-INFINITY, -INFINITY};
#pragma unroll 1
        for (int j0 = 0; j0 < kPos; j0 += 32) {
          uint32_t x[32];
          tmem_load32(s + j0, x);
#pragma unroll
          for (int j = 0; j < 32; j += 2)
            m2[(j >> 1) & 1] = fmaxf(fmaxf(m2[(j >> 1) & 1], __uint_as_float(x[j])), __uint_as_float(x[j + 1]));
        }
        up_to = __fmul_ru(fmaxf(m2[0], m2[1]), mul);  // rounded up, so that no weight passes 2^15
      }
      float keep = 1.0f;
      if (up_to > top) {
        const float now = __fadd_ru(up_to, -15.0f);
        keep = top == -INFINITY ? 0.0f : exp2_approx(off - now);
        top = up_to, off = now;
      }
      c.corr[g % kAhead][row] = keep;
      const float2 mul2 = make_float2(mul, mul), off2 = make_float2(-off, -off);
      float2 sum2 = {};
#pragma unroll 1
      for (int j0 = 0; j0 < kPos; j0 += 16) {
        uint32_t x[16], y[16];
        tmem_load16(s + j0, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float2 v = fma2(make_float2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])), mul2, off2);
          v.x = exp2_approx(v.x), v.y = exp2_approx(v.y);
          sum2 = fma2(v, make_float2(1.0f, 1.0f), sum2);
          split_weights(v, y[j], y[8 + j]);
        }
        tmem_store16(s + j0, y);
      }
      const float sum = sum2.x + sum2.y;
      den = fmaf(den, keep, sum);
      tmem_wait_stores();
      tmem_fence_before();
      mbar_arrive(&c.c_full[g % kAhead]);
      mbar_arrive(&c.p_full[g & 1]);
    }
    if (n > 0 && !wait_warp(&c.fin_empty, (n - 1) & 1, p.err, DEVERR_EMPTY_WAIT, n)) return;
    c.off[row] = top == -INFINITY ? -INFINITY : off;
    c.den[row] = den;
    mbar_arrive(&c.fin_full);
  }
}

// ------------------------------------------------------------------ output
template <int kD>
__device__ void output_role(const PromptParams &p, Control &c) {
  using S = Shape<kD>;
  const int row = threadIdx.x & 127;
  const uint32_t tm = c.tmem + (static_cast<uint32_t>(row & ~31) << 16) + S::kT;
  for (int n = 0;; ++n) {
    if (!wait_warp(&c.item_full[n % kItems], (n / kItems) & 1, p.err, DEVERR_FULL_WAIT, n)) return;
    const Item &it = c.item[n % kItems];  // kept until the end
    const int tiles = it.tiles, begin = it.before;
    if (tiles == 0) return;
    float2 o[kCols / 2];
#pragma unroll
    for (int i = 0; i < kCols / 2; ++i) o[i] = make_float2(0.0f, 0.0f);
#pragma unroll 1
    for (int g = begin; g < begin + tiles; ++g) {
      if (!wait_warp(&c.c_full[g % kAhead], (g / kAhead) & 1, p.err, DEVERR_FULL_WAIT, g)) return;
      const float keep = c.corr[g % kAhead][row];
      const Entry &e = c.entry[g % kAhead];
      float mul[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) mul[b] = e.vmul[b];
      if (!wait_warp(&c.t_full, g & 1, p.err, DEVERR_FULL_WAIT, g)) return;
      tmem_fence_after();
      if (!__all_sync(0xffffffffu, keep == 1.0f)) {
        const float2 keep2 = make_float2(keep, keep), none = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < kCols / 2; ++i) o[i] = fma2(o[i], keep2, none);
      }
#pragma unroll
      for (int j = 0; j < kCols; j += 16) {
        uint32_t x[16];
        tmem_load16(tm + j, x);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          o[j / 2 + i] = fma2(make_float2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])),
                              make_float2(mul[j / 32], mul[j / 32]), o[j / 2 + i]);
      }
      tmem_fence_before();
      mbar_arrive(&c.t_free);
      mbar_arrive(&c.entry_free[g % kAhead]);
    }
    if (!wait_warp(&c.fin_full, n & 1, p.err, DEVERR_FULL_WAIT, n)) return;
    const float off = c.off[row], den = c.den[row];
    mbar_arrive(&c.fin_empty);
    const int r = it.rt * kRows + row;
    float scale = 1.0f;
    float4 *to = nullptr;
    if (it.slot >= 0) {
      to = reinterpret_cast<float4 *>(p.parts + (static_cast<int64_t>(2 * blockIdx.x + it.slot) * kRows + row) * kPartLd);
      to[kCols / 4] = make_float4(off, den, 0.0f, 0.0f);
    } else if (r < it.rows) {
      to = reinterpret_cast<float4 *>(p.out + (static_cast<int64_t>(it.s) * p.ntok + r / p.group) * p.n_heads * kD +
                                      (it.h * p.group + r % p.group) * kD + it.col);
      scale = den != 0.0f ? __fdiv_rn(1.0f, den) : 0.0f;
    }
    if (to) {
#pragma unroll
      for (int i = 0; i < kCols / 4; ++i)
        to[i] = make_float4(o[2 * i].x * scale, o[2 * i].y * scale, o[2 * i + 1].x * scale, o[2 * i + 1].y * scale);
    }
    item_done(c, n);
  }
}

template <int kD>
__global__ void __launch_bounds__(kThreads, 1) prompt_kernel(const __grid_constant__ PromptParams p) {
  using S = Shape<kD>;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  const uint32_t pad = (1024 - (smem_addr(smem_raw) & 1023)) & 1023;
  uint8_t *smem = smem_raw + pad;
  Control &c = *reinterpret_cast<Control *>(smem + S::kBytes);
  const int tid = threadIdx.x, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c.s_full[i], 1);
      mbar_init(&c.p_full[i], 128);
    }
    for (int i = 0; i < 2 * kRaw; ++i) {
      mbar_init(&c.raw_full[i / kRaw][i % kRaw], 1);
      mbar_init(&c.raw_free[i / kRaw][i % kRaw], 8);
    }
    mbar_init(&c.k_full, 8);
    mbar_init(&c.v_full, 8);
    mbar_init(&c.drain, 1);
    mbar_init(&c.t_full, 1);
    mbar_init(&c.t_free, 128);
    mbar_init(&c.q_full, 128);
    mbar_init(&c.fin_full, 128);
    mbar_init(&c.fin_empty, 128);
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&c.item_full[i], 1);
      mbar_init(&c.item_free[i], kThreads / 32);
    }
    for (int i = 0; i < kAhead; ++i) {
      mbar_init(&c.c_full[i], 128);
      mbar_init(&c.scan_full[i], 2);
      mbar_init(&c.entry_free[i], 128);
    }
    fence_mbar_init();
  }
  pdl_launch_dependents();
  pdl_wait();
  find_work<kD>(p, c);  // with CTA barriers
  const bool work = c.begin < c.end;
  if (work && warp == 16) tmem_alloc(&c.tmem);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (warp < 4) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsWeights));
    if (work) weights_role<kD>(p, c);
  } else if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsOutput));
    if (work) output_role<kD>(p, c);
  } else if (warp < 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOperand));
    if (work) operands_role<kD>(p, c, smem);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    if (warp == 16) {
      if (work && (tid & 31) == 0) products_role<kD>(p, c, smem_addr(smem));
      __syncwarp();
    } else if (warp == 17) {
      if ((tid & 31) == 0) p.notes[2 * blockIdx.x] = p.notes[2 * blockIdx.x + 1] = Part{};
      if (work) copies_role<kD>(p, c, smem);
      // tokens beyond a sequence's have an output of 0
      if (p.n_tok) {
        const int width = p.n_heads * kD;
        for (int64_t r = blockIdx.x; r < static_cast<int64_t>(p.v.n_seq) * p.ntok; r += gridDim.x) {
          if (r % p.ntok < c.seq[r / p.ntok].y) continue;
          float4 *o = reinterpret_cast<float4 *>(p.out + r * width);
          for (int i = tid & 31; i < width / 4; i += 32) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
    } else {
      if (work) scan_role<kD>(p, c);
    }
  }
  tmem_fence_before();
  __syncthreads();
  if (work && warp == 16) {
    tmem_fence_after();
    tmem_free(c.tmem);
  }
}

// The parts of an item, joined in the order of their positions: block x is the
// CTA that holds an item's first part, block y a group of rows, a warp a row.
template <int kD>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const __grid_constant__ PromptParams p, int ctas) {
  pdl_launch_dependents();
  pdl_wait();
  const int c0 = blockIdx.x, lane = threadIdx.x & 31, row = blockIdx.y * kJoinWarps + (threadIdx.x >> 5);
  const auto heads = [](const Part &x) { return x.tiles > 0 && x.a == 0 && x.b < x.tiles; };
  int slot = 2 * c0;
  Part x = p.notes[slot];
  if (!heads(x)) x = p.notes[++slot];
  if (!heads(x)) return;
  const int r = x.rt * kRows + row, n = p.n_tok ? min(max(p.n_tok[x.s], 0), p.ntok) : p.ntok;
  if (r >= n * p.group) return;
  float top = -INFINITY, den = 0.0f;
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
  int upto = x.b;
  for (int c = c0;; slot = 2 * ++c) {
    if (c > c0) {  // the item goes on at the start of the next CTA's share
      if (c >= ctas || upto >= x.tiles) break;
      upto = p.notes[slot].b;
    }
    const float *from = p.parts + (static_cast<int64_t>(slot) * kRows + row) * kPartLd;
    const float2 ml = *reinterpret_cast<const float2 *>(from + kCols);
    const float4 a = reinterpret_cast<const float4 *>(from)[lane];
    const float up = fmaxf(top, ml.x), ref = up == -INFINITY ? 0.0f : up;
    const float keep = exp2f(top - ref), f = exp2f(ml.x - ref);  // 0 for a part that saw nothing
    top = up;
    den = fmaf(den, keep, f * ml.y);
    y = make_float4(fmaf(f, a.x, y.x * keep), fmaf(f, a.y, y.y * keep), fmaf(f, a.z, y.z * keep), fmaf(f, a.w, y.w * keep));
  }
  const int h = x.y / Shape<kD>::kSplit, split = x.y % Shape<kD>::kSplit;
  float4 *to = reinterpret_cast<float4 *>(p.out + (static_cast<int64_t>(x.s) * p.ntok + r / p.group) * p.n_heads * kD +
                                          (h * p.group + r % p.group) * kD + split * kCols);
  to[lane] = den != 0.0f ? make_float4(y.x / den, y.y / den, y.z / den, y.w / den) : make_float4(0.f, 0.f, 0.f, 0.f);
}

bool sizes_ok(const epq_pages *pages, int n_heads, int ntok) {
  return pages_sizes_ok(pages) && n_heads >= 1 && n_heads % pages->n_kv_heads == 0 &&
         n_heads / pages->n_kv_heads <= kMaxGroupPrompt && ntok >= 1 &&
         static_cast<int64_t>(pages->n_seq) * ntok < (1 << 24);
}

template <int kD>
cudaError_t launch(const PromptParams &p, const DeviceInfo &dev, cudaStream_t s) {
  static LaunchOnce once;
  const size_t smem = 1024 + Shape<kD>::kBytes + sizeof(Control);
  cudaError_t e = once.prepare(dev.device, prompt_kernel<kD>, kThreads, smem, false, nullptr);
  const int ctas = std::min(dev.sm_count, kMaxCtas);
  if (e == cudaSuccess) e = launch_pdl(prompt_kernel<kD>, dim3(ctas), dim3(kThreads), smem, s, p);
  if (e == cudaSuccess)
    e = launch_pdl(join_kernel<kD>, dim3(ctas, kRows / kJoinWarps), dim3(32 * kJoinWarps), 0, s, p, ctas);
  return e;
}

}  // namespace
}  // namespace epq

using namespace epq;

extern "C" size_t epq_attention_prompt_workspace_bytes(const epq_pages *pages, int n_heads, int ntok) {
  return sizes_ok(pages, n_heads, ntok) ? 2 * kMaxCtas * (sizeof(Part) + 4 * kRows * kPartLd) : 0;
}

extern "C" epq_status epq_attention_prompt(const epq_pages *pages, int layer, const float *q, int n_heads, int ntok,
                                           float scale, const epq_attention_prompt_opts *opts, float *out, void *ws,
                                           size_t ws_bytes, epq_stream_t stream) {
  static const epq_attention_prompt_opts kNone = {};
  const epq_attention_prompt_opts &o = opts ? *opts : kNone;
  PromptParams p;
  const epq_status st = pages_view(pages, &p.v);
  if (st != EPQ_OK) return st;
  if (!q || !out || layer < 0 || layer >= p.v.n_layers || !(scale > 0.0f) || !std::isfinite(scale) || o.window < 0)
    return EPQ_ERR_ARG;
  if (!sizes_ok(pages, n_heads, ntok)) return EPQ_ERR_SHAPE;
  p.q_ld = o.q_ld ? o.q_ld : static_cast<int64_t>(n_heads) * p.v.D;
  p.q_seq_ld = o.q_seq_ld ? o.q_seq_ld : ntok * p.q_ld;
  if (o.q_ld < 0 || o.q_seq_ld < 0) return EPQ_ERR_ARG;
  if (!aligned16(q) || !aligned16(out) || p.q_ld % 4 || p.q_seq_ld % 4 || !aligned_to(4, o.n_tok)) return EPQ_ERR_ALIGN;
  if (!ws || ws_bytes < epq_attention_prompt_workspace_bytes(pages, n_heads, ntok)) return EPQ_ERR_WORKSPACE;
  if (!aligned16(ws)) return EPQ_ERR_ALIGN;
  // in place: a row's queries are read before its output is written, but both
  // halves of the output of heads of 256 are items that read the whole row
  const int64_t width = static_cast<int64_t>(n_heads) * p.v.D;
  if (q == out && (p.v.D != kCols || p.q_ld != width || p.q_seq_ld != ntok * width)) return EPQ_ERR_ARG;
  p.q = q, p.n_tok = o.n_tok, p.layer = layer, p.n_heads = n_heads, p.group = n_heads / p.v.n_kv, p.ntok = ntok;
  p.window = o.window, p.scale = scale, p.out = out;
  p.notes = static_cast<Part *>(ws);
  p.parts = reinterpret_cast<float *>(p.notes + 2 * kMaxCtas);
  DeviceInfo dev;
  if (!current_device(&dev) || dev.major * 10 + dev.minor != 103) return EPQ_ERR_DEVICE;
  p.err = device_error_slot();
  if (!p.err) return EPQ_ERR_DEVICE;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = p.v.D == 128 ? launch<128>(p, dev, s) : launch<256>(p, dev, s);
  return e == cudaSuccess ? EPQ_OK : cuda_fail(e);
}
